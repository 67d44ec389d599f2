"""Build libraattn.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ is compiled in parallel to an object file in
_build/, then linked into rational_softmax_attention_gb300/libraattn.so.  The
CUDA runtime is linked statically, so the library needs only the driver at run
time.  csrc/calls.c becomes _calls.so beside it, a Python module over the serving
calls; without Python's headers it is left out, and ctypes makes those calls too.  `python -m rational_softmax_attention_gb300.build` runs it by hand.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libraattn.so")
CALLS_PATH = os.path.join(PKG_DIR, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "calls.c")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libraattn")
    return path


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src):
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = os.path.join(BUILD_DIR, os.path.basename(src) + ".log")
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr[-4000:]}")
    return obj


def _stale(srcs):
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = srcs + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    deps.append(os.path.join(ROOT, "include", "raattn.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _build_calls(force):
    headers = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(headers, "Python.h")):
        return
    deps = [CALLS_SRC, LIB_PATH, os.path.join(ROOT, "include", "raattn.h")]
    if not force and os.path.exists(CALLS_PATH) and os.path.getmtime(CALLS_PATH) >= max(map(os.path.getmtime, deps)):
        return
    tmp = CALLS_PATH + ".tmp"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-shared", "-fPIC", "-I", headers, "-I", os.path.join(ROOT, "include"),
           CALLS_SRC, "-o", tmp, "-L", PKG_DIR, "-l:libraattn.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"gcc failed on {CALLS_SRC}:\n{res.stderr[-4000:]}")
    os.replace(tmp, CALLS_PATH)


def build(force=False, verbose=False):
    """Compile and link libraattn.so and _calls.so; returns the former's path.  Skips what is up to date."""
    path = _build_lib(force, verbose)
    _build_calls(force)
    return path


def _build_lib(force, verbose):
    srcs = _sources()
    if not force and not _stale(srcs):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr[-4000:]}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        for src in srcs:
            with open(os.path.join(BUILD_DIR, os.path.basename(src) + ".log")) as f:
                sys.stdout.write(f.read())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
