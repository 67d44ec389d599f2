"""Every kernel launch's own status is read before another launch of the same function, or its end: a launch
that failed otherwise passes for one that ran, and what follows reads a workspace that nobody wrote.
cudaLaunchKernelEx returns the status of its own launch alone, so it does not stand in for an earlier one's.
Read from the sources: no valid argument makes a single launch of a call fail."""
import os
import re

import pytest

import rational_softmax_attention_gb300 as ra

CSRC = os.path.join(os.path.dirname(ra.__file__), "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))
LAUNCH = re.compile(r"<<<[^;]*?>>>\s*\([^;]*\);", re.S)


def code(text):
    return re.sub(r"//[^\n]*", "", text)


def unread_launches(text):
    """Triple-bracket launches that another launch, or the end of the function, follows first."""
    text = code(text)
    marks = [(m.end(), "launch") for m in LAUNCH.finditer(text)]
    marks += [(m.start(), "read") for m in re.finditer(r"cudaGetLastError\s*\(", text)]
    marks += [(m.start(), "other") for m in re.finditer(r"launch_dependent\s*\(|cudaLaunchKernelEx\s*\(", text)]
    marks += [(m.start(), "end") for m in re.finditer(r"^}", text, re.M)]
    marks.sort()
    bad = []
    for i, (at, kind) in enumerate(marks):
        if kind != "launch":
            continue
        # branches of one choice: launches that no statement of their own separates
        after = [k for _, k in marks[i + 1:] if k != "launch"]
        if not after or after[0] != "read":
            bad.append(text[:at].rsplit("\n", 1)[-1].strip())
    return bad


# a launcher without a status of its own; its caller reads it at once
CALLER_READS = {"norm_rope_fwd.cu"}


@pytest.mark.parametrize("name", [s for s in SOURCES if s not in CALLER_READS])
def test_every_launch_has_its_status_read(name):
    with open(os.path.join(CSRC, name)) as f:
        assert unread_launches(f.read()) == []


def test_the_forward_of_the_norm_reads_it_in_the_caller():
    with open(os.path.join(CSRC, "norm_rope_fwd.cu")) as f:
        text = code(f.read())
    last = text[text.index("cudaError_t launch_norm_rope_fwd"):]
    assert "<<<" not in last and re.search(r"go<float, 128>.*return cudaGetLastError\(\);", last, re.S)
    assert len(re.findall(r"\bgo<", text)) == 8 and "launch_dependent" not in text


def test_the_reading_finds_what_it_looks_for():
    assert unread_launches("void f() {\n  k<<<1, 2>>>(a);\n  launch_dependent(j, 1);\n}\n") == ["k<<<1, 2>>>(a);"]
    assert unread_launches("void f() {\n  k<<<1, 2>>>(a);\n}\nint g() {\n  return cudaGetLastError();\n}\n") == ["k<<<1, 2>>>(a);"]
    assert unread_launches("int f() {\n  if (x) k<<<1, 2>>>(a);\n  else j<<<1, 2>>>(b);\n  return cudaGetLastError();\n}\n") == []
