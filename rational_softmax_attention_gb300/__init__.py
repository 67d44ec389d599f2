"""Python binding of libraattn: rational-softmax (Ra-family) attention on GB300.

Argument marshalling only.  Every computation runs in the CUDA kernels of
libraattn.so, reached through its C ABI (include/raattn.h) with ctypes; torch
provides device memory and the current stream.  There is no CPU path: when the
library is not built, or the tensors are not on a CUDA device, the calls raise.

Functional API, after the page "Ra-Family: Rational Neural Architecture",
section 3 "Rational Attention & Softmax":
    ra_softmax(x)                                   last-dim rational soft-argmax
    ra_attention(q, k, v, attn_mask=None, is_causal=False, scale=None)   drop-in for SDPA, autograd-aware
around it, for positions and for serving (serving.py):
    ra_qk_norm_rope(qkv, ...)          per-head norm and rotation of q and k, autograd-aware
    ra_cache_append, ra_attention_decode, ra_cache_evict, RaCache        single tokens against a cache
plus the explicit forward/backward entry points used by tests and benchmarks.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

__all__ = [
    "RaError", "lib", "ra_softmax", "ra_softmax_backward", "ra_attention", "ra_attention_forward", "RaAttention",
    "ra_attention_backward", "pack_attn_mask", "device_status", "set_wait_limit_ns", "exported_symbols", "LIB_PATH",
    "debug_kernel_events", "ra_rope_frequencies", "ra_qk_norm_rope", "ra_qk_norm_rope_backward", "ra_cache_append",
    "ra_attention_decode", "ra_cache_evict", "RaCache",
]

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libraattn.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "raattn.h")

RA_F32, RA_BF16 = 0, 1
_STATUS = {0: "RA_OK", 1: "RA_ERR_ARG", 2: "RA_ERR_UNSUPPORTED", 3: "RA_ERR_LAUNCH", 4: "RA_ERR_TIMEOUT"}


class RaError(RuntimeError):
    """A libraattn call returned a status other than RA_OK."""

    def __init__(self, fn, code, text):
        super().__init__(f"{fn}: {text} (status {code})")
        self.code = code


_lib = None
_vp, _i64, _i32, _f32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_uint64

_SIGNATURES = {
    "ra_status_string": ([_i32], ctypes.c_char_p),
    "ra_softmax_fwd": ([_vp, _vp, _i64, _i64, _i32, _vp], _i32),
    "ra_softmax_bwd": ([_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp], _i32),
    "ra_attention_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                          _i32, _i32, _vp], _i32),
    "ra_attention_fwd_workspace_size": ([_i32, _i32, _i32, _i32, _i32], ctypes.c_size_t),
    "ra_attention_bwd_workspace_size": ([_i32, _i32, _i32, _i32, _i32], ctypes.c_size_t),
    "ra_attention_bwd": ([_vp] * 12 + [_i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _i32, _vp], _i32),
    "ra_attention_mask_words": ([_i32], _i32),
    "ra_attention_mask_pack": ([_vp, _i32, _i32, _i32, _vp, _vp, _vp], _i32),
    "ra_attention_fwd_masked": ([_vp] * 9 + [_i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp, _i32, _i32,
                                               _vp], _i32),
    "ra_attention_bwd_masked": ([_vp] * 12 + [_i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _i32, _vp, _vp,
                                                _i32, _i32, _vp], _i32),
    "ra_qk_norm_rope_fwd": ([_vp, _i64, _i64] + [_vp] * 4 + [_i32, _f32, _vp, _vp, _i64, _i64, _vp, _i32, _i32]
                            + [_vp] * 5 + [_i32] * 7 + [_vp], _i32),
    "ra_qk_norm_rope_bwd_workspace_size": ([_i32], ctypes.c_size_t),
    "ra_qk_norm_rope_bwd": ([_vp, _i64, _i64] + [_vp] * 4 + [_i32, _f32, _vp, _vp, _i64, _i64, _vp, _i32, _i32]
                            + [_vp] * 6 + [_i32] * 6 + [_vp], _i32),
    "ra_attention_decode_workspace_size": ([_i32] * 7, ctypes.c_size_t),
    "ra_attention_decode": ([_vp] * 9 + [_i32] * 6 + [_f32, _i32, _vp], _i32),
    "ra_cache_evict": ([_vp] * 9 + [_i32] * 8 + [_vp], _i32),
    "ra_device_status": ([_vp], _i32),
    "ra_set_wait_limit_ns": ([_u64], None),
    "ra_debug_force_timeout": ([_i32], None),
    "ra_debug_fwd_pair": ([_i32], None),
    "ra_debug_kernel_events": ([ctypes.POINTER(ctypes.c_void_p), _i32], None),
}


def lib():
    """The loaded libraattn (ctypes.CDLL).  Raises if the library has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libraattn.so is not built ({LIB_PATH}); run "
                               "`python -m rational_softmax_attention_gb300.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def exported_symbols():
    """Names of the functions include/raattn.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w]*\**\s+\**(ra_\w+)\s*\(", text, re.M)))


def _check(fn, code):
    if code != 0:
        raise RaError(fn, code, lib().ra_status_string(code).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(dt):
    if dt == torch.float32:
        return RA_F32
    if dt == torch.bfloat16:
        return RA_BF16
    raise TypeError(f"unsupported dtype {dt}: libraattn takes float32 or bfloat16")


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libraattn takes contiguous CUDA tensors (there is no CPU path)")


def _require_attention(q, k, v, mask):
    """The kernels take B, H and the dtype from q alone and read k, v and the mask by them."""
    s, t = q.shape, k.shape
    if len(s) != 4 or len(t) != 4 or t[0] != s[0] or t[1] != s[1] or t[3] != s[3] or v.shape != t:
        raise ValueError("q must be [B, H, N_Q, D] and k and v both [B, H, N_K, D], with as many heads as q, not "
                         f"{list(q.shape)}, {list(k.shape)} and {list(v.shape)}")
    _require_like(q.dtype, q.device, k=k, v=v)
    if mask is None:
        return
    mask_q, mask_k, MB, MH = mask
    (B, H, n_q, _), n_k, words = q.shape, k.shape[2], lib().ra_attention_mask_words
    if MB not in (1, B) or MH not in (1, H) or mask_q.shape != (MB * MH, n_q, words(n_k)) \
            or mask_k.shape != (MB * MH, n_k, words(n_q)):
        raise ValueError("mask must come from pack_attn_mask for these sizes")
    _require_like(torch.int32, q.device, mask_q=mask_q, mask_k=mask_k)
    _require_cuda(mask_q, mask_k)


def _require_like(dtype, device, **tensors):
    for name, t in tensors.items():
        if t.dtype != dtype or t.device != device:
            raise ValueError(f"{name} must be {dtype} on {device}, not {t.dtype} on {t.device}")


def ra_softmax(x):
    """ra_softmax along the last dimension of a float32 or bfloat16 CUDA tensor (same dtype out)."""
    _require_cuda(x)
    y = torch.empty_like(x)
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    _check("ra_softmax_fwd", lib().ra_softmax_fwd(_ptr(x), _ptr(y), rows, cols, _dtype_code(x.dtype),
                                                   _stream(x.device)))
    return y


def ra_softmax_backward(x, p, dy, out=None):
    """Closed-form gradient of sum(dy * ra_softmax(x)) with respect to x (last dimension).

    out: optional tensor for dx, shaped like x; it may be dy itself (gradient in place)."""
    _require_cuda(x, p, dy)
    if p.dtype != x.dtype or dy.dtype != x.dtype or p.shape != x.shape or dy.shape != x.shape:
        raise ValueError("x, p and dy must share one shape and dtype (float32 or bfloat16)")
    if out is not None:
        _require_cuda(out)
        if out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor shaped like x")
    dx = torch.empty_like(x) if out is None else out
    cols = x.shape[-1]
    rows = x.numel() // cols
    _check("ra_softmax_bwd", lib().ra_softmax_bwd(_ptr(x), _ptr(p), _ptr(dy), _ptr(dx), rows, cols,
                                                   _dtype_code(x.dtype), _stream(x.device)))
    return dx


def pack_attn_mask(attn_mask, B, H, n_q, n_k):
    """Bit-packs a boolean attn_mask broadcastable to [B, H, N_Q, N_K] (True = the query may
    attend to the key, as in scaled_dot_product_attention) for the masked attention calls.

    Returns (mask_q, mask_k, MB, MH): the packed mask with a row per query and with a row
    per key, and how many batch and head entries it has (1 = shared)."""
    if attn_mask.dtype != torch.bool:
        raise NotImplementedError("only boolean attention masks are supported")
    _require_cuda(attn_mask.contiguous())
    m = attn_mask
    while m.dim() < 4:
        m = m.unsqueeze(0)
    if m.dim() != 4:
        raise ValueError("attn_mask must broadcast to [B, H, N_Q, N_K]")
    MB, MH = m.shape[0], m.shape[1]
    if MB not in (1, B) or MH not in (1, H):
        raise ValueError("attn_mask must broadcast to [B, H, N_Q, N_K]")
    m8 = m.expand(MB, MH, n_q, n_k).contiguous().view(torch.uint8)
    L = lib()
    mask_q = torch.empty((MB * MH, n_q, L.ra_attention_mask_words(n_k)), dtype=torch.int32, device=m.device)
    mask_k = torch.empty((MB * MH, n_k, L.ra_attention_mask_words(n_q)), dtype=torch.int32, device=m.device)
    _check("ra_attention_mask_pack", L.ra_attention_mask_pack(_ptr(m8), MB * MH, n_q, n_k, _ptr(mask_q),
                                                                _ptr(mask_k), _stream(m.device)))
    return mask_q, mask_k, MB, MH


def ra_attention_forward(q, k, v, *, scale=None, causal=False, out_dtype=None, with_stats=True,
                         tile_counts=False, mask=None):
    """O = ra_softmax(scale q k^T [causal] [mask]) v for [B, H, N, D] tensors.

    mask: None, or the tuple pack_attn_mask returns (bf16 inputs only).
    Returns (o, row_m, row_s, row_arg, counts): the statistics are None unless
    with_stats; counts is an int64 CUDA tensor [pairs visited, pairs skipped]
    when tile_counts, else None.
    """
    _require_attention(q, k, v, mask)
    _require_cuda(q, k, v)
    B, H, NQ, D = q.shape
    NK = k.shape[2]
    out_dtype = out_dtype or q.dtype
    o = torch.empty((B, H, NQ, D), dtype=out_dtype, device=q.device)
    stats = None
    if with_stats:
        stats = (torch.empty((B, H, NQ), dtype=torch.float32, device=q.device),
                 torch.empty((B, H, NQ), dtype=torch.float32, device=q.device),
                 torch.empty((B, H, NQ), dtype=torch.int32, device=q.device))
    counts = torch.empty(2, dtype=torch.int64, device=q.device) if tile_counts else None
    rm, rs, ra = stats if stats else (None, None, None)
    L = lib()
    ws = None
    if q.dtype == torch.bfloat16:
        ws = torch.empty(L.ra_attention_fwd_workspace_size(B, H, NQ, NK, D), dtype=torch.uint8, device=q.device)
    if mask is None:
        _check("ra_attention_fwd", L.ra_attention_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(rm), _ptr(rs), _ptr(ra), _ptr(counts), _ptr(ws),
            B, H, NQ, NK, D, float(scale or 0.0), 1 if causal else 0, _dtype_code(q.dtype), _dtype_code(out_dtype),
            _stream(q.device)))
    else:
        mask_q, _, MB, MH = mask
        _check("ra_attention_fwd_masked", L.ra_attention_fwd_masked(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(rm), _ptr(rs), _ptr(ra), _ptr(counts), _ptr(ws),
            B, H, NQ, NK, D, float(scale or 0.0), 1 if causal else 0, _dtype_code(q.dtype), _dtype_code(out_dtype),
            _ptr(mask_q), MB, MH, _stream(q.device)))
    return o, rm, rs, ra, counts


def ra_attention_backward(q, k, v, o, dout, row_m, row_s, row_arg, *, scale=None, causal=False,
                          grad_dtype=torch.float32, workspace=None, mask=None):
    """Gradients (dq, dk, dv) of sum(dout * O) for the forward that produced o and the row
    statistics; mask as given to that forward."""
    _require_attention(q, k, v, mask)
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must be shaped like q")
    if any(t.shape != q.shape[:3] for t in (row_m, row_s, row_arg)):
        raise ValueError("row_m, row_s and row_arg must be [B, H, N_Q], as the forward gives them")
    _require_like(q.dtype, q.device, dout=dout)
    _require_like(o.dtype, q.device, o=o)
    _require_like(torch.float32, q.device, row_m=row_m, row_s=row_s)
    _require_like(torch.int32, q.device, row_arg=row_arg)
    B, H, NQ, D = q.shape
    NK = k.shape[2]
    L = lib()
    nbytes = L.ra_attention_bwd_workspace_size(B, H, NQ, NK, D)
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace must hold {nbytes} bytes")
        _require_like(workspace.dtype, q.device, workspace=workspace)
    _require_cuda(q, k, v, o, dout, row_m, row_s, row_arg, workspace)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    dq = torch.empty((B, H, NQ, D), dtype=grad_dtype, device=q.device)
    dk = torch.empty((B, H, NK, D), dtype=grad_dtype, device=q.device)
    dv = torch.empty((B, H, NK, D), dtype=grad_dtype, device=q.device)
    if mask is None:
        _check("ra_attention_bwd", L.ra_attention_bwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(row_m), _ptr(row_s), _ptr(row_arg),
            _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, NQ, NK, D, float(scale or 0.0),
            1 if causal else 0, _dtype_code(q.dtype), _dtype_code(o.dtype), _dtype_code(grad_dtype),
            _stream(q.device)))
    else:
        mask_q, mask_k, MB, MH = mask
        _check("ra_attention_bwd_masked", L.ra_attention_bwd_masked(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(row_m), _ptr(row_s), _ptr(row_arg),
            _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, NQ, NK, D, float(scale or 0.0),
            1 if causal else 0, _dtype_code(q.dtype), _dtype_code(o.dtype), _dtype_code(grad_dtype),
            _ptr(mask_q), _ptr(mask_k), MB, MH, _stream(q.device)))
    return dq, dk, dv


class _RaAttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, attn_mask):
        mask = None
        if attn_mask is not None:
            mask = pack_attn_mask(attn_mask, q.shape[0], q.shape[1], q.shape[2], k.shape[2])
        o, rm, rs, ra, _ = ra_attention_forward(q, k, v, scale=scale, causal=causal, out_dtype=q.dtype, mask=mask)
        ctx.save_for_backward(q, k, v, o, rm, rs, ra)
        ctx.causal, ctx.scale, ctx.mask = causal, scale, mask
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, rm, rs, ra = ctx.saved_tensors
        dq, dk, dv = ra_attention_backward(q, k, v, o, do.contiguous().to(q.dtype), rm, rs, ra,
                                           scale=ctx.scale, causal=ctx.causal, grad_dtype=q.dtype, mask=ctx.mask)
        return dq, dk, dv, None, None, None


def ra_attention(q, k, v, attn_mask=None, is_causal=False, scale=None):
    """Rational-softmax attention, a drop-in for scaled_dot_product_attention (no dropout): q [B, H, N_Q, D],
    k and v [B, H, N_K, D] of one dtype, with as many key heads as query heads.

    attn_mask: optional boolean mask broadcastable to [B, H, N_Q, N_K], True where the query
    may attend to the key (bf16 inputs only); combined with is_causal."""
    return _RaAttentionFn.apply(q.contiguous(), k.contiguous(), v.contiguous(), bool(is_causal), scale, attn_mask)


from .serving import (RaCache, ra_attention_decode, ra_cache_append, ra_cache_evict, ra_qk_norm_rope,  # noqa: E402
                      ra_qk_norm_rope_backward, ra_rope_frequencies)


class RaAttention(torch.nn.Module):
    """Multi-head attention with ra_softmax (page "Ra-Family: Rational Neural Architecture",
    section 3, "ra_attention & RaAttention").

    x [B, N, dim] -> one projection to q, k, v of every head ([B, heads, N, dim/heads])
    -> optional layer normalisation of q and k over the head dimension (qk_norm)
    -> optional rotation of q and k by position (rope_sections: pairs of dimensions per position
    axis; with it, norm and rotation are one kernel, ra_qk_norm_rope)
    -> ra_attention (this library's kernels, with autograd) -> heads merged -> output
    projection.  The two projections are plain library GEMMs (torch Linear, cuBLAS).
    Dropout is not part of this path: attn_drop and proj_drop must be 0.

    Serving (causal modules): new_cache, then prefill for a prompt and decode for single tokens.
    """

    def __init__(self, dim, num_heads=8, qkv_bias=False, qk_norm=False, attn_drop=0.0, proj_drop=0.0,
                 causal=False, device=None, dtype=None, rope_sections=None, rope_theta=10000.0,
                 rope_interleaved=False):
        super().__init__()
        if dim % num_heads != 0:
            raise ValueError("dim must be a multiple of num_heads")
        if attn_drop != 0.0 or proj_drop != 0.0:
            raise NotImplementedError("dropout is not supported (attn_drop and proj_drop must be 0)")
        self.num_heads = num_heads
        self.head_dim = dim // num_heads
        self.causal = bool(causal)
        kw = {"device": device, "dtype": dtype}
        self.qkv = torch.nn.Linear(dim, 3 * dim, bias=qkv_bias, **kw)
        self.q_norm = torch.nn.LayerNorm(self.head_dim, eps=1e-5, **kw) if qk_norm else None
        self.k_norm = torch.nn.LayerNorm(self.head_dim, eps=1e-5, **kw) if qk_norm else None
        self.proj = torch.nn.Linear(dim, dim, **kw)
        self.rope_sections = tuple(int(s) for s in rope_sections) if rope_sections else None
        if self.rope_sections and (min(self.rope_sections) < 1 or 2 * sum(self.rope_sections) > self.head_dim):
            raise ValueError("rope_sections must be positive pair counts with 2 * sum(rope_sections) <= dim / num_heads")
        if self.rope_sections and not rope_interleaved and sum(self.rope_sections) % 8:
            raise ValueError("rope_sections must sum to a multiple of 8 pairs unless rope_interleaved")
        if self.rope_sections and self.head_dim not in (16, 32, 64, 128):
            raise ValueError("rope_sections need a head dimension (dim / num_heads) of 16, 32, 64 or 128")
        if self.rope_sections and len(self.rope_sections) > 4:
            raise ValueError("rope_sections are at most four, one per position axis")
        self.rope_theta = float(rope_theta)
        self.rope_interleaved = bool(rope_interleaved)
        # float64 whatever the module's dtype becomes, so not a buffer; made on a device's first call
        self._frequencies = {}

    def _how(self, positions, dtype=None):
        """ra_qk_norm_rope's keyword arguments for this module and a projection of this dtype."""
        how = {"norm": "none"}
        if self.q_norm is not None:
            how = {"q_weight": self.q_norm.weight, "q_bias": self.q_norm.bias, "k_weight": self.k_norm.weight,
                   "k_bias": self.k_norm.bias}
            # under autocast the projection has another type than the parameters; the kernels take one
            how = {n: t if dtype is None else t.to(dtype) for n, t in how.items()}
            how.update(norm="layer", eps=self.q_norm.eps)
        if self.rope_sections:
            device = self.proj.weight.device
            if device not in self._frequencies:
                with torch.inference_mode(False):   # a later training step saves them for its backward
                    self._frequencies[device] = ra_rope_frequencies(self.rope_sections, self.rope_theta, device=device)
            how.update(frequencies=self._frequencies[device], sections=self.rope_sections, positions=positions,
                       interleaved=self.rope_interleaved)
        return how

    def _merge(self, o):
        B, _, N, _ = o.shape
        return self.proj(o.transpose(1, 2).reshape(B, N, self.num_heads * self.head_dim))

    def forward(self, x, positions=None):
        """positions (with rope_sections): integers that int32 holds, [N], [B, N] or [axes, B, N]; 0 .. N - 1 when not
        given."""
        B, N, C = x.shape
        if self.rope_sections:
            if positions is None:
                positions = torch.arange(N, device=x.device, dtype=torch.int32)
            qkv = self.qkv(x)
            q, k, v = ra_qk_norm_rope(qkv, self.num_heads, **self._how(positions, qkv.dtype))
            return self._merge(ra_attention(q, k, v, is_causal=self.causal))
        if positions is not None:
            raise ValueError("positions need rope_sections")
        q, k, v = self.qkv(x).reshape(B, N, 3, self.num_heads, self.head_dim).permute(2, 0, 3, 1, 4).unbind(0)
        if self.q_norm is not None:
            q, k = self.q_norm(q).to(v.dtype), self.k_norm(k).to(v.dtype)   # autocast's norms return fp32
        o = ra_attention(q, k, v, is_causal=self.causal)
        return self.proj(o.transpose(1, 2).reshape(B, N, C))

    def new_cache(self, batch, capacity, *, prefix=None, track_weight=False, dtype=None):
        """An empty RaCache for this module, of its dtype or (under autocast, the projection's) the one given."""
        return RaCache(batch, self.num_heads, capacity, self.head_dim, prefix=prefix, track_weight=track_weight,
                       device=self.proj.weight.device, dtype=dtype or self.proj.weight.dtype)

    @torch.no_grad()
    def prefill(self, x, cache, positions=None, count=None):
        """forward of a prompt x [B, N, dim] whose keys and values go into an empty cache; returns y.
        count: optional int32 [B], the tokens of a padded batch (rows of y behind them mean nothing).
        Behind a prefix the prompt attends to it too (bf16 only: a masked attention call)."""
        if not self.causal:
            raise ValueError("serving needs a causal module")
        if cache.bound:
            raise ValueError("prefill needs an empty cache")
        B, N, _ = x.shape
        if cache.k.shape[:2] != (B, self.num_heads) or cache.k.shape[3] != self.head_dim:
            raise ValueError("the cache must have the batch size, heads and head dimension of x in this module")
        cache.require_room(N)
        qkv = self.qkv(x)
        if cache.k.dtype != qkv.dtype:
            raise ValueError(f"the cache must have the projection's dtype, {qkv.dtype}")
        P = cache.prefix_length
        if P and qkv.dtype != torch.bfloat16:
            raise NotImplementedError("prefill behind a prefix takes bf16 modules only")
        if self.rope_sections and positions is None:
            positions = torch.arange(P, P + N, device=x.device, dtype=torch.int32)
        q, k, v = ra_qk_norm_rope(qkv, self.num_heads, **self._how(positions, qkv.dtype))
        cache.k[:, :, :N].copy_(k)
        cache.v[:, :, :N].copy_(v)
        cache.advance(N, count)
        if not P:
            return self._merge(ra_attention(q, k, v, is_causal=True))
        k = torch.cat([cache.prefix_k.expand(B, -1, -1, -1), k], 2)
        v = torch.cat([cache.prefix_v.expand(B, -1, -1, -1), v], 2)
        seen = torch.ones(N, P + N, dtype=torch.bool, device=x.device).tril(P)
        return self._merge(ra_attention(q, k, v, attn_mask=seen))

    @torch.no_grad()
    def decode(self, x, cache, positions=None):
        """One token per sequence, x [B, 1, dim], appended to the cache and attended over all of it;
        returns y [B, 1, dim].  positions: as in forward; the cache's own when not given."""
        if not self.causal:
            raise ValueError("serving needs a causal module")
        if x.dim() != 3 or x.shape[1] != 1:
            raise ValueError("decode takes one token per sequence: x [B, 1, dim]")
        if self.rope_sections and positions is None:
            positions = cache.position.view(1, -1, 1)
        qkv = self.qkv(x)
        q = cache.append(qkv, self.num_heads, **self._how(positions, qkv.dtype))
        return self._merge(cache.attend(q[:, :, 0]).unsqueeze(2))


def device_status(stream=None):
    """Synchronise and return the device-side status name ('RA_OK', 'RA_ERR_TIMEOUT', ...), clearing it."""
    s = stream if stream is not None else torch.cuda.current_stream()
    return _STATUS.get(lib().ra_device_status(ctypes.c_void_p(s.cuda_stream)), "unknown")


def set_wait_limit_ns(ns):
    """Limit on every device-side wait of later launches (0 restores the 2 s default)."""
    lib().ra_set_wait_limit_ns(int(ns))


def debug_force_timeout(on):
    """Test knob: make later tensor-core launches take their timeout and wind-down path."""
    lib().ra_debug_force_timeout(1 if on else 0)


def debug_fwd_pair(mode):
    """Layout of later bf16 D = 128 forward calls: 0 automatic (CTA pairs when N_Q > 256),
    1 single CTAs, 2 CTA pairs."""
    lib().ra_debug_fwd_pair(int(mode))


def debug_kernel_events(events):
    """Measurement knob: later bf16 attention calls record these torch.cuda.Event objects
    (up to four, created with enable_timing=True) at their kernel boundaries; None turns it
    off.  Forward: [before the V conversion, before the attention kernel, after it];
    backward: [before the conversion, before dQ, before dK/dV, after dK/dV]."""
    if not events:
        lib().ra_debug_kernel_events(None, 0)
        return
    stream = torch.cuda.current_stream()
    handles = []
    for e in events:
        if e.cuda_event == 0:      # torch creates the CUDA event on its first record
            e.record(stream)
        handles.append(e.cuda_event)
    arr = (ctypes.c_void_p * len(handles))(*handles)
    lib().ra_debug_kernel_events(arr, len(handles))
