"""Positions, key/value caches and single-token attention: the binding of their libraattn calls.

Argument marshalling only, as in the package's other calls: every computation runs in the CUDA
kernels behind include/raattn.h, on torch's current stream of the tensors' device.

    ra_qk_norm_rope(qkv, ...)          q, k and v of every head: norm and rotation, autograd-aware
    ra_cache_append(qkv, k, v, ...)    the same step for new tokens, written into a cache
    ra_attention_decode(q, k, v, ...)  one query token per sequence, own cache and shared prefix
    ra_cache_evict(k, v, weight, ...)  the most attended and the last entries, compacted
    RaCache                            one layer's cache, with its lengths, positions and weights
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import _check, _dtype_code, lib

_NORMS = {"none": 0, "layer": 1, "rms": 2}


# These calls are short on the GPU (single tokens), so their marshalling is kept lean: addresses are
# passed as plain integers, and what follows from sizes and options alone is worked out once.
def _addr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=None)
def _entry(name):
    lib()                       # raises if the library has not been built
    try:
        from . import _calls    # its marshalling in C
    except ImportError:
        return getattr(lib(), name)
    return getattr(_calls, name)


def _call(name, device, *args):
    """Calls a libraattn entry point on torch's current stream of `device`, which becomes the current one."""
    fn, index = _entry(name), device.index
    # the stream's address without a torch.cuda.Stream around it, whose making takes 2 us
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            code = fn(*args, stream)
    if code:
        _check(name, code)


def _check_tensor(name, t, shape, dtype, device):
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _check_cuda(name, t):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor (there is no CPU path)")


def ra_rope_frequencies(sections, theta=10000.0, per_axis=False, device="cuda"):
    """Radians per position of each rotated pair, as a float64 tensor [sum(sections)].

    One ladder theta^(-i / R) over all R pairs, whose consecutive parts the axes take; or, with
    per_axis, a ladder theta^(-i / n) of its own for each axis of n pairs."""
    sections = tuple(int(s) for s in sections)
    if not sections or min(sections) < 1:
        raise ValueError("sections must be positive pair counts, one per axis")
    parts = sections if per_axis else (sum(sections),)
    return torch.cat([float(theta) ** (-torch.arange(n, dtype=torch.float64) / n) for n in parts]).to(device)


@functools.lru_cache(maxsize=256)
def _norm_rope_sizes(width, num_heads, num_kv_heads, sections):
    """(Hq, Hkv, D, pairs, axes, host array of the sections, its address) of a projection `width` wide."""
    Hq, Hkv = int(num_heads), int(num_heads if num_kv_heads is None else num_kv_heads)
    if Hq < 1 or Hkv < 1 or width < 1 or width % (Hq + 2 * Hkv):
        raise ValueError("qkv must be [B, N, (num_heads + 2 num_kv_heads) * head_dim]")
    D = width // (Hq + 2 * Hkv)
    if not sections:
        return Hq, Hkv, D, 0, 0, None, None
    secs = [int(s) for s in sections]
    if min(secs) < 1 or 2 * sum(secs) > D:
        raise ValueError("sections must be positive pair counts with 2 * sum(sections) <= head_dim")
    host = (ctypes.c_int32 * len(secs))(*secs)
    return Hq, Hkv, D, sum(secs), len(secs), host, ctypes.addressof(host)


def _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies, sections, positions, interleaved):
    """Checks the arguments that the forward, the append and the backward share; returns the C call's
    leading arguments, the tensors that have to stay alive until it returns, and (B, N, Hq, Hkv, D, dtype code)."""
    if qkv.dim() != 3 or not qkv.is_cuda:
        raise ValueError("qkv must be a CUDA tensor [B, N, (num_heads + 2 num_kv_heads) * head_dim]")
    dtype, device = qkv.dtype, qkv.device
    code = _dtype_code(dtype)
    B, N, width = qkv.shape
    Hq, Hkv, D, pairs, axes, host, secs = _norm_rope_sizes(width, num_heads, num_kv_heads,
                                                     None if sections is None else tuple(sections))
    if B < 1 or N < 1:
        raise ValueError("qkv must hold at least one token")
    mask = 7 if code else 3
    row, tok, one = qkv.stride()
    if one != 1 or row & mask or tok & mask or qkv.data_ptr() & 15:
        qkv = qkv.contiguous()
        row, tok, one = qkv.stride()
    kind = _NORMS.get(norm)
    if kind is None:
        raise ValueError("norm must be 'none', 'layer' or 'rms'")
    qw, qb, kw, kb = params
    if kind == 0:
        if not (qw is None and qb is None and kw is None and kb is None):
            raise ValueError("norm='none' takes no weights and no biases")
    else:
        if qw is None or kw is None:
            raise ValueError("q_weight and k_weight are required with a norm")
        _check_tensor("q_weight", qw, (D,), dtype, device)
        _check_tensor("k_weight", kw, (D,), dtype, device)
        if qb is not None or kb is not None:
            if kind == 2:
                raise ValueError("norm='rms' takes no biases")
            if qb is not None:
                _check_tensor("q_bias", qb, (D,), dtype, device)
            if kb is not None:
                _check_tensor("k_bias", kb, (D,), dtype, device)
    pos, pos_axis, pos_batch = None, 0, 0
    if axes:
        if frequencies is None or positions is None:
            raise ValueError("sections need frequencies and positions")
        _check_tensor("frequencies", frequencies, (pairs,), torch.float64, device)
        pos = positions
        if pos.dtype is not torch.int32:
            if pos.dtype is not torch.int64:
                raise ValueError("positions must be an int32 or int64 tensor")
            pos = pos.to(torch.int32)
        d = pos.dim()
        shape = pos.shape
        if (pos.device != device or not 1 <= d <= 3 or shape[-1] != N or (d > 1 and shape[-2] not in (1, B))
                or (d > 2 and shape[0] not in (1, axes))):
            raise ValueError("positions must be [N], [B, N] or [axes, B, N] on qkv's device, or broadcast to it")
        if pos.stride(-1) != 1 and N > 1:
            pos = pos.contiguous()
        if d > 1 and shape[-2] > 1:
            pos_batch = pos.stride(-2)
        if d > 2 and shape[0] > 1:
            pos_axis = pos.stride(0)
    elif frequencies is not None or positions is not None:
        raise ValueError("frequencies and positions need sections")
    lead = (qkv.data_ptr(), row, tok, _addr(qw), _addr(qb), _addr(kw), _addr(kb), kind, eps,
            frequencies.data_ptr() if axes else None, pos.data_ptr() if axes else None, pos_axis, pos_batch, secs,
            axes, 1 if interleaved else 0)
    return lead, (qkv, pos, host), (B, N, Hq, Hkv, D, code)


def _norm_rope_forward(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies, sections, positions, interleaved):
    lead, keep, (B, N, Hq, Hkv, D, code) = _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps,
                                                           frequencies, sections, positions, interleaved)
    q = qkv.new_empty((B, Hq, N, D))
    k = qkv.new_empty((B, Hkv, N, D))
    v = qkv.new_empty((B, Hkv, N, D))
    _call("ra_qk_norm_rope_fwd", qkv.device, *lead, q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, 0, B, N, Hq,
          Hkv, D, code)
    return q, k, v


def _dense(t):
    """A gradient as the kernels read it, whatever view of another tensor autograd hands over."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


class _RaQkNormRopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, q_weight, q_bias, k_weight, k_bias, frequencies, positions, how):
        ctx.save_for_backward(qkv, q_weight, q_bias, k_weight, k_bias, frequencies, positions)
        ctx.how = how
        heads, kv_heads, norm, eps, sections, interleaved = how
        return _norm_rope_forward(qkv, heads, kv_heads, norm, (q_weight, q_bias, k_weight, k_bias), eps, frequencies,
                                  sections, positions, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk, dv):
        qkv, qw, qb, kw, kb, frequencies, positions = ctx.saved_tensors
        heads, kv_heads, norm, eps, sections, interleaved = ctx.how
        dqkv, *dparams = ra_qk_norm_rope_backward(
            qkv, _dense(dq), _dense(dk), _dense(dv), heads, kv_heads, norm=norm, q_weight=qw, q_bias=qb, k_weight=kw,
            k_bias=kb, eps=eps, frequencies=frequencies, sections=sections, positions=positions,
            interleaved=interleaved)
        dparams = [None if d is None else d.to(p.dtype) for d, p in zip(dparams, (qw, qb, kw, kb))]
        return (dqkv, *dparams, None, None, None)


def _asks(t):
    return t is not None and t.requires_grad


def ra_qk_norm_rope(qkv, num_heads, num_kv_heads=None, *, norm="layer", q_weight=None, q_bias=None, k_weight=None,
                    k_bias=None, eps=1e-5, frequencies=None, sections=None, positions=None, interleaved=False):
    """q [B, num_heads, N, D], k and v [B, num_kv_heads, N, D], ready for ra_attention, from the packed
    projection qkv [B, N, (num_heads + 2 num_kv_heads) * D] (query heads, key heads, value heads).

    norm: 'layer' (weights, optional biases), 'rms' (weights) or 'none', over each head's D elements
    of q and k.  sections: pairs of dimensions per position axis (None: no rotation); frequencies:
    float64 [sum(sections)], see ra_rope_frequencies; positions: integer [N], [B, N] or
    [axes, B, N].  Pair i is dimensions (i, i + R) of the first 2 R, or (2 i, 2 i + 1) when
    interleaved.  Differentiable (once) in qkv, weights and biases; as with any torch operator, a backward
    pass is captured into a CUDA graph only while no eager graph of the same leaves is alive."""
    if torch.is_grad_enabled() and (qkv.requires_grad or _asks(q_weight) or _asks(k_weight) or _asks(q_bias)
                                    or _asks(k_bias)):
        return _RaQkNormRopeFn.apply(qkv, q_weight, q_bias, k_weight, k_bias, frequencies, positions,
                                     (num_heads, num_kv_heads, norm, eps, sections, interleaved))
    return _norm_rope_forward(qkv, num_heads, num_kv_heads, norm, (q_weight, q_bias, k_weight, k_bias), eps,
                              frequencies, sections, positions, interleaved)


def ra_qk_norm_rope_backward(qkv, dq, dk, dv, num_heads, num_kv_heads=None, *, norm="layer", q_weight=None,
                             q_bias=None, k_weight=None, k_bias=None, eps=1e-5, frequencies=None, sections=None,
                             positions=None, interleaved=False):
    """Gradients of sum(dq q) + sum(dk k) + sum(dv v): (dqkv, dq_weight, dq_bias, dk_weight, dk_bias),
    the parameters' as float32 [D] (None where there is no such parameter)."""
    params = (q_weight, q_bias, k_weight, k_bias)
    lead, keep, (B, N, Hq, Hkv, D, code) = _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps,
                                                           frequencies, sections, positions, interleaved)
    device = qkv.device
    _check_tensor("dq", dq, (B, Hq, N, D), qkv.dtype, device)
    _check_tensor("dk", dk, (B, Hkv, N, D), qkv.dtype, device)
    _check_tensor("dv", dv, (B, Hkv, N, D), qkv.dtype, device)
    dqkv = qkv.new_empty(qkv.shape)
    dparams = ws = None
    if norm != "none":
        dparams = torch.empty((4, D), dtype=torch.float32, device=device)
        ws = torch.empty(_norm_rope_workspace(D), dtype=torch.uint8, device=device)
    _call("ra_qk_norm_rope_bwd", device, *lead, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dqkv.data_ptr(),
          _addr(dparams), _addr(ws), B, N, Hq, Hkv, D, code)
    if dparams is None:
        return dqkv, None, None, None, None
    dqw, dqb, dkw, dkb = dparams.unbind(0)
    return dqkv, dqw, None if q_bias is None else dqb, dkw, None if k_bias is None else dkb


@functools.lru_cache(maxsize=64)
def _norm_rope_workspace(D):
    return lib().ra_qk_norm_rope_bwd_workspace_size(D) or 16


def ra_cache_append(qkv, k, v, length, num_heads, num_kv_heads=None, *, count=None, norm="layer", q_weight=None,
                    q_bias=None, k_weight=None, k_bias=None, eps=1e-5, frequencies=None, sections=None,
                    positions=None, interleaved=False):
    """ra_qk_norm_rope for new tokens, their keys and values written into a cache: token n of
    sequence b to slot length[b] + n of k and v [B, num_kv_heads, C, D].  Returns q.

    count: optional int32 [B], how many of a padded batch's N tokens each sequence has.  Tokens from
    count[b] on, and slots outside the cache, are not written.  length (int32 [B]) is read, not
    advanced.  No autograd."""
    params = (q_weight, q_bias, k_weight, k_bias)
    lead, keep, (B, N, Hq, Hkv, D, code) = _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps,
                                                           frequencies, sections, positions, interleaved)
    dtype, device = qkv.dtype, qkv.device
    if k.dim() != 4 or k.shape[2] < 1:
        raise ValueError("the cache must be [B, num_kv_heads, C, head_dim] with C >= 1")
    shape = (B, Hkv, k.shape[2], D)
    _check_tensor("k", k, shape, dtype, device)
    _check_tensor("v", v, shape, dtype, device)
    _check_tensor("length", length, (B,), torch.int32, device)
    if count is not None:
        _check_tensor("count", count, (B,), torch.int32, device)
    q = qkv.new_empty((B, Hq, N, D))
    _call("ra_qk_norm_rope_fwd", device, *lead, q.data_ptr(), k.data_ptr(), v.data_ptr(), length.data_ptr(),
          _addr(count), shape[2], B, N, Hq, Hkv, D, code)
    return q


def ra_attention_decode(q, k, v, length, *, prefix_k=None, prefix_v=None, scale=None, weight=None):
    """ra_attention of one query token per sequence: o [B, H, D] for q [B, H, D] over the P keys
    of a prefix that the whole batch shares (prefix_k, prefix_v [H_kv, P, D], or None) and the first
    length[b] (int32 [B]) of the sequence's own cache k, v [B, H_kv, C, D].

    H is a multiple of H_kv; consecutive query heads share a key head.  weight: optional float32
    [B, H_kv, C], to which each own key's attention weights, summed over its query heads, are added in
    place.  A sequence without any key gives zeros.  bf16 with head dimension 64 or 128, fp32 with
    16, 32, 64 or 128.  No autograd."""
    if q.dim() != 3 or k.dim() != 4:
        raise ValueError("q must be [B, H, D] and the cache [B, H_kv, C, D]")
    _check_cuda("q", q)
    B, Hq, D = q.shape
    Hkv, C = k.shape[1], k.shape[2]
    dtype, device = q.dtype, q.device
    code = _dtype_code(dtype)
    shape = (B, Hkv, C, D)
    _check_tensor("k", k, shape, dtype, device)
    _check_tensor("v", v, shape, dtype, device)
    _check_tensor("length", length, (B,), torch.int32, device)
    if B < 1 or Hkv < 1 or C < 1 or Hq < 1 or D < 1 or Hq % Hkv:
        raise ValueError("the number of query heads must be a multiple of the key heads', and no size 0")
    P = 0
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError("prefix_k and prefix_v come together")
    if prefix_k is not None:
        P = prefix_k.shape[1] if prefix_k.dim() == 3 else -1
        _check_tensor("prefix_k", prefix_k, (Hkv, P, D), dtype, device)
        _check_tensor("prefix_v", prefix_v, (Hkv, P, D), dtype, device)
        if P == 0:
            prefix_k = prefix_v = None
    if weight is not None:
        _check_tensor("weight", weight, (B, Hkv, C), torch.float32, device)
    o = q.new_empty((B, Hq, D))
    nbytes = _decode_workspace(B, Hq, Hkv, C, P, D, code)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _call("ra_attention_decode", device, q.data_ptr(), k.data_ptr(), v.data_ptr(), length.data_ptr(), _addr(prefix_k),
          _addr(prefix_v), o.data_ptr(), _addr(weight), ws.data_ptr(), B, Hq, Hkv, C, P, D, scale or 0.0, code)
    return o


@functools.lru_cache(maxsize=256)
def _decode_workspace(B, Hq, Hkv, C, P, D, code):
    return max(lib().ra_attention_decode_workspace_size(B, Hq, Hkv, C, P, D, code), 16)


def ra_cache_evict(k, v, weight, length, keep, *, recent=0, out=None):
    """A cache cut down to at most `keep` entries per sequence and key head: the last `recent` ones and
    the ones of the largest accumulated weight among the others (of equal weights the oldest), in
    their order.  Returns (k, v, weight, length, index): the compacted cache, its int32 lengths [B] and
    the kept slots int32 [B, H_kv, keep] (ascending, then -1).

    out: optional (k, v, weight) with room for at least `keep` entries, other tensors than the inputs;
    slots behind the new length are left as they are.  Without it, tensors of exactly `keep`
    entries are made, zero behind the new length."""
    if k.dim() != 4:
        raise ValueError("the cache must be [B, H_kv, C, D]")
    _check_cuda("k", k)
    B, Hkv, C, D = k.shape
    device, code = k.device, _dtype_code(k.dtype)
    keep, recent = int(keep), int(recent)
    if min(B, Hkv, C, D) < 1 or keep < 1 or not 0 <= recent <= keep:
        raise ValueError("keep must be at least 1, recent between 0 and keep, and no size 0")
    _check_tensor("v", v, (B, Hkv, C, D), k.dtype, device)
    _check_tensor("weight", weight, (B, Hkv, C), torch.float32, device)
    _check_tensor("length", length, (B,), torch.int32, device)
    if out is None:
        out = (torch.zeros((B, Hkv, keep, D), dtype=k.dtype, device=device),
               torch.zeros((B, Hkv, keep, D), dtype=k.dtype, device=device),
               torch.zeros((B, Hkv, keep), dtype=torch.float32, device=device))
    ko, vo, wo = out
    Co = ko.shape[2] if ko.dim() == 4 else 0
    if Co < keep:
        raise ValueError("out must have room for `keep` entries")
    _check_tensor("out[0]", ko, (B, Hkv, Co, D), k.dtype, device)
    _check_tensor("out[1]", vo, (B, Hkv, Co, D), k.dtype, device)
    _check_tensor("out[2]", wo, (B, Hkv, Co), torch.float32, device)
    new_length = length.new_empty((B,))
    index = length.new_empty((B, Hkv, keep))
    _call("ra_cache_evict", device, k.data_ptr(), v.data_ptr(), weight.data_ptr(), length.data_ptr(), ko.data_ptr(),
          vo.data_ptr(), wo.data_ptr(), new_length.data_ptr(), index.data_ptr(), B, Hkv, C, Co, D, keep, recent, code)
    return ko, vo, wo, new_length, index


class RaCache:
    """One attention layer's key/value cache: `batch` sequences of up to `capacity` own entries, behind
    an optional prefix that all of them share.

    k, v [B, H_kv, C, D]; length int32 [B] (entries held) and position int32 [B] (position of the
    next token: evicted entries still count, and so does the prefix), both on the device; weight
    float32 [B, H_kv, C] with track_weight, the attention each entry has received from attend (a
    module's prefill adds none).

    A captured graph of append and attend advances length and position when it is replayed, but not
    `bound`, which is the host's: whoever replays it sees to it that there is room (tokens beyond the
    capacity are not stored).  evict changes which tensors the cache uses, so graphs of it are
    captured anew afterwards."""

    def __init__(self, batch, num_kv_heads, capacity, head_dim, *, prefix=None, track_weight=False, device="cuda",
                 dtype=torch.bfloat16):
        shape = (int(batch), int(num_kv_heads), int(capacity), int(head_dim))
        if min(shape) < 1:
            raise ValueError("batch, num_kv_heads, capacity and head_dim must be at least 1")
        _dtype_code(dtype)
        self.k = torch.zeros(shape, device=device, dtype=dtype)
        self.v = torch.zeros(shape, device=device, dtype=dtype)
        self.weight = torch.zeros(shape[:3], device=device, dtype=torch.float32) if track_weight else None
        self.length = torch.zeros(shape[0], device=device, dtype=torch.int32)
        self.prefix_k = self.prefix_v = None
        if prefix is not None:
            pk, pv = (t.contiguous() for t in prefix)
            if pk.dim() != 3 or pk.shape[0] != shape[1] or pk.shape[2] != shape[3] or pk.shape != pv.shape:
                raise ValueError("prefix must be (k, v), each [num_kv_heads, P, head_dim]")
            if pk.dtype != dtype or pv.dtype != dtype or pk.device != self.k.device or pv.device != self.k.device:
                raise ValueError("prefix must have the cache's dtype and device")
            self.prefix_k, self.prefix_v = pk, pv
        self.position = torch.full_like(self.length, self.prefix_length)
        self.bound = 0            # no sequence holds more entries than this

    @property
    def capacity(self):
        return self.k.shape[2]

    @property
    def prefix_length(self):
        return 0 if self.prefix_k is None else self.prefix_k.shape[1]

    def advance(self, tokens, count=None):
        """Counts `tokens` new entries (or count[b] of them, int32 [B])."""
        step = tokens if count is None else count.clamp(0, tokens)
        self.length.add_(step)
        self.position.add_(step)
        self.bound += tokens

    def require_room(self, tokens):
        if self.bound + tokens > self.capacity:
            raise ValueError(f"the cache holds up to {self.bound} of {self.capacity} entries: no room for {tokens} more")

    def append(self, qkv, num_heads, *, count=None, **how):
        """ra_cache_append at this cache's lengths, which advance; returns q."""
        self.require_room(qkv.shape[1])
        q = ra_cache_append(qkv, self.k, self.v, self.length, num_heads, self.k.shape[1], count=count, **how)
        self.advance(qkv.shape[1], count)
        return q

    def attend(self, q, scale=None):
        """ra_attention_decode of q [B, H, D] against everything this cache holds."""
        return ra_attention_decode(q, self.k, self.v, self.length, prefix_k=self.prefix_k, prefix_v=self.prefix_v,
                                   scale=scale, weight=self.weight)

    def evict(self, keep, *, recent=0, spare=None):
        """Cuts every sequence down to `keep` entries (ra_cache_evict); needs track_weight.  The cache moves
        to `spare`, a (k, v) pair of the same shape (made when not given), and the pair it held
        before is returned: one spare pair serves all layers in turn."""
        if self.weight is None:
            raise ValueError("eviction needs a cache with track_weight=True")
        if keep > self.capacity:
            raise ValueError("keep exceeds the cache's capacity")
        if spare is None:
            spare = (torch.zeros_like(self.k), torch.zeros_like(self.v))
        if any(s.shape != self.k.shape for s in spare):
            raise ValueError("spare must be a pair shaped like the cache")
        weight = torch.zeros_like(self.weight)     # entries appended later start from 0
        *_, length, _ = ra_cache_evict(self.k, self.v, self.weight, self.length, keep, recent=recent,
                                       out=(*spare, weight))
        before = (self.k, self.v)
        (self.k, self.v), self.weight = spare, weight
        self.length.copy_(length)
        self.bound = min(self.bound, int(keep))
        return before
