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

import contextlib

import torch

from . import _check, _dtype_code, _ptr, _require_cuda, _stream, lib

_NORMS = {"none": 0, "layer": 1, "rms": 2}
_SAME = contextlib.nullcontext()


def _on(device):
    """Makes `device` current for a call whose tensors live there."""
    return _SAME if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _check_tensor(name, t, shape, dtype, device):
    if t.device != device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def ra_rope_frequencies(sections, theta=10000.0, per_axis=False, device="cuda"):
    """Radians per position of each rotated pair, as a float64 tensor [sum(sections)].

    One ladder theta^(-i / R) over all R pairs, whose consecutive parts the axes take; or, with
    per_axis, a ladder theta^(-i / n) of its own for each axis of n pairs."""
    sections = tuple(int(s) for s in sections)
    if not sections or min(sections) < 1:
        raise ValueError("sections must be positive pair counts, one per axis")
    parts = sections if per_axis else (sum(sections),)
    return torch.cat([float(theta) ** (-torch.arange(n, dtype=torch.float64) / n) for n in parts]).to(device)


def _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies, sections, positions, interleaved):
    """Checks the arguments that the forward, the append and the backward share; returns the C
    call's leading arguments, what has to stay alive until it returns, and (B, N, Hq, Hkv, D)."""
    if qkv.dim() != 3 or not qkv.is_cuda:
        raise ValueError("qkv must be a CUDA tensor [B, N, (num_heads + 2 num_kv_heads) * head_dim]")
    dtype, device = qkv.dtype, qkv.device
    _dtype_code(dtype)
    Hq, Hkv = int(num_heads), int(num_heads if num_kv_heads is None else num_kv_heads)
    B, N, W = qkv.shape
    if Hq < 1 or Hkv < 1 or W % (Hq + 2 * Hkv) or B < 1 or N < 1 or W < 1:
        raise ValueError("qkv must be [B, N, (num_heads + 2 num_kv_heads) * head_dim], with at least one token")
    D = W // (Hq + 2 * Hkv)
    vec = 16 // qkv.element_size()
    if qkv.stride(2) != 1 or qkv.stride(0) % vec or qkv.stride(1) % vec or qkv.data_ptr() % 16:
        qkv = qkv.contiguous()
    if norm not in _NORMS:
        raise ValueError("norm must be 'none', 'layer' or 'rms'")
    qw, qb, kw, kb = params
    if norm == "none" and any(p is not None for p in params):
        raise ValueError("norm='none' takes no weights and no biases")
    if norm != "none" and (qw is None or kw is None):
        raise ValueError("q_weight and k_weight are required with a norm")
    if norm == "rms" and (qb is not None or kb is not None):
        raise ValueError("norm='rms' takes no biases")
    for name, p in zip(("q_weight", "q_bias", "k_weight", "k_bias"), params):
        if p is not None:
            _check_tensor(name, p, (D,), dtype, device)
    keep = [qkv, frequencies]
    axes, pos, pos_axis, pos_batch, secs = 0, None, 0, 0, None
    if sections is not None and len(sections):
        secs = tuple(int(s) for s in sections)
        axes, pairs = len(secs), sum(secs)
        if min(secs) < 1 or 2 * pairs > D:
            raise ValueError("sections must be positive pair counts with 2 * sum(sections) <= head_dim")
        if frequencies is None or positions is None:
            raise ValueError("sections need frequencies and positions")
        _check_tensor("frequencies", frequencies, (pairs,), torch.float64, device)
        pos = positions
        if pos.dtype not in (torch.int32, torch.int64) or pos.device != device or not 1 <= pos.dim() <= 3:
            raise ValueError("positions must be an int32 or int64 tensor [N], [B, N] or [axes, B, N] on qkv's device")
        pos = pos.to(torch.int32)
        pos = pos.view((1,) * (3 - pos.dim()) + tuple(pos.shape))
        if pos.shape[0] not in (1, axes) or pos.shape[1] not in (1, B) or pos.shape[2] != N:
            raise ValueError("positions must broadcast to [axes, B, N]")
        if pos.stride(2) != 1 and N > 1:
            pos = pos.contiguous()
        pos_axis = pos.stride(0) if pos.shape[0] > 1 else 0
        pos_batch = pos.stride(1) if pos.shape[1] > 1 else 0
        keep.append(pos)
        secs = _int_array(secs)
        keep.append(secs)
    elif frequencies is not None or positions is not None:
        raise ValueError("frequencies and positions need sections")
    lead = (_ptr(qkv), qkv.stride(0), qkv.stride(1), _ptr(qw), _ptr(qb), _ptr(kw), _ptr(kb), _NORMS[norm], float(eps),
            _ptr(frequencies) if axes else None, _ptr(pos), pos_axis, pos_batch, secs, axes, 1 if interleaved else 0)
    return lead, keep, (B, N, Hq, Hkv, D)


def _int_array(values):
    import ctypes
    return (ctypes.c_int32 * len(values))(*values)


def _norm_rope_forward(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies, sections, positions, interleaved):
    lead, keep, (B, N, Hq, Hkv, D) = _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies,
                                                     sections, positions, interleaved)
    q = torch.empty((B, Hq, N, D), dtype=qkv.dtype, device=qkv.device)
    k = torch.empty((B, Hkv, N, D), dtype=qkv.dtype, device=qkv.device)
    v = torch.empty((B, Hkv, N, D), dtype=qkv.dtype, device=qkv.device)
    with _on(qkv.device):
        _check("ra_qk_norm_rope_fwd", lib().ra_qk_norm_rope_fwd(
            *lead, _ptr(q), _ptr(k), _ptr(v), None, None, 0, B, N, Hq, Hkv, D, _dtype_code(qkv.dtype),
            _stream(qkv.device)))
    return q, k, v


class _RaQkNormRopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, q_weight, q_bias, k_weight, k_bias, frequencies, positions, how):
        ctx.save_for_backward(qkv, q_weight, q_bias, k_weight, k_bias, frequencies, positions)
        ctx.how = how
        heads, kv_heads, norm, eps, sections, interleaved = how
        return _norm_rope_forward(qkv, heads, kv_heads, norm, (q_weight, q_bias, k_weight, k_bias), eps, frequencies,
                                  sections, positions, interleaved)

    @staticmethod
    def backward(ctx, dq, dk, dv):
        qkv, qw, qb, kw, kb, frequencies, positions = ctx.saved_tensors
        heads, kv_heads, norm, eps, sections, interleaved = ctx.how
        dqkv, *dparams = ra_qk_norm_rope_backward(
            qkv, dq.contiguous(), dk.contiguous(), dv.contiguous(), heads, kv_heads, norm=norm, q_weight=qw,
            q_bias=qb, k_weight=kw, k_bias=kb, eps=eps, frequencies=frequencies, sections=sections,
            positions=positions, interleaved=interleaved)
        dparams = [None if d is None else d.to(p.dtype) for d, p in zip(dparams, (qw, qb, kw, kb))]
        return (dqkv, *dparams, None, None, None)


def ra_qk_norm_rope(qkv, num_heads, num_kv_heads=None, *, norm="layer", q_weight=None, q_bias=None, k_weight=None,
                    k_bias=None, eps=1e-5, frequencies=None, sections=None, positions=None, interleaved=False):
    """q [B, num_heads, N, D], k and v [B, num_kv_heads, N, D], ready for ra_attention, from the packed
    projection qkv [B, N, (num_heads + 2 num_kv_heads) * D] (query heads, key heads, value heads).

    norm: 'layer' (weights, optional biases), 'rms' (weights) or 'none', over each head's D elements
    of q and k.  sections: pairs of dimensions per position axis (None: no rotation); frequencies:
    float64 [sum(sections)], see ra_rope_frequencies; positions: integer [N], [B, N] or
    [axes, B, N].  Pair i is dimensions (i, i + R) of the first 2 R, or (2 i, 2 i + 1) when
    interleaved.  Differentiable in qkv, weights and biases."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (qkv, q_weight, q_bias, k_weight, k_bias)):
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
    lead, keep, (B, N, Hq, Hkv, D) = _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies,
                                                     sections, positions, interleaved)
    for name, t, h in (("dq", dq, Hq), ("dk", dk, Hkv), ("dv", dv, Hkv)):
        _check_tensor(name, t, (B, h, N, D), qkv.dtype, qkv.device)
    L = lib()
    dqkv = torch.empty(qkv.shape, dtype=qkv.dtype, device=qkv.device)
    dparams = ws = None
    if norm != "none":
        dparams = torch.empty((4, D), dtype=torch.float32, device=qkv.device)
        ws = torch.empty(max(L.ra_qk_norm_rope_bwd_workspace_size(D), 16), dtype=torch.uint8, device=qkv.device)
    with _on(qkv.device):
        _check("ra_qk_norm_rope_bwd", L.ra_qk_norm_rope_bwd(
            *lead, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dqkv), _ptr(dparams), _ptr(ws), B, N, Hq, Hkv, D,
            _dtype_code(qkv.dtype), _stream(qkv.device)))
    return (dqkv, *(None if p is None else dparams[i] for i, p in enumerate(params)))


def ra_cache_append(qkv, k, v, length, num_heads, num_kv_heads=None, *, count=None, norm="layer", q_weight=None,
                    q_bias=None, k_weight=None, k_bias=None, eps=1e-5, frequencies=None, sections=None,
                    positions=None, interleaved=False):
    """ra_qk_norm_rope for new tokens, their keys and values written into a cache: token n of
    sequence b to slot length[b] + n of k and v [B, num_kv_heads, C, D].  Returns q.

    count: optional int32 [B], how many of a padded batch's N tokens each sequence has.  Tokens from
    count[b] on, and slots outside the cache, are not written.  length (int32 [B]) is read, not
    advanced.  No autograd."""
    params = (q_weight, q_bias, k_weight, k_bias)
    lead, keep, (B, N, Hq, Hkv, D) = _norm_rope_args(qkv, num_heads, num_kv_heads, norm, params, eps, frequencies,
                                                     sections, positions, interleaved)
    device = qkv.device
    if k.dim() != 4 or k.shape[2] < 1:
        raise ValueError("the cache must be [B, num_kv_heads, C, head_dim] with C >= 1")
    C = k.shape[2]
    _check_tensor("k", k, (B, Hkv, C, D), qkv.dtype, device)
    _check_tensor("v", v, (B, Hkv, C, D), qkv.dtype, device)
    _check_tensor("length", length, (B,), torch.int32, device)
    if count is not None:
        _check_tensor("count", count, (B,), torch.int32, device)
    q = torch.empty((B, Hq, N, D), dtype=qkv.dtype, device=device)
    with _on(device):
        _check("ra_qk_norm_rope_fwd", lib().ra_qk_norm_rope_fwd(
            *lead, _ptr(q), _ptr(k), _ptr(v), _ptr(length), _ptr(count), C, B, N, Hq, Hkv, D,
            _dtype_code(qkv.dtype), _stream(device)))
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
    _require_cuda(q)
    B, Hq, D = q.shape
    Hkv, C = k.shape[1], k.shape[2]
    device, code = q.device, _dtype_code(q.dtype)
    _check_tensor("k", k, (B, Hkv, C, D), q.dtype, device)
    _check_tensor("v", v, (B, Hkv, C, D), q.dtype, device)
    _check_tensor("length", length, (B,), torch.int32, device)
    if B < 1 or Hkv < 1 or C < 1 or Hq < 1 or D < 1 or Hq % Hkv:
        raise ValueError("the number of query heads must be a multiple of the key heads', and no size 0")
    P = 0
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError("prefix_k and prefix_v come together")
    if prefix_k is not None:
        P = prefix_k.shape[1] if prefix_k.dim() == 3 else -1
        _check_tensor("prefix_k", prefix_k, (Hkv, P, D), q.dtype, device)
        _check_tensor("prefix_v", prefix_v, (Hkv, P, D), q.dtype, device)
        if P == 0:
            prefix_k = prefix_v = None
    if weight is not None:
        _check_tensor("weight", weight, (B, Hkv, C), torch.float32, device)
    L = lib()
    o = torch.empty_like(q)
    ws = torch.empty(max(L.ra_attention_decode_workspace_size(B, Hq, Hkv, C, P, D, code), 16), dtype=torch.uint8,
                     device=device)
    with _on(device):
        _check("ra_attention_decode", L.ra_attention_decode(
            _ptr(q), _ptr(k), _ptr(v), _ptr(length), _ptr(prefix_k), _ptr(prefix_v), _ptr(o), _ptr(weight), _ptr(ws),
            B, Hq, Hkv, C, P, D, float(scale or 0.0), code, _stream(device)))
    return o


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
    _require_cuda(k)
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
    new_length = torch.empty_like(length)
    index = torch.empty((B, Hkv, keep), dtype=torch.int32, device=device)
    with _on(device):
        _check("ra_cache_evict", lib().ra_cache_evict(
            _ptr(k), _ptr(v), _ptr(weight), _ptr(length), _ptr(ko), _ptr(vo), _ptr(wo), _ptr(new_length), _ptr(index),
            B, Hkv, C, Co, D, keep, recent, code, _stream(device)))
    return ko, vo, wo, new_length, index


class RaCache:
    """One attention layer's key/value cache: `batch` sequences of up to `capacity` own entries, behind
    an optional prefix that all of them share.

    k, v [B, H_kv, C, D]; length int32 [B] (entries held) and position int32 [B] (position of the
    next token: evicted entries still count, and so does the prefix), both on the device; weight
    float32 [B, H_kv, C] with track_weight, the attention each entry has received."""

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
        step = tokens if count is None else count
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
