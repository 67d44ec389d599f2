"""Positions, key/value caches and single-token attention: the public functions.

Their checks, outputs and argument marshalling are in csrc/calls.cpp (the module _calls), since these
calls' kernels are short; every computation runs in the CUDA kernels behind include/raattn.h, on torch's
current stream of the tensors' device.

    ra_qk_norm_rope(qkv, ...)          q, k and v of every head: norm and rotation, autograd-aware
    ra_cache_append(qkv, k, v, ...)    the same step for new tokens, written into a cache
    ra_attention_decode(q, k, v, ...)  one query token per sequence, own cache and shared prefix
    ra_cache_evict(k, v, weight, ...)  the most attended and the last entries, compacted
    RaCache                            one layer's cache, with its lengths, positions and weights
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _dtype_code, lib

_calls = None


def _native():
    """The module _calls; raises if it has not been built."""
    global _calls
    if _calls is None:
        lib()
        try:
            from . import _calls as module
        except ImportError as e:
            raise RuntimeError("_calls.so is not built; run `python -m rational_softmax_attention_gb300.build`") from e
        _calls = module
    return _calls


def ra_rope_frequencies(sections, theta=10000.0, per_axis=False, device="cuda"):
    """Radians per position of each rotated pair, as a float64 tensor [sum(sections)].

    One ladder theta^(-i / R) over all R pairs, whose consecutive parts the axes take; or, with
    per_axis, a ladder theta^(-i / n) of its own for each axis of n pairs."""
    sections = tuple(int(s) for s in sections)
    if not sections or min(sections) < 1:
        raise ValueError("sections must be positive pair counts, one per axis")
    parts = sections if per_axis else (sum(sections),)
    return torch.cat([float(theta) ** (-torch.arange(n, dtype=torch.float64) / n) for n in parts]).to(device)


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
        return _native().norm_rope(qkv, heads, kv_heads, norm, q_weight, q_bias, k_weight, k_bias, eps, frequencies,
                                   sections, positions, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk, dv):
        qkv, qw, qb, kw, kb, frequencies, positions = ctx.saved_tensors
        heads, kv_heads, norm, eps, sections, interleaved = ctx.how
        dqkv, *dparams = _native().norm_rope_backward(qkv, heads, kv_heads, norm, qw, qb, kw, kb, eps, frequencies,
                                                      sections, positions, interleaved, _dense(dq), _dense(dk), _dense(dv))
        dparams = [None if d is None else d.to(p.dtype) for d, p in zip(dparams, (qw, qb, kw, kb))]
        return (dqkv, *dparams, None, None, None)


def _asks(t):
    return t is not None and t.requires_grad


def ra_qk_norm_rope(qkv, num_heads, num_kv_heads=None, *, norm="layer", q_weight=None, q_bias=None, k_weight=None,
                    k_bias=None, eps=1e-5, frequencies=None, sections=None, positions=None, interleaved=False):
    """q [B, num_heads, N, D], k and v [B, num_kv_heads, N, D] from the packed projection
    qkv [B, N, (num_heads + 2 num_kv_heads) * D] (query heads, key heads, value heads).  They are what
    ra_attention takes where num_kv_heads is num_heads; it takes no fewer key heads than query heads.

    norm: 'layer' (weights, optional biases), 'rms' (weights) or 'none', over each head's D elements
    of q and k.  sections: pairs of dimensions per position axis (None: no rotation); frequencies:
    float64 [sum(sections)], see ra_rope_frequencies; positions: int32, or int64 of values that
    int32 holds (converted, one more kernel; greater ones wrap), [N], [B, N] or [axes, B, N].  Pair i is dimensions (i, i + R) of the first 2 R, or (2 i, 2 i + 1) when
    interleaved.  Differentiable (once, in reverse mode) in qkv, weights and biases; as with any torch operator, a backward
    pass is captured into a CUDA graph only while no eager graph of the same leaves is alive."""
    if torch.is_grad_enabled() and (qkv.requires_grad or _asks(q_weight) or _asks(k_weight) or _asks(q_bias)
                                    or _asks(k_bias)):
        return _RaQkNormRopeFn.apply(qkv, q_weight, q_bias, k_weight, k_bias, frequencies, positions,
                                     (num_heads, num_kv_heads, norm, eps, sections, interleaved))
    return _native().norm_rope(qkv, num_heads, num_kv_heads, norm, q_weight, q_bias, k_weight, k_bias, eps, frequencies,
                               sections, positions, interleaved)


def ra_qk_norm_rope_backward(qkv, dq, dk, dv, num_heads, num_kv_heads=None, *, norm="layer", q_weight=None,
                             q_bias=None, k_weight=None, k_bias=None, eps=1e-5, frequencies=None, sections=None,
                             positions=None, interleaved=False):
    """Gradients of sum(dq q) + sum(dk k) + sum(dv v): (dqkv, dq_weight, dq_bias, dk_weight, dk_bias),
    the parameters' as float32 [D] (None where there is no such parameter)."""
    return _native().norm_rope_backward(qkv, num_heads, num_kv_heads, norm, q_weight, q_bias, k_weight, k_bias, eps,
                                        frequencies, sections, positions, interleaved, dq, dk, dv)


def ra_cache_append(qkv, k, v, length, num_heads, num_kv_heads=None, *, count=None, norm="layer", q_weight=None,
                    q_bias=None, k_weight=None, k_bias=None, eps=1e-5, frequencies=None, sections=None,
                    positions=None, interleaved=False):
    """ra_qk_norm_rope for new tokens, their keys and values written into a cache: token n of
    sequence b to slot length[b] + n of k and v [B, num_kv_heads, C, D].  Returns q.

    count: optional int32 [B], how many of a padded batch's N tokens each sequence has.  Tokens from
    count[b] on, and slots outside the cache, are not written.  length (int32 [B]) is read, not
    advanced.  No autograd."""
    return _native().cache_append(qkv, num_heads, num_kv_heads, norm, q_weight, q_bias, k_weight, k_bias, eps, frequencies,
                                  sections, positions, interleaved, k, v, length, count)


def ra_attention_decode(q, k, v, length, *, prefix_k=None, prefix_v=None, scale=None, weight=None):
    """ra_attention of one query token per sequence: o [B, H, D] for q [B, H, D] over the P keys
    of a prefix that the whole batch shares (prefix_k, prefix_v [H_kv, P, D], or None) and the first
    length[b] (int32 [B]) of the sequence's own cache k, v [B, H_kv, C, D].

    H is a multiple of H_kv; consecutive query heads share a key head.  weight: optional float32
    [B, H_kv, C], to which each own key's attention weights, summed over its query heads, are added in
    place.  A sequence without any key gives zeros.  bf16 with head dimension 64 or 128, fp32 with
    16, 32, 64 or 128.  No autograd."""
    return _native().attention_decode(q, k, v, length, prefix_k, prefix_v, scale, weight)


def ra_cache_evict(k, v, weight, length, keep, *, recent=0, out=None):
    """A cache cut down to at most `keep` entries per sequence and key head: the last `recent` ones and
    the ones of the largest accumulated weight among the others (of equal weights the oldest), in
    their order.  Returns (k, v, weight, length, index): the compacted cache, its int32 lengths [B] and
    the kept slots int32 [B, H_kv, keep] (ascending, then -1).

    out: optional (k, v, weight) with room for at least `keep` entries, other tensors than the inputs;
    slots behind the new length are left as they are.  Without it, tensors of exactly `keep`
    entries are made, zero behind the new length."""
    return _native().cache_evict(k, v, weight, length, keep, recent, None if out is None else tuple(out))


class RaCache:
    """One attention layer's key/value cache: `batch` sequences of up to `capacity` own entries, behind
    an optional prefix that all of them share.

    k, v [B, H_kv, C, D]; length int32 [B] (entries held) and position int32 [B] (position of the
    next token: evicted entries still count, and so does the prefix), both on the device; weight
    float32 [B, H_kv, C] with track_weight, the attention each entry has received from attend (a
    module's prefill adds none).

    `bound` is the host's count of the entries of the longest sequence, or more (padding included until
    require_room reads the lengths back).  A captured graph of append and attend advances length and position when it is replayed, but not
    `bound`: whoever replays it sees to it that there is room (tokens beyond the
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
        self.bound = min(self.bound + tokens, self.capacity)   # require_room has seen to it that there is room

    def require_room(self, tokens, count=None):
        """Raises unless every sequence has room for `tokens` more entries, or count[b] of them.  `bound` counts a
        padded batch's padding too: where it leaves no room, the lengths are read back, which waits for the
        device (not while a graph is captured)."""
        if self.bound + tokens <= self.capacity:
            return
        room = False
        if not (self.length.is_cuda and torch.cuda.is_current_stream_capturing()):
            held = self.length.clamp(0, self.capacity)
            after = held + (tokens if count is None else count.clamp(0, tokens))
            self.bound, most = (int(n.max()) for n in (held, after))
            room = most <= self.capacity
        if not room:
            raise ValueError(f"the cache holds up to {self.bound} of {self.capacity} entries: no room for {tokens} more")

    def append(self, qkv, num_heads, *, count=None, **how):
        """ra_cache_append at this cache's lengths, which advance; returns q."""
        self.require_room(qkv.shape[1], count)
        q = ra_cache_append(qkv, self.k, self.v, self.length, num_heads, self.k.shape[1], count=count, **how)
        self.advance(qkv.shape[1], count)
        return q

    def attend(self, q, scale=None):
        """ra_attention_decode of q [B, H, D] against everything this cache holds."""
        return ra_attention_decode(q, self.k, self.v, self.length, prefix_k=self.prefix_k, prefix_v=self.prefix_v,
                                   scale=scale, weight=self.weight)

    def evict(self, keep, *, recent=0, spare=None):
        """Cuts every sequence down to `keep` entries (ra_cache_evict); needs track_weight.  Weights come from
        attend: straight after a prefill all are 0, and the oldest entries are kept beside the last `recent`.  The cache moves
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
