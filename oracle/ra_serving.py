"""Float64 CPU oracle of the position and serving operators.

TEST INFRASTRUCTURE, NOT PRODUCT CODE; imports nothing from the product package.  Pins:
tests/test_oracle_serving.py (finite differences, the attention oracle on concatenated keys,
rotations as relative positions, hand-made evictions).
"""
from __future__ import annotations

import numpy as np

from .ra_oracle import ra_softmax


def _angles(frequencies, sections, positions, B, N):
    """[B, N, R] angles of every pair; positions broadcastable to [axes, B, N]."""
    pos = np.broadcast_to(np.asarray(positions, dtype=np.float64), (len(sections), B, N))
    axis = np.repeat(np.arange(len(sections)), sections)
    return pos[axis].transpose(1, 2, 0) * np.asarray(frequencies, dtype=np.float64)


def _pairs(D, R, interleaved):
    i = np.arange(R)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R)


def _turn(x, angle, interleaved):
    """x [B, N, H, D] with its first 2 R dimensions turned by angle [B, N, R]."""
    R = angle.shape[-1]
    a, b = _pairs(x.shape[-1], R, interleaved)
    c, s = np.cos(angle)[:, :, None], np.sin(angle)[:, :, None]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _norm(x, norm, eps):
    if norm == "none":
        return x, np.ones(x.shape[:-1] + (1,))
    if norm == "layer":
        x = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def _split(qkv, Hq, Hkv):
    B, N, W = qkv.shape
    x = np.asarray(qkv, dtype=np.float64).reshape(B, N, Hq + 2 * Hkv, -1)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


def qk_norm_rope(qkv, Hq, Hkv, norm="none", params=(None,) * 4, eps=1e-5, frequencies=None, sections=None,
                 positions=None, interleaved=False):
    """q [B, Hq, N, D], k, v [B, Hkv, N, D]; params = (q weight, q bias, k weight, k bias)."""
    q, k, v = _split(qkv, Hq, Hkv)
    out = []
    for x, w, b in ((q, params[0], params[1]), (k, params[2], params[3])):
        y, _ = _norm(x, norm, eps)
        y = y if w is None else y * w
        y = y if b is None else y + b
        if sections:
            y = _turn(y, _angles(frequencies, sections, positions, *qkv.shape[:2]), interleaved)
        out.append(y.transpose(0, 2, 1, 3))
    return out[0], out[1], v.transpose(0, 2, 1, 3)


def qk_norm_rope_bwd(qkv, dq, dk, dv, Hq, Hkv, norm="none", params=(None,) * 4, eps=1e-5, frequencies=None,
                     sections=None, positions=None, interleaved=False):
    """(dqkv, [dq weight, dq bias, dk weight, dk bias]); the parameters' gradients always given with a norm."""
    q, k, _ = _split(qkv, Hq, Hkv)
    dx, dparams = [], []
    for x, dy, w in ((q, dq, params[0]), (k, dk, params[2])):
        g = np.asarray(dy, dtype=np.float64).transpose(0, 2, 1, 3)
        if sections:
            g = _turn(g, -_angles(frequencies, sections, positions, *qkv.shape[:2]), interleaved)
        if norm == "none":
            dx.append(g)
            dparams += [None, None]
            continue
        xhat, r = _norm(x, norm, eps)
        dparams += [(g * xhat).sum((0, 1, 2)), g.sum((0, 1, 2))]
        t = g * w
        d = t - xhat * (t * xhat).mean(-1, keepdims=True)
        if norm == "layer":
            d = d - t.mean(-1, keepdims=True)
        dx.append(d * r)
    dx.append(np.asarray(dv, dtype=np.float64).transpose(0, 2, 1, 3))
    return np.concatenate(dx, 2).reshape(qkv.shape), dparams


def attention_decode(q, k, v, length, prefix_k=None, prefix_v=None, scale=None):
    """(o [B, Hq, D], weight [B, Hkv, C], spread [B, Hq, D] = sum_j p_j |v_j|, sums [B, Hq]) of one query
    token per sequence over the shared prefix and its own first length[b] keys."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    B, Hq, D = q.shape
    _, Hkv, C, _ = k.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if not scale or scale <= 0 else scale
    o, spread = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    weight, sums = np.zeros((B, Hkv, C)), np.zeros((B, Hq))
    for b in range(B):
        n = min(max(int(length[b]), 0), C)
        for h in range(Hq):
            c = h // G
            keys, vals = k[b, c, :n], v[b, c, :n]
            P = 0
            if prefix_k is not None:
                P = prefix_k.shape[1]
                keys = np.concatenate([np.asarray(prefix_k[c], dtype=np.float64), keys])
                vals = np.concatenate([np.asarray(prefix_v[c], dtype=np.float64), vals])
            if len(keys) == 0:
                continue
            p, _, s, _ = ra_softmax((keys @ q[b, h] * scale)[None])
            o[b, h], spread[b, h] = p[0] @ vals, p[0] @ np.abs(vals)
            weight[b, c, :n] += p[0, P:]
            sums[b, h] = s[0]
    return o, weight, spread, sums


def cache_evict(weight, length, keep, recent):
    """index [B, Hkv, keep] (kept slots ascending, then -1) and the new lengths [B]."""
    weight = np.asarray(weight)
    B, H, C = weight.shape
    index = np.full((B, H, keep), -1, dtype=np.int64)
    new = np.zeros(B, dtype=np.int64)
    for b in range(B):
        n = min(max(int(length[b]), 0), C)
        m, last = min(n, keep), min(recent, n)
        new[b] = m
        for h in range(H):
            w = weight[b, h, :n - last].astype(np.float64)
            w = np.where(np.isnan(w), np.inf, w)
            nan_first = np.isnan(weight[b, h, :n - last])
            order = np.lexsort((np.arange(n - last), -w, ~nan_first))[:m - last]
            index[b, h, :m] = np.concatenate([np.sort(order), np.arange(n - last, n)])
    return index, new
