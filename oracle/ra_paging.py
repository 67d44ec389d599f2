"""CPU oracle of the paged 4-bit cache: plain loops, float64 and exact fractions.

TEST INFRASTRUCTURE, NOT PRODUCT CODE; imports nothing from the product package.  Pins: tests/test_oracle_paging.py.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

GROUP = 64


def bf16_bits_down(x):
    """The largest bfloat16 number <= x (a finite Python float), as a float; -inf below the range."""
    m, e = math.frexp(x)
    if x == 0.0:
        return 0.0
    step = 2.0 ** (max(e, -125) - 8)
    y = math.floor(x / step) * step
    return y if abs(y) < 2.0 ** 128 else math.copysign(math.inf, y)


def bf16_up(x):
    """The least bfloat16 number >= a non-negative Fraction, as a Fraction (possibly beyond the range)."""
    if x == 0:
        return Fraction(0)
    e = math.frexp(float(x))[1]
    for k in (e - 1, e, e + 1):            # float(x) may round to the next power of two
        step = Fraction(2) ** (max(k, -125) - 8)
        n = -((-x) // step)
        if n <= 256:
            return n * step
    raise AssertionError


def quantise_group(x):
    """(codes [64], s, lo) of one group of float64 values that fp32 holds."""
    if not np.all(np.isfinite(x)):
        return np.zeros(GROUP, dtype=np.int64), 0.0, math.nan
    lo = bf16_bits_down(float(x.min()))
    if math.isinf(lo):
        return np.zeros(GROUP, dtype=np.int64), 0.0, math.nan
    span = Fraction(float(x.max())) - Fraction(lo)
    s = bf16_up(span / 15)
    with np.errstate(over="ignore"):
        if np.isinf(np.float32(float(span))) or s >= Fraction(2) ** 128:
            return np.zeros(GROUP, dtype=np.int64), 0.0, math.nan
    if s < Fraction(1, 2 ** 100):
        return np.zeros(GROUP, dtype=np.int64), 0.0, lo
    codes = np.array([round((Fraction(float(v)) - Fraction(lo)) / s) for v in x], dtype=np.int64)   # ties to even
    return codes, float(s), lo


def quantise(x):
    """x [.., D] -> (codes [.., D], s [.., G], lo [.., G])."""
    x = np.asarray(x, dtype=np.float64)
    G = x.shape[-1] // GROUP
    rows = x.reshape(-1, GROUP)
    codes, s, lo = np.zeros(rows.shape, dtype=np.int64), np.zeros(len(rows)), np.zeros(len(rows))
    for i, r in enumerate(rows):
        codes[i], s[i], lo[i] = quantise_group(r)
    lead = x.shape[:-1]
    return codes.reshape(x.shape), s.reshape(*lead, G), lo.reshape(*lead, G)


def held(codes, s, lo):
    shape = codes.shape
    c = codes.reshape(*shape[:-1], -1, GROUP)
    return (lo[..., None] + s[..., None] * c).reshape(shape)


def row_bytes(D):
    return D // 2 + D // 16


def _bf16_bytes(x):
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def store_row(part, page, slot, codes, s, lo):
    """One token's codes [D], s [G], lo [G] into a part: uint8 [page * row]."""
    D = len(codes)
    G = D // GROUP
    words = np.zeros(8 * G, dtype=np.uint32)
    for d in range(D):
        g, w, n = d // 64, d % 64 // 8, d % 8
        words[w * G + g] |= np.uint32(int(codes[d]) << (4 * n))
    row = words.view(np.uint8)
    if D == 128 and slot & 2:
        row = np.concatenate([row[32:], row[:32]])
    part[slot * (D // 2):(slot + 1) * (D // 2)] = row
    at = page * (D // 2) + slot * 4 * G
    bits = np.where(np.isnan(np.concatenate([s, lo])), np.uint16(0x7fc0), _bf16_bytes(np.concatenate([s, lo])))
    part[at:at + 4 * G] = bits.astype(np.uint16).view(np.uint8)


def load_row(part, page, slot, D):
    """(codes, s, lo) of one token of a part."""
    G = D // GROUP
    row = part[slot * (D // 2):(slot + 1) * (D // 2)]
    if D == 128 and slot & 2:
        row = np.concatenate([row[32:], row[:32]])
    words = np.ascontiguousarray(row).view(np.uint32)
    codes = np.array([int(words[(d % 64 // 8) * G + d // 64]) >> (4 * (d % 8)) & 15 for d in range(D)])
    at = page * (D // 2) + slot * 4 * G
    bits = np.ascontiguousarray(part[at:at + 4 * G]).view(np.uint16)
    meta = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return codes, meta[:G], meta[G:]


def _place(table, b, t, page, pages):
    if t < 0 or t >= table.shape[1] * page:
        return -1
    p = int(table[b, t // page])
    return p if 0 <= p < pages else -1


def write(k, v, pool, table, start, count):
    """The pool after the write (a copy), and (codes, s, lo) of k and of v."""
    pool = pool.copy()
    pages, H, _, page, row = pool.shape
    B, _, N, D = k.shape
    flat = pool.reshape(pages, H, 2, page * row)
    parts = [quantise(x) for x in (k, v)]
    for b in range(B):
        for n in range(N if count is None else min(int(count[b]), N)):
            t = n + (0 if start is None else int(start[b]))
            p = _place(table, b, t, page, pages)
            if p < 0:
                continue
            for h in range(H):
                for i, (c, s, lo) in enumerate(parts):
                    store_row(flat[p, h, i], page, t % page, c[b, h, n], s[b, h, n], lo[b, h, n])
    return pool, parts


def dense(pool, table, tokens, D, start=None, length=None):
    """(values, s u, |lo|) [2, B, H, tokens, D] of slots start[b] .. in float64; zeros where nothing is."""
    pages, H, _, page, row = pool.shape
    B = table.shape[0]
    flat = pool.reshape(pages, H, 2, page * row)
    out = np.zeros((3, 2, B, H, tokens, D))
    for b in range(B):
        for n in range(tokens):
            t = n + (0 if start is None else int(start[b]))
            if length is not None and t >= int(length[b]):
                continue
            p = _place(table, b, t, page, pages)
            if p < 0:
                continue
            for h in range(H):
                for i in range(2):
                    c, s, lo = load_row(flat[p, h, i], page, t % page, D)
                    out[0, i, b, h, n] = held(c, s, lo)
                    out[1, i, b, h, n] = c * np.repeat(s, GROUP)
                    out[2, i, b, h, n] = np.abs(np.repeat(lo, GROUP))
    return out


def fork(table, length, uses, parent):
    B = table.shape[0]
    t, n, u = table.copy(), length.copy(), uses.copy()
    for b in range(B):
        p = int(parent[b])
        t[b], n[b] = (table[p], length[p]) if 0 <= p < B else (-1, 0)
    for before, by in ((table, -1), (t, 1)):
        for p in before.ravel():
            if 0 <= p < len(u):
                u[p] += by
    return t, n, u


def reserve(pool, table, length, uses, tokens, count=None):
    """(pool, table, uses, granted) after the call."""
    pool, t, u = pool.copy(), table.copy(), uses.copy()
    page = pool.shape[3]
    B, M = table.shape
    free = [p for p in range(len(uses)) if uses[p] == 0]
    granted = np.zeros(B, dtype=np.int64)
    for b in range(B):
        L = min(max(int(length[b]), 0), M * page)
        n = tokens if count is None else min(max(int(count[b]), 0), tokens)
        granted[b] = min(n, M * page - L)
        if n == 0:
            continue
        for at in range(L // page, min((L + n - 1) // page + 1, M)):
            old = int(table[b, at])
            old = old if 0 <= old < len(uses) else -1
            if old >= 0 and uses[old] <= 1:
                continue
            if not free:
                granted[b] = min(granted[b], max(at * page - L, 0))
                continue
            new = free.pop(0)
            t[b, at] = new
            u[new] += 1
            if old >= 0:
                u[old] -= 1
                if at == L // page and L % page:
                    pool[new] = pool[old]
    return pool, t, u, granted


def compact(pool, table, uses, out):
    """(table, uses, live, out) after the call."""
    out = out.copy()
    live = [p for p in range(len(uses)) if uses[p] > 0]
    kept = live[:len(out)]
    place = {p: i for i, p in enumerate(kept)}
    u = np.zeros(len(out), dtype=np.int64)
    for p, i in place.items():
        out[i] = pool[p]
        u[i] = uses[p]
    t = np.array([[place.get(int(p), -1) for p in row] for row in table]).reshape(table.shape)
    return t, u, len(live), out
