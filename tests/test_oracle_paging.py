"""Pins of the paged cache's oracle: what defines a held group, the layout as a bijection, tables by hand."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import ra_paging as P


def bf16(x):
    return float(torch.tensor(x, dtype=torch.float64).to(torch.bfloat16))


def neighbours(x):
    """The bfloat16 numbers below and above a finite one."""
    bits = int(np.float32(x).view(np.uint32)) >> 16
    def of(b):
        return float(np.uint32(b << 16).view(np.float32))
    if x == 0:
        return -2.0 ** -133, 2.0 ** -133
    return (of(bits - 1), of(bits + 1)) if x > 0 else (of(bits + 1), of(bits - 1))


def test_sixteen_bit_numbers_on_either_side():
    rng = np.random.default_rng(0)
    for x in list(rng.standard_normal(200) * 10.0 ** rng.integers(-39, 38, 200)) + [0.0, 1.0, -1.0, 0.1, 2.0 ** -130, -3e-40, 255.99]:
        x = float(np.float32(x))
        d = P.bf16_bits_down(x)
        assert d == bf16(d) and d <= x < neighbours(d)[1]
        if x > 0:
            u = float(P.bf16_up(Fraction(x)))
            assert u == bf16(u) and neighbours(u)[0] < x <= u
    assert P.bf16_bits_down(-3.4028e38) == -np.inf and P.bf16_up(Fraction(0)) == 0


def test_a_group_is_held_as_defined():
    rng = np.random.default_rng(1)
    for i in range(60):
        x = rng.standard_normal(64) * 10.0 ** rng.integers(-6, 6) + rng.standard_normal()
        x = (torch.from_numpy(x).to(torch.bfloat16 if i % 2 else torch.float32)).double().numpy()
        c, s, lo = P.quantise_group(x)
        assert lo <= x.min() < neighbours(lo)[1] and s == bf16(s)
        span = Fraction(float(x.max())) - Fraction(lo)
        assert 15 * Fraction(s) >= span > 15 * Fraction(neighbours(s)[0])
        assert c.min() >= 0 and c.max() <= 15
        off = np.abs(P.held(c, np.array([s]), np.array([lo])) - x)
        assert np.all(off <= s / 2) and np.all(off <= np.abs(lo + s * np.clip(c + 1, 0, 15) - x))


def test_groups_that_have_no_steps():
    c, s, lo = P.quantise_group(np.full(64, -2.5))
    assert s == 0 and lo == -2.5 and not c.any()
    c, s, lo = P.quantise_group(np.linspace(0, 2.0 ** -99, 64))
    assert s == 0 and lo == 0
    for bad in (np.nan, np.inf, -np.inf):
        x = np.zeros(64)
        x[7] = bad
        c, s, lo = P.quantise_group(x)
        assert s == 0 and np.isnan(lo) and not c.any()
    assert np.isnan(P.quantise_group(np.linspace(-3e38, 3e38, 64))[2])
    # a tie goes to the even code
    x = np.zeros(64)
    x[1], x[2], x[3], x[4] = 15.0, 0.5, 1.5, 2.5
    assert P.quantise_group(x)[0][:5].tolist() == [0, 15, 0, 2, 2]


@pytest.mark.parametrize("D", [64, 128])
def test_the_layout_is_a_bijection(D):
    rng = np.random.default_rng(2)
    page, G = 16, D // 64
    part = np.zeros(page * P.row_bytes(D), dtype=np.uint8)
    rows = [(rng.integers(0, 16, D), np.float32(2.0) ** rng.integers(-9, 9, G), np.float32(-2.0) ** rng.integers(-9, 9, G))
            for _ in range(page)]
    touched = np.zeros(part.shape, dtype=int)
    for t, (c, s, lo) in enumerate(rows):
        before = part.copy()
        part[:] = 0xAA
        P.store_row(part, page, t, c, s, lo)
        one = part.copy()
        part[:] = 0x55
        P.store_row(part, page, t, c, s, lo)
        touched += one == part
        part[:] = before
        P.store_row(part, page, t, c, s, lo)
    assert (touched == 1).all()
    for t, (c, s, lo) in enumerate(rows):
        got = P.load_row(part, page, t, D)
        assert all(np.array_equal(a, b) for a, b in zip(got, (c, s, lo)))


def test_layout_by_hand():
    part = np.zeros(16 * 72, dtype=np.uint8)
    codes = np.zeros(128, dtype=int)
    codes[64 + 8 * 3 + 5] = 9                    # group 1, word 3, nibble 5: word 7, byte 30, high half
    P.store_row(part, 16, 1, codes, np.array([1.0, 2.0]), np.array([-1.0, 0.5]))
    assert part[64 + 30] == 9 << 4 and part[:1024].sum() == 9 << 4
    assert part[1024 + 8:1024 + 16].view(np.uint16).tolist() == [0x3F80, 0x4000, 0xBF80, 0x3F00]
    P.store_row(part, 16, 2, codes, np.zeros(2), np.zeros(2))
    assert part[128 + 32 + 30] == 9 << 4         # bit 1 of the slot: the halves change places


def test_tables_by_hand():
    table = np.array([[3, 1, -1], [3, 4, 0], [-1, -1, -1]], dtype=np.int32)
    length, uses = np.array([20, 40, 0], dtype=np.int32), np.array([1, 1, 0, 2, 1, 0, 0])
    t, n, u = P.fork(table, length, uses, [1, 0, 7])
    assert t.tolist() == [[3, 4, 0], [3, 1, -1], [-1, -1, -1]] and n.tolist() == [40, 20, 0] and u.tolist() == uses.tolist()
    t, n, u = P.fork(table, length, uses, [0, 0, 0])
    assert t.tolist() == [[3, 1, -1]] * 3 and n.tolist() == [20] * 3 and u.tolist() == [0, 3, 0, 3, 0, 0, 0]
    pool = np.arange(7 * 16, dtype=np.uint8).reshape(7, 1, 1, 16, 1)
    p, t2, u2, got = P.reserve(pool, t, n, u, 13)
    # pages 0, 2 and 4 (the lowest free ones) take page 1's place, whose content goes along; then 5, 6 and none
    assert t2.tolist() == [[3, 0, 2], [3, 4, 5], [3, 6, -1]] and got.tolist() == [13, 13, 12]
    assert u2.tolist() == [1, 0, 1, 3, 1, 1, 1] and all(np.array_equal(p[i], pool[1]) for i in (0, 4, 6))
    t3, u3, live, out = P.compact(p, t2, u2, np.zeros((4, 1, 1, 16, 1), dtype=np.uint8))
    assert live == 6 and t3.tolist() == [[2, 0, 1], [2, 3, -1], [2, -1, -1]] and u3.tolist() == [1, 1, 3, 1]
    assert np.array_equal(out, p[[0, 2, 3, 4]])
