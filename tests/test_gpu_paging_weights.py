"""Weights of the paged single-token attention: what a row's output is worth when values differ by many powers of two,
between a token's two groups, between tokens inside and outside the support, and between rows that share a key head.

Every query has one non-zero dimension, a power of two, so that a score is one exact product, times a scale, plus one: the
weights' own errors are what is left.  Bounds, with p the exact weights, s a group's scale, A_j = |q| (|lo| + s u):
  scores and phi   delta = scale 8 2^-24 max_j A_j (three roundings of a score, the scale's, the maximum's difference), phi
                   as in test_gpu_paging.py: e = 2 delta + 64 * 2^-23 of p_j + 1 / s_phi over the support
  weights          p s as two fp16: 2^-22 of each, and 2^-38 of the row's largest (fp16's steps end there), times u <= 15
  codes (bf16)     a code is an fp16 subnormal, up to 2^10 below the exponent that the tensor cores align by: 2^-24 of the
                   largest of sixteen products, each of them and the sum cut: 17 * 2^-14 of the largest p s of sixteen
  sums             n keys, sixteen a product: (n / 16 + 64) 2^-23 of sum_j p_j (|lo| + s u)
and half a step of the output's dtype."""
import numpy as np
import pytest
import torch

from oracle import ra_paging as P
from oracle.ra_oracle import ra_softmax
import rational_softmax_attention_gb300 as ra

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def f64(t):
    return t.detach().cpu().double().numpy()


def bounds(q, held, su, lo, n, dtype, scale):
    """(want, bound) [D] of one row: q [D], and of its key head held, su, |lo| [2, n, D]."""
    D = len(q)
    z = held[0] @ q * scale
    p, _, s, _ = ra_softmax(z[None])
    p, near = p[0], z.max() - z < 16.0 + 1e-3
    want = p @ held[1]
    delta = scale * 8 * 2.0 ** -24 * ((su[0] + lo[0]) @ np.abs(q)).max()
    e = 2 * delta + 64 * 2.0 ** -23
    size = su[1] + lo[1]
    S = p @ size
    codes = p[:, None] * su[1]
    # the largest p s of a group, from its largest s u and u <= 15 (u = 15 occurs in every group that has a step)
    ps = (codes.reshape(n, D // 64, 64).max(-1) / 15.0).repeat(64, -1)
    sixteens = np.add.reduceat(np.maximum.reduceat(ps, np.arange(0, n, 16), 0), [0], 0)[0]
    align = 17 * 2.0 ** -14 * sixteens if dtype == torch.bfloat16 else 0.0
    bound = torch.finfo(dtype).eps / 2 * np.abs(want) + e * (S + size[near].sum(0) / s[0]) + 2.0 ** -22 * codes.sum(0) \
        + 15 * n * 2.0 ** -38 * ps.max(0) + align + (n / 16 + 64) * 2.0 ** -23 * S + 1e-30
    return want, bound


def hold(k, v, page=16):
    """A pool with k, v [B, H, N, D], and its table."""
    B, H, N, D = k.shape
    M = -(-N // page)
    pool = torch.full((B * M, H, 2, page, P.row_bytes(D)), 0xff, dtype=torch.uint8, device="cuda")
    table = torch.arange(B * M, dtype=torch.int32, device="cuda").view(B, M)
    ra.ra_page_write(k.cuda(), v.cuda(), pool, table)
    return pool, table


def one_hot_queries(g, B, Hq, D, low=-1, high=3):
    """Queries with one non-zero dimension, a power of two."""
    q = torch.zeros(B, Hq, D)
    at = torch.randint(0, D, (B, Hq, 1), generator=g)
    size = 2.0 ** torch.randint(low, high, (B, Hq, 1), generator=g).float() * (torch.randint(0, 2, (B, Hq, 1), generator=g) * 2 - 1)
    return q.scatter_(2, at, size)


def check(q, k, v, dtype, length=None):
    B, Hq, D = q.shape
    H, N = k.shape[1:3]
    pool, table = hold(k, v)
    n = [N] * B if length is None else length
    o = f64(ra.ra_attention_decode_paged(q.to(dtype).cuda(), pool, table, torch.tensor(n, dtype=torch.int32, device="cuda"), scale=1.0))
    held, su, lo = P.dense(pool.cpu().numpy(), table.cpu().numpy(), N, D)
    worst = 0.0
    for b in range(B):
        for h in range(Hq):
            c = h // (Hq // H)
            want, bound = bounds(f64(q[b, h]), held[:, b, c, :n[b]], su[:, b, c, :n[b]], lo[:, b, c, :n[b]], n[b], dtype, 1.0)
            worst = max(worst, float((np.abs(o[b, h] - want) / bound).max()))
    assert worst <= 1.0, f"{worst:.3g} times the bound"


HEADS = [(1, 1), (4, 1), (6, 2), (8, 1), (12, 1), (20, 1)]   # the products' forms: up to four rows a key head, eight, sixteen, more


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("N", [8, 12])
def test_more_than_eleven_bits_of_a_weight(N, heads, dtype):
    """Pairs of keys with opposite values: what is left of their sum is small, and so is its rounding; weights of eleven bits
    are beyond the bound (up to 2.2 times it)."""
    g = torch.Generator().manual_seed(3)
    Hq, H = heads
    k, v = (torch.randn(4, H, N, 64, generator=g).repeat_interleave(2, 2)[:, :, :N] for _ in range(2))
    v[:, :, 1::2] *= -1.0
    check(one_hot_queries(g, 4, Hq, 64), k, v, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("apart", [-60, -40, -30, 30, 40, 60])
def test_groups_of_very_different_values(apart, heads, dtype):
    """A token's second group of values 2^apart times its first."""
    g = torch.Generator().manual_seed(heads[0] + apart)
    Hq, H = heads
    k, v = torch.randn(2, H, 45, 128, generator=g), torch.randn(2, H, 45, 128, generator=g)
    v[..., 64:] *= 2.0 ** apart
    check(one_hot_queries(g, 2, Hq, 128), k, v, dtype, [45, 13])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_large_values_outside_the_support(D, heads, dtype):
    """Keys with values 2^45 times the others', which no row or only every other row of a key head sees: their weights are exactly 0
    in the others, before, after and among the keys that count."""
    g = torch.Generator().manual_seed(D + heads[0])
    Hq, H = heads
    N = 150
    k, v = torch.randn(3, H, N, D, generator=g) * 0.5, torch.randn(3, H, N, D, generator=g)
    far = [0, 33, 70, 149]
    v[:, :, far] *= 2.0 ** 45
    k[..., 0] = torch.rand(3, H, N, generator=g) * 8.0
    k[:, :, far, 0] = -40.0                                 # 40 and more below the others for q = 1 in dimension 0
    q = torch.zeros(3, Hq, D)
    q[..., 0] = 1.0
    check(q, k, v, dtype)
    q[:, 1::2, 0] = -1.0                                    # these rows see nothing but the large ones
    check(q, k, v, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_a_value_that_is_not_finite_shows_whatever_its_weight(heads, dtype):
    """0 NaN is NaN: also where all the weights of a block's 32 keys are exactly 0, as where there are others beside it.  It shows in
    every dimension of its group, in the rows of its key head and sequence, and nowhere else."""
    g = torch.Generator().manual_seed(11)
    Hq, H = heads
    B, N, D, G = 4, 100, 128, Hq // H
    k, v = torch.randn(B, H, N, D, generator=g) * 0.25, torch.randn(B, H, N, D, generator=g)
    k[:, :, :, 0] = 30.0
    k[:, :, 32:64, 0] = 0.0                                 # 30 below: a block of weights that are 0
    k[:, :, 70, 0] = 0.0
    v[0, 0, 40, 3], v[1, H - 1, 70, 100], v[2, 0, 63, 64] = float("nan"), float("inf"), -float("inf")
    q = torch.zeros(B, Hq, D)
    q[..., 0] = 1.0
    pool, table = hold(k, v)
    o = ra.ra_attention_decode_paged(q.to(dtype).cuda(), pool, table, torch.full((B,), N, dtype=torch.int32, device="cuda"), scale=1.0)
    want = torch.zeros(B, Hq, D, dtype=torch.bool)
    want[0, :G, :64] = True
    want[1, Hq - G:, 64:] = True
    want[2, :G, 64:] = True
    assert torch.equal(~torch.isfinite(o).cpu(), want)


def test_zeros_of_an_fp32_call_are_zeros():
    """Groups with lo = -8, s = 1: a value of 0 is code 8, exactly.  Dimensions in which all values are 0 come out as 0, and dimensions in
    which all keys are 0 do not move a score, however large the query is there."""
    g = torch.Generator().manual_seed(21)
    for Hq, H in HEADS:
        k, v = (torch.randint(-8, 8, (2, H, 77, 128), generator=g).float() for _ in range(2))
        for t in (k, v):
            t[..., [0, 64]], t[..., [1, 65]] = -8.0, 7.0
        k[..., 5:60], v[..., 70:120] = 0.0, 0.0
        pool, table = hold(k, v)
        n = torch.tensor([77, 40], dtype=torch.int32, device="cuda")
        q = one_hot_queries(g, 2, Hq, 128) * 0.25
        q[..., 5:60] = 0.0
        large = q.clone()
        large[..., 5:60] = torch.randn(2, Hq, 55, generator=g) * 1e4
        o = ra.ra_attention_decode_paged(q.cuda(), pool, table, n, scale=1.0)
        assert (o[..., 70:120] == 0).all() and (o[..., 121:] != 0).any()
        # the large dimensions' products are exact zeros; the small ones are powers of two, 2^-9 at least beside 2^14 for the largest, and
        # fp16 holds them: the scores are the same but for a power of two of the row
        assert torch.equal(o, ra.ra_attention_decode_paged(large.cuda(), pool, table, n, scale=1.0))


@pytest.mark.parametrize("shape", [(8, 3, 3, 64, 5000), (6, 6, 3, 64, 6000), (2, 24, 3, 64, 67), (16, 10, 2, 64, 3), (8, 3, 3, 128, 66), (2, 64, 8, 128, 191)], ids=str)
def test_fp32_errors_are_those_of_a_plain_form(shape):
    """The error against 64 bits over all outputs, next to that of fp32 products, sums and quotients of torch's on the held values: at most
    twice as large."""
    B, Hq, H, D, N = shape
    g = torch.Generator().manual_seed(N)
    k, v = torch.randn(B, H, N, D, generator=g), torch.randn(B, H, N, D, generator=g)
    pool, table = hold(k, v)
    q = torch.randn(B, Hq, D, generator=g).cuda()
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    kh, vh = ra.ra_page_read(pool, table, n, N, dtype=torch.float32)

    def plain(q, kh, vh):
        z = torch.matmul(q.view(B, H, Hq // H, D), kh.transpose(-1, -2)) * D ** -0.5
        u = ((z.amax(-1, keepdim=True) - z) / 16.0).clamp(max=1.0)
        p = ((1.0 - u) / (1.0 + u)) ** 8
        return (torch.matmul(p, vh) / p.sum(-1, keepdim=True)).view(B, Hq, D)

    want = plain(q.double(), kh.double(), vh.double())
    own, other = ((x.double() - want).norm().item() for x in (ra.ra_attention_decode_paged(q, pool, table, n), plain(q, kh, vh)))
    assert own <= 2.0 * other, own / other
