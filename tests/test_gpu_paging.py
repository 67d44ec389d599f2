"""GPU parity of the paged 4-bit cache against its oracle: the pool's bytes, tables and counts exactly; single-token
attention within bounds that follow from its arithmetic.

Tolerances of the attention.  With k_jd = lo + s u, A_j = sum_d |q_d| (|lo| + s u_jd) and delta = scale (D + 4) 2^-23
max_j A_j: a score sums D products and 2 G more in fp32 (the products of codes are exact), and an fp32 query's two
fp16 lose 2^-22 of an element.  phi is off by 2 delta (|d phi / d Delta| <= 1 after the row's maximum, both scores) and by
its own forming, at most 64 * 2^-23 as in test_gpu_decode.py.  So with e = 2 delta + 64 * 2^-23 a weight p_j is off by
e (p_j + 1 / s), s the row's sum of phi; over the values' parts: e (S + R / s), S = sum_j p_j (|lo| + s u), R the same
without weights over the support.  phi s enters the products as fp16, half a step: 2^-11 (fp32: two, 2^-22) of sum_j p_j s u.
Sums over n keys, sixteen a product: (n / 16 + 64) 2^-23 S.  The output's rounding: half a step."""
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


def host(t):
    return t.detach().cpu().numpy()


def table_for(g, lengths, page, M, pages, spare=0):
    """Rows of distinct pages in random order (int32 [B, M], -1 behind them) and the uses."""
    B = len(lengths)
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((B, M), -1, dtype=torch.int32)
    uses = torch.zeros(pages, dtype=torch.int32)
    for b, n in enumerate(lengths):
        for i in range(min(-(-max(n, 0) // page) + spare, M)):
            table[b, i] = p = order.pop()
            uses[p] = 1
    return table, uses


def random_pool(g, pages, H, page, D):
    """Any bytes, with NaNs among what the scales and minima would be."""
    pool = torch.randint(0, 256, (pages, H, 2, page, P.row_bytes(D)), generator=g, dtype=torch.uint8)
    return pool


def filled(g, lengths, H, page, D, M, sigma=1.0, extra=3, bad=()):
    """A pool that holds quantised random rows for these lengths, every other byte 0xff (NaN scales and minima), its table."""
    B = len(lengths)
    pages = sum(-(-max(min(n, M * page), 0) // page) for n in lengths) + extra
    table, _ = table_for(g, [min(n, M * page) for n in lengths], page, M, pages)
    N = max(1, max(min(n, M * page) for n in lengths))
    k = (torch.randn(B, H, N, D, generator=g) + 0.5 * torch.randn(1, H, 1, D, generator=g)) * sigma
    v = torch.randn(B, H, N, D, generator=g)
    pool = torch.full((pages, H, 2, page, P.row_bytes(D)), 0xff, dtype=torch.uint8).cuda()
    n = torch.tensor(lengths, dtype=torch.int32)
    for b, at in bad:
        table[b, at] = (-1, pages, 1 << 30, -(1 << 31))[at % 4]
    table = table.cuda()
    ra.ra_page_write(k.cuda(), v.cuda(), pool, table, count=n.cuda())
    return pool, table, n.cuda()


# ---- rows in and out ----------------------------------------------------------------------------------------
ROWS = [  # B, H, N, D, page, starts
    (1, 1, 1, 64, 16, [0]),
    (3, 2, 5, 128, 16, [0, 14, 31]),
    (2, 3, 37, 64, 32, [11, 90]),
    (2, 1, 130, 128, 64, [63, 0]),
    (5, 4, 1, 128, 256, [0, 255, 256, 3, 511]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_rows_are_held_bit_for_bit(case, dtype):
    B, H, N, D, page, starts = case
    g = torch.Generator().manual_seed(N + D)
    M = -(-(max(starts) + N) // page) + 1
    table, _ = table_for(g, [s + N for s in starts], page, M, B * M + 2)
    pool = random_pool(g, B * M + 2, H, page, D)
    k, v = ((torch.randn(B, H, N, D, generator=g) * s + o).to(dtype) for s, o in ((1.0, 0.3), (20.0, 0.0)))
    want, parts = P.write(f64(k), f64(v), host(pool), host(table), starts, None)
    cu = pool.cuda()
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    kh, vh = ra.ra_page_write(k.cuda(), v.cuda(), cu, table.cuda(), start, held=True)
    assert np.array_equal(host(cu), want)
    again = pool.cuda()
    assert ra.ra_page_write(k.cuda(), v.cuda(), again, table.cuda(), start) is None and torch.equal(again, cu)
    for x, got, (c, s, lo) in ((k, kh, parts[0]), (v, vh, parts[1])):
        exact = torch.from_numpy(P.held(c, s, lo))
        assert got.dtype == dtype and torch.equal(got.cpu(), exact.to(torch.float32).to(dtype))
        assert np.all(np.abs(exact.numpy() - f64(x)) <= np.repeat(s, 64, -1) / 2)
    for r, t in zip(ra.ra_page_read(cu, table.cuda(), None, N, start=start, dtype=dtype), (kh, vh)):
        assert torch.equal(r, t)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_many_tokens_and_heads(D):
    """Several steps of the grid; compared with what one call per head writes, and bit for bit at some rows."""
    g = torch.Generator(device="cuda").manual_seed(5)
    B, H, N, page = 3, 5, 3001, 64
    M = -(-N // page)
    table = torch.randperm(B * M, generator=g, device="cuda").to(torch.int32).view(B, M)
    k, v = (torch.randn(B, H, N, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pool = torch.zeros(B * M, H, 2, page, P.row_bytes(D), dtype=torch.uint8, device="cuda")
    kh, vh = ra.ra_page_write(k, v, pool, table, held=True)
    for h in range(H):
        one = torch.zeros(B * M, 1, 2, page, P.row_bytes(D), dtype=torch.uint8, device="cuda")
        k1, v1 = ra.ra_page_write(k[:, h:h + 1], v[:, h:h + 1], one, table, held=True)
        assert torch.equal(one[:, 0], pool[:, h]) and torch.equal(k1[:, 0], kh[:, h]) and torch.equal(v1[:, 0], vh[:, h])
    at = [0, 1, 63, 64, 1500, 2999, 3000]
    for x, y in ((k, kh), (v, vh)):
        assert torch.equal(torch.from_numpy(P.held(*P.quantise(f64(x[:, 4, at])))).float().bfloat16(), y[:, 4, at].cpu())
    for x, y in zip(ra.ra_page_read(pool, table, None, N), (kh, vh)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_at_every_border(dtype):
    """Ties between codes, constant rows, zeros of both signs, the largest and smallest magnitudes, mixed exponents
    (differences that fp32 rounds), infinities and NaN."""
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(3)
    rows = [torch.arange(64) * 0.25, torch.arange(64) * 15.0 / 63, torch.full((64,), 3.7), torch.zeros(64),
            -torch.zeros(64), torch.cat([torch.zeros(63), -torch.zeros(1)]), torch.randn(64, generator=g) * 1e-37,
            torch.randn(64, generator=g) * 2.0 ** -101, torch.randn(64, generator=g) * 1e37,
            torch.linspace(-3.38e38, 3.38e38, 64), torch.linspace(-1e38, 2e38, 64), torch.full((64,), -3.4e38),
            torch.cat([torch.tensor([-3.0, 12.0]), 2.0 ** -torch.arange(62).float()]),
            torch.cat([torch.tensor([-3.0, 12.0]), -2.0 ** -torch.arange(62).float()]),
            torch.cat([torch.tensor([2.0 ** -20, 15.0]), torch.arange(62) * 0.25]),
            torch.cat([torch.tensor([-2.0 ** -30]), torch.arange(63) * 0.5]),
            torch.cat([torch.tensor([0.0, 15.0]), torch.arange(62) + 0.5]),
            torch.cat([torch.tensor([inf]), torch.randn(63, generator=g)]),
            torch.cat([torch.randn(63, generator=g), torch.tensor([-inf])]), torch.full((64,), inf),
            torch.cat([torch.randn(31, generator=g), torch.tensor([nan]), torch.randn(32, generator=g)]), torch.full((64,), nan)]
    rows += [torch.randint(-40, 41, (64,), generator=g) * 2.0 ** int(e) for e in torch.randint(-12, 12, (40,), generator=g)]
    rows += [torch.randn(64, generator=g) * 2.0 ** (torch.randint(-24, 1, (64,), generator=g)) for _ in range(20)]
    x = torch.stack(rows).float()
    x = x.view(1, 1, len(rows), 64)
    x = torch.cat([x, x.flip(2)], -1).to(dtype)                    # two groups per row
    N = x.shape[2]
    pool = torch.zeros(-(-N // 16), 1, 2, 16, 72, dtype=torch.uint8)
    table = torch.arange(pool.shape[0], dtype=torch.int32).view(1, -1)
    want, parts = P.write(f64(x), f64(-x), host(pool), host(table), None, None)
    cu = pool.cuda()
    kh, vh = ra.ra_page_write(x.cuda(), (-x).cuda(), cu, table.cuda(), held=True)
    assert np.array_equal(host(cu), want)
    for got, (c, s, lo) in ((kh, parts[0]), (vh, parts[1])):
        exact = torch.from_numpy(P.held(c, s, lo)).float().to(dtype)
        assert torch.equal(got.cpu().nan_to_num(nan=7.0), exact.nan_to_num(nan=7.0))
    for a, b in zip(ra.ra_page_read(cu, table.cuda(), None, N, dtype=dtype), (kh, vh)):
        assert torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))


def test_strides_counts_and_slots_outside():
    """Slices of a packed projection, transposed, expanded and misaligned tensors; counts; slots and pages that are
    none; every byte that is not addressed stays."""
    g = torch.Generator().manual_seed(8)
    B, H, N, D, page = 3, 2, 20, 128, 16
    packed = torch.randn(B, N, 4 * H * D, generator=g).bfloat16()
    k = packed[..., :H * D].view(B, N, H, D).transpose(1, 2)
    v = packed[..., H * D:2 * H * D].view(B, N, H, D).transpose(1, 2)
    table = torch.tensor([[4, -1, 2, 9], [0, 1, 3, 5], [99, 6, -7, 7]], dtype=torch.int32)
    starts, counts = [10, -5, 30], [20, 99, -1]
    pool = random_pool(g, 10, H, page, D)
    want, _ = P.write(f64(k), f64(v), host(pool), host(table), starts, [20, 20, 0])
    shift = torch.empty(B * H * N * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(B, H, N, D)
    shift.copy_(k)
    forms = {"slices": (packed.cuda()[..., :H * D].view(B, N, H, D).transpose(1, 2),
                        packed.cuda()[..., H * D:2 * H * D].view(B, N, H, D).transpose(1, 2)),
             "misaligned": (shift, v.cuda()),
             "strided": (k.cuda().repeat_interleave(2, -1)[..., ::2], v.cuda().transpose(-1, -2).contiguous().transpose(-1, -2))}
    for name, (kk, vv) in forms.items():
        cu = pool.cuda()
        ra.ra_page_write(kk, vv, cu, table.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(),
                         count=torch.tensor(counts, dtype=torch.int32).cuda())
        assert np.array_equal(host(cu), want), name
    kk, vv = ra.ra_page_read(pool.cuda(), table.cuda(), torch.tensor([64, 9, 40], dtype=torch.int32).cuda(), 50,
                             start=torch.tensor([-3, 0, 25], dtype=torch.int32).cuda(), dtype=torch.float32)
    d = P.dense(host(pool), host(table), 50, D, [-3, 0, 25], [64, 9, 40])[0]
    for got, w in ((kk, d[0]), (vv, d[1])):
        with np.errstate(over="ignore", invalid="ignore"):
            assert np.array_equal(host(got), w.astype(np.float32), equal_nan=True)
    one = torch.randn(1, H, 1, D, generator=g).bfloat16().cuda().expand(B, H, N, D)
    cu, cd = pool.cuda(), pool.cuda()
    ra.ra_page_write(one, one, cu, table.cuda())
    ra.ra_page_write(one.contiguous(), one.contiguous(), cd, table.cuda())
    assert torch.equal(cu, cd)


# ---- single tokens --------------------------------------------------------------------------------------------
def check_decode(q, pool, table, length, scale=None):
    """Runs the call, checks it against the oracle on the values that the pool holds; returns o."""
    B, Hq, D = q.shape
    pages, H, _, page, _ = pool.shape
    o = ra.ra_attention_decode_paged(q.cuda(), pool, table, length, scale=scale)
    torch.cuda.synchronize()
    assert o.dtype == q.dtype and o.shape == q.shape
    n = [min(max(int(x), 0), table.shape[1] * page) for x in length.tolist()]
    held, su, lo = P.dense(host(pool), host(table), max(1, max(n)), D, None, n)
    sc = D ** -0.5 if not scale else scale
    got, G = f64(o), Hq // H
    loss = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22
    half = torch.finfo(q.dtype).eps / 2
    for b in range(B):
        for h in range(Hq):
            if n[b] == 0:
                assert np.all(got[b, h] == 0)
                continue
            c, qd = h // G, f64(q[b, h])
            z = held[0, b, c, :n[b]] @ qd * sc
            p, _, s, _ = ra_softmax(z[None])
            p = p[0]
            want = p @ held[1, b, c, :n[b]]
            delta = sc * (D + 4) * 2.0 ** -23 * ((su[0, b, c, :n[b]] + lo[0, b, c, :n[b]]) @ np.abs(qd)).max()
            e = 2 * delta + 64 * 2.0 ** -23
            near = z.max() - z < 16.0 + 1e-3
            size = su[1, b, c, :n[b]] + lo[1, b, c, :n[b]]
            S = p @ size
            bound = half * np.abs(want) + e * (S + size[near].sum(0) / s[0]) + loss * (p @ su[1, b, c, :n[b]]) \
                + (n[b] / 16 + 64) * 2.0 ** -23 * S + 1e-30
            err = np.abs(got[b, h] - want)
            assert np.all(err <= bound), f"sequence {b}, head {h}: beyond its bound by {np.max(err - bound):.3e}"
    return o


CASES = [  # B, Hq, Hkv, D, page, M, sigma, lengths
    (1, 1, 1, 64, 16, 1, 1.0, [1]),
    (1, 16, 16, 128, 64, 8, 1.0, [300]),
    (2, 4, 2, 64, 16, 3, 1.0, [0, 33]),                     # a sequence without any key
    (3, 6, 2, 128, 32, 5, 1.0, [31, 32, 129]),
    (3, 8, 1, 64, 256, 2, 2.0, [300, 1, 257]),
    (2, 20, 1, 128, 64, 11, 1.0, [700, 513]),               # more query heads than a block of rows
    (2, 9, 1, 128, 16, 11, 1.0, [170, 3]),
    (2, 16, 1, 64, 128, 3, 1.0, [384, 383]),
    (9, 16, 8, 128, 16, 5, 3.0, [65, 64, 63, 33, 32, 31, 1, 0, 2]),
    (1, 5, 5, 64, 64, 40, 3.0, [2500]),
    (2, 2, 1, 128, 16, 1, 1.0, [-3, 99]),                   # lengths outside the cache
    (150, 4, 1, 64, 16, 3, 1.0, [i % 48 for i in range(150)]),
    (40, 8, 4, 128, 32, 9, 1.0, [7 * i for i in range(40)]),
    (8192, 1, 1, 64, 16, 1, 1.0, [i % 4 for i in range(8192)]),   # as many sequences as there may be
    (1, 1024, 1, 64, 32, 3, 1.0, [69]),                     # and as many query heads per key head
    (70, 2, 1, 64, 16, 300, 1.0, [4700 if i == 9 else i % 5 for i in range(70)]),
    # a warp's runs, each sequence cut for itself or not; a CTA's runs over several sequences
    (70, 8, 8, 64, 16, 20, 1.0, [(37 * i) % 321 for i in range(70)]),
    (300, 4, 4, 64, 16, 5, 1.0, [i % 71 for i in range(300)]),
    (310, 24, 4, 128, 32, 1, 1.0, [i % 31 for i in range(310)]),
    (50, 16, 8, 128, 32, 6, 1.0, [150 - 3 * i for i in range(50)]),
    (45, 72, 8, 64, 16, 8, 2.0, [11 + i % 100 for i in range(45)]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode_matches_the_oracle(case, dtype):
    B, Hq, H, D, page, M, sigma, lengths = case
    g = torch.Generator().manual_seed(Hq + M)
    pool, table, n = filled(g, lengths, H, page, D, M, sigma)
    q = (torch.randn(B, Hq, D, generator=g) * sigma).to(dtype)
    check_decode(q, pool, table, n)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_scales_of_every_size(dtype):
    """Values and queries far from 1, scales that grow from page to page (the products' power of two follows them), rows of
    queries of very different sizes, queries of zeros."""
    g = torch.Generator().manual_seed(4)
    B, Hq, H, D, page, N = 2, 8, 2, 128, 16, 200
    pages = B * 13
    table = torch.arange(pages, dtype=torch.int32).view(B, 13).cuda()
    for size in (1e-30, 1e-6, 1e6, 1e30):
        k = torch.randn(B, H, N, D, generator=g)
        v = torch.randn(B, H, N, D, generator=g) * 2.0 ** torch.linspace(-20, 12, N).view(1, 1, N, 1) * size
        q = torch.randn(B, Hq, D, generator=g) * 10.0 ** torch.linspace(-30, 0, Hq).view(1, Hq, 1)
        q[1, 3] = 0.0
        pool = torch.full((pages, H, 2, page, 72), 0xff, dtype=torch.uint8, device="cuda")
        ra.ra_page_write(k.cuda(), v.cuda(), pool, table)
        check_decode(q.to(dtype), pool, table, torch.tensor([N, 77], dtype=torch.int32).cuda())
        # large queries against small keys: the same scores
        ra.ra_page_write((k * 1e-20).cuda(), v.cuda(), pool, table)
        check_decode((q * 1e20).to(dtype), pool, table, torch.tensor([N, 77], dtype=torch.int32).cuda())


def test_decode_of_bad_and_shared_pages():
    g = torch.Generator().manual_seed(6)
    for page in (16, 64):
        pool, table, n = filled(g, [150, 100, 200], 2, page, 128, 13, bad=[(0, 0), (1, 1), (2, 2), (2, 0)])
        q = torch.randn(3, 8, 128, generator=g).bfloat16()
        check_decode(q, pool, table, n)
    table[1], table[2] = table[0], table[0]
    o = check_decode(q[:1].expand(3, -1, -1).contiguous(), pool, table, n[:1].expand(3).contiguous())
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])


def test_decode_not_finite():
    """A NaN in a key or value shows in the heads that read it, and nowhere else."""
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(2, 2, 50, 64, generator=g) for _ in range(2))
    k[0, 0, 17, 5], v[1, 1, 3, 9] = float("nan"), float("inf")
    pool = torch.zeros(8, 2, 2, 16, 36, dtype=torch.uint8, device="cuda")
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    ra.ra_page_write(k.cuda(), v.cuda(), pool, table)
    for dtype in DTYPES:
        q = torch.randn(2, 4, 64, generator=g).to(dtype).cuda()
        bad = (~torch.isfinite(ra.ra_attention_decode_paged(q, pool, table, torch.full((2,), 50, dtype=torch.int32, device="cuda")))).cpu()
        assert bad[0, :2].any(-1).all() and not bad[0, 2:].any() and not bad[1, :2].any() and bad[1, 2:].any(-1).all()


def test_decode_long_context_and_layers():
    """Many parts per row, a pool that is one layer's slice of a larger tensor, offsets beyond 2^31 bytes."""
    g = torch.Generator(device="cuda").manual_seed(9)
    N, page, H, D, layers = 40000, 64, 1, 64, 64
    M = -(-N // page)
    whole = torch.empty(7600, layers, H, 2, page, 36, dtype=torch.uint8, device="cuda")       # 2.2 GB
    pool = whole[:, layers - 1]
    assert pool.stride(0) * 7599 > 1 << 31
    table = (7599 - torch.arange(M, device="cuda", dtype=torch.int32)).view(1, M).contiguous()
    k, v = (torch.randn(1, H, N, D, generator=g, device="cuda") for _ in range(2))
    before = whole[:, :layers - 1].sum(dtype=torch.int64)
    kh, vh = ra.ra_page_write(k, v, pool, table, held=True)
    assert whole[:, :layers - 1].sum(dtype=torch.int64) == before
    for dtype in DTYPES:
        q = torch.randn(1, 24, D, generator=g, device="cuda").to(dtype)
        o = ra.ra_attention_decode_paged(q, pool, table, torch.tensor([N], dtype=torch.int32, device="cuda"))
        z = (q.double().view(24, D) @ kh[0, 0].double().T) / 8.0
        gap = z.max(-1, keepdim=True).values - z
        p = torch.where(gap < 16.0, (16.0 - gap) / (16.0 + gap), 0.0) ** 8
        p = p / p.sum(-1, keepdim=True)
        want = p @ vh[0, 0].double()
        # scores of up to about 40 (2^-18 off), sums of 40000: far below the rounding of bf16, 1e-4 of the spread in fp32
        half = torch.finfo(dtype).eps / 2
        spread = p @ vh[0, 0].double().abs()
        assert ((o[0].double() - want).abs() <= half * want.abs() + (2.0 ** -11 if dtype == torch.bfloat16 else 1e-4) * spread).all()
        assert torch.equal(o, ra.ra_attention_decode_paged(q, pool, table, torch.tensor([N], dtype=torch.int32, device="cuda")))


def test_decode_with_a_workspace_at_any_16_bytes():
    """The C call takes a workspace at a 16-byte address, and stays inside it."""
    L = ra.lib()
    g = torch.Generator().manual_seed(12)
    pool, table, n = filled(g, [500, 90, 0], 2, 16, 128, 40)
    for G in (4, 8, 16):
        q = torch.randn(3, 2 * G, 128, generator=g).bfloat16().cuda()
        want = ra.ra_attention_decode_paged(q, pool, table, n)
        size = L.ra_attention_decode_paged_workspace_size(3, 2 * G, 2, 40, 16, 128)
        ws = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        for off in (16, 48, 112, 128):
            o = torch.zeros_like(q)
            code = L.ra_attention_decode_paged(q.data_ptr(), pool.data_ptr(), pool.stride(0), table.data_ptr(), n.data_ptr(), o.data_ptr(),
                                               ws.data_ptr() + off, 3, 2 * G, 2, 128, pool.shape[0], 16, 40, 0.0, 1,
                                               torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert code == 0 and torch.equal(o, want)
            assert (ws[:16] == 0xA5).all() and (ws[off + size:] == 0xA5).all()


# ---- the table ------------------------------------------------------------------------------------------------
def same(*pairs):
    for got, want in pairs:
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("seed", range(6))
def test_table_operations_match_the_oracle(seed):
    """Forks, reservations (shared pages copied, some without enough pages) and compactions in turn."""
    g = torch.Generator().manual_seed(seed)
    page, H, D = (16, 32, 64)[seed % 3], 1 + seed % 2, (64, 128)[seed % 2]
    B, M, pages = (1, 7, 40, 33, 12, 300)[seed], 6, (9, 30, 150, 60, 50, 700)[seed]
    pool = random_pool(g, pages, H, page, D)
    start = torch.randint(0, max(2, pages * page // B // 2), (B,), generator=g).clamp(max=M * page)
    table, uses = table_for(g, start.tolist(), page, M, pages)
    length = start.to(torch.int32)
    dev = [t.cuda() for t in (pool, table, length, uses)]
    h = [host(t) for t in (pool, table, length, uses)]
    for turn in range(6):
        parent = torch.randint(-1, B, (B,), generator=g).to(torch.int32)
        keep = torch.rand(B, generator=g) < 0.5
        parent = torch.where(keep, torch.arange(B, dtype=torch.int32), parent)
        if turn == 3:
            parent[0] = B + 5
        ra.ra_page_fork(dev[1], dev[2], dev[3], parent.cuda())
        h[1], h[2], h[3] = P.fork(h[1], h[2], h[3], parent.numpy())
        same((dev[1], h[1]), (dev[2], h[2]), (dev[3], h[3]))
        tokens = int(torch.randint(1, 3 * page, (1,), generator=g)) if turn % 2 else 1
        count = torch.randint(-1, tokens + 2, (B,), generator=g).to(torch.int32) if turn % 3 else None
        granted = ra.ra_page_reserve(dev[0], dev[1], dev[2], dev[3], tokens, count=None if count is None else count.cuda())
        h[0], h[1], h[3], want = P.reserve(h[0], h[1], h[2], h[3], tokens, count)
        same((dev[0], h[0]), (dev[1], h[1]), (dev[3], h[3]), (granted, want))
        assert np.array_equal(np.bincount(h[1][h[1] >= 0], minlength=pages), h[3])
        dev[2] += granted
        h[2] = (h[2] + want).astype(np.int32)
        for size in (pages, int((h[3] > 0).sum()) // 2 + 1):
            out = random_pool(g, size, H, page, D)
            got = out.cuda()
            t, u, live = ra.ra_page_compact(dev[0], dev[1], dev[3], got)
            wt, wu, wl, wo = P.compact(h[0], h[1], h[3], host(out))
            same((t, wt), (u, wu), (got, wo))
            assert live.item() == wl


@pytest.mark.parametrize("pages", [1, 255, 2048, 8192, 65537, 200000])
def test_pages_of_large_pools(pages):
    """Ranks over many warps and CTAs; tables wider than a CTA's columns."""
    g = torch.Generator().manual_seed(pages)
    uses = (torch.rand(pages, generator=g) < 0.6).to(torch.int32)
    free = (uses == 0).nonzero().flatten()
    B, M, page = 33, 1000, 16
    table = torch.full((B, M), -1, dtype=torch.int32)
    live = (uses > 0).nonzero().flatten().to(torch.int32)[:B * M // 2]
    uses.zero_()
    uses[live.long()] = 1
    free = (uses == 0).nonzero().flatten()
    table.view(-1)[:live.numel()] = live
    length = ((table >= 0).sum(1) * page).to(torch.int32)
    pool = torch.zeros(pages, 1, 2, page, 36, dtype=torch.uint8, device="cuda")
    pool[:, 0, 0, 0, :4] = torch.arange(pages, device="cuda", dtype=torch.int32).view(-1, 1).view(torch.uint8)
    t, n, u = table.cuda(), length.cuda(), uses.cuda()
    out = torch.zeros(live.numel() + 3, 1, 2, page, 36, dtype=torch.uint8, device="cuda")
    ct, cu, count = ra.ra_page_compact(pool, t, u, out)
    assert count.item() == live.numel()
    order = live.sort().values
    assert torch.equal(out[:live.numel(), 0, 0, 0, :4].contiguous().view(torch.int32).flatten().cpu(), order)
    assert (cu[:live.numel()] == 1).all() and (cu[live.numel():] == 0).all() and torch.equal(ct >= 0, t >= 0)
    assert torch.equal(order[ct[ct >= 0].long().cpu()], table[table >= 0])
    granted = ra.ra_page_reserve(pool, t, n, u, 300)
    want = []
    left = free.numel()
    for b in range(B):
        touched = min(-(-300 // page), M - int(length[b]) // page)
        got = min(touched, left)
        left -= got
        want.append(min(got * page, 300, M * page - int(length[b])))
    assert granted.tolist() == want
    took = t[(t >= 0) & (table.cuda() < 0)]
    assert torch.equal(took.cpu().long(), free[:took.numel()]) and (u[took.long()] == 1).all()
    parent = torch.randint(0, B, (B,), generator=g, dtype=torch.int32)
    before = t.clone()
    ra.ra_page_fork(t, n, u, parent.cuda())
    assert torch.equal(t, before[parent.long().cuda()])
    assert torch.equal(torch.bincount(t[t >= 0].long(), minlength=pages), u.long())


def test_fork_of_as_many_rows_as_there_may_be():
    g = torch.Generator(device="cuda").manual_seed(1)
    B, M = 8192, 13
    table = torch.arange(B * M, device="cuda", dtype=torch.int32).view(B, M)
    t, n, u = table.clone(), torch.arange(B, device="cuda", dtype=torch.int32), torch.ones(B * M, device="cuda", dtype=torch.int32)
    parent = torch.randperm(B, generator=g, device="cuda").to(torch.int32)
    ra.ra_page_fork(t, n, u, parent)
    assert torch.equal(t, table[parent.long()]) and torch.equal(n, parent) and (u == 1).all()


# ---- together -------------------------------------------------------------------------------------------------
def make_module(dtype=torch.bfloat16, dim=256, heads=4):
    torch.manual_seed(0)
    return ra.RaAttention(dim, num_heads=heads, qk_norm=True, causal=True, rope_sections=(32,), device="cuda", dtype=dtype)


def test_module_prompt_and_single_tokens_see_the_same_cache():
    """A prompt attends to what the cache holds, so its rows are those of single tokens one after the other: fp32
    scores on both sides (the two kernels' scores and sums differ by their order, 1e-4 at most at these sizes)."""
    m = make_module(torch.float32)
    x = torch.randn(3, 40, 256, device="cuda")
    count = torch.tensor([40, 23, 1], dtype=torch.int32, device="cuda")
    a, b = (m.new_cache(3, 64, page_size=16) for _ in range(2))
    y = m.prefill(x, a, count=count)
    for i in range(40):
        z = m.decode(x[:, i:i + 1], b)
        assert all((z[s, 0] - y[s, i]).abs().max() < 1e-4 for s in range(3) if i < count[s])
    assert a.length.tolist() == count.tolist() and b.length.tolist() == [40, 40, 40] and a.bound == 40
    for s in range(3):
        c = int(count[s])
        for p, q in zip(a.read(c), b.read(c)):
            assert torch.equal(p[s, :, :c], q[s, :, :c])


def test_module_generation_with_forks():
    """One prompt forked into four, continued by different prompts, then single tokens, a reordering and a compaction on
    the way: the same numbers as every sequence gives from its own start.  Both sides round to bf16 once per
    projection and output (values of about 1: 2^-8 each, some ten of them): 6e-2, as in the smoke test."""
    m = make_module()
    prompt, parts = torch.randn(1, 50, 256, device="cuda").bfloat16(), torch.randn(4, 21, 256, device="cuda").bfloat16()
    steps = torch.randn(4, 30, 256, device="cuda").bfloat16()
    c = m.new_cache(4, 128, page_size=16, pages=30)
    m.prefill(prompt.expand(4, -1, -1), c, count=torch.tensor([50, 0, 0, 0], dtype=torch.int32, device="cuda"))
    assert (c.uses > 0).sum() == 4
    c.fork(torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert c.length.tolist() == [50] * 4 and c.position.tolist() == [50] * 4 and (c.uses > 0).sum() == 4
    got = [m.prefill(parts, c)]
    assert c.length.tolist() == [71] * 4 and (c.uses > 0).sum() == 3 + 4 * 2
    order = list(range(4))
    for i in range(30):
        if i == 10:
            c.fork(torch.tensor([1, 1, 3, 0], dtype=torch.int32, device="cuda"))
            order = [order[p] for p in (1, 1, 3, 0)]
        if i == 20:
            c.compact()
            assert (c.uses > 0).all() and c.pages == c.uses.numel()
            c.compact(40)
        got.append(m.decode(steps[order, i:i + 1], c))
    own = torch.cat([prompt.expand(4, -1, -1), parts, steps], 1)
    full = m.new_cache(4, 128, page_size=64)
    want = m.prefill(own, full)
    for i, y in enumerate(got):
        rows = [0, 1, 2, 3] if i <= 10 else order
        w = want[:, 50:71] if i == 0 else want[rows, 70 + i:71 + i]
        assert (y.float() - w.float()).abs().max() < 6e-2, i
    assert c.length.tolist() == [101] * 4
    c.free([1, 3])
    assert c.length.tolist() == [101, 0, 101, 0] and c.position.tolist() == [101, 0, 101, 0]
    c.free([0, 2])
    assert (c.uses == 0).all() and (c.table == -1).all()


def test_a_freed_cache_takes_prompts_again():
    """Also in fp32, where only an empty cache does."""
    m = make_module(torch.float32)
    x = torch.randn(2, 9, 256, device="cuda")
    c = m.new_cache(2, 16, page_size=16)
    want = m.prefill(x, c)
    with pytest.raises(NotImplementedError, match="bf16"):
        m.prefill(x[:, :2], c)
    c.free([0, 1])
    assert c.bound == 0 and torch.equal(m.prefill(x, c), want)
    with pytest.raises(ValueError, match="no room"):
        for _ in range(8):
            m.decode(x[:, :1], c)
    assert c.length.tolist() == [16, 16]


def test_refusals_on_the_device():
    """What the host's checks let through only as far as the device's tensors."""
    pool, table = ra.ra_page_pool(4, 2, 64, 16), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    n, k = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 5, 64, device="cuda")
    uses = torch.zeros(4, dtype=torch.int32, device="cuda")
    for call in (lambda: ra.ra_page_write(k[:, :1], k[:, :1], pool, table), lambda: ra.ra_page_write(k, k.bfloat16(), pool, table),
                 lambda: ra.ra_page_write(k, k, pool, table.long()), lambda: ra.ra_page_write(k, k, pool, table[:1]),
                 lambda: ra.ra_page_write(k, k, pool, table, n[:1]), lambda: ra.ra_page_write(k, k, pool, table, n.cpu()),
                 lambda: ra.ra_page_write(k, k, pool.transpose(0, 1), table), lambda: ra.ra_page_write(k, k, pool[..., :35], table),
                 lambda: ra.ra_page_write(k, k, pool[:, :, :, ::2], table), lambda: ra.ra_page_write(k, k, pool[:1].expand(4, -1, -1, -1, -1), table),
                 lambda: ra.ra_page_read(pool, table, n, 0), lambda: ra.ra_page_read(pool, table.t(), n, 1),
                 lambda: ra.ra_attention_decode_paged(torch.zeros(2, 3, 64, device="cuda"), pool, table, n),
                 lambda: ra.ra_attention_decode_paged(torch.zeros(2, 4, 128, device="cuda"), pool, table, n),
                 lambda: ra.ra_attention_decode_paged(torch.zeros(1, 4, 64, device="cuda"), pool, table, n),
                 lambda: ra.ra_attention_decode_paged(torch.zeros(2, 64, 4, device="cuda").transpose(1, 2), pool, table, n),
                 lambda: ra.ra_page_fork(table, n, uses, uses), lambda: ra.ra_page_fork(table, n, uses.float(), n),
                 lambda: ra.ra_page_reserve(pool, table, n, uses[:3], 1), lambda: ra.ra_page_reserve(pool, table, n, uses, 0),
                 lambda: ra.ra_page_compact(pool, table, uses, pool), lambda: ra.ra_page_compact(pool, table, uses, pool[2:]),
                 lambda: ra.ra_page_compact(pool, table, uses, ra.ra_page_pool(4, 2, 128, 16)),
                 lambda: ra.ra_page_compact(pool, table, uses, ra.ra_page_pool(4, 1, 64, 16))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ra.ra_page_write(k.half(), k.half(), pool, table)
    with pytest.raises(ra.RaError):
        ra.ra_attention_decode_paged(torch.zeros(2, 4, 64, device="cuda"), pool, table, n, scale=float("inf"))
    with pytest.raises(ra.RaError):
        ra.ra_page_fork(torch.zeros(8193, 1, dtype=torch.int32, device="cuda"), torch.zeros(8193, dtype=torch.int32, device="cuda"), uses,
                        torch.zeros(8193, dtype=torch.int32, device="cuda"))
    layers = torch.zeros(4, 3, 2, 2, 16, 36, dtype=torch.uint8, device="cuda")
    ra.ra_page_compact(layers[:, 0], table, uses, layers[:, 2])          # layers of one tensor do not overlap


def test_a_captured_step_replays():
    """reserve, write and attend in a graph, over page borders, next to the same steps outside."""
    m = make_module()
    x = torch.randn(2, 40, 256, device="cuda").bfloat16()
    a, b = (m.new_cache(2, 64, page_size=16) for _ in range(2))
    static = torch.zeros(2, 1, 256, device="cuda", dtype=torch.bfloat16)
    m.prefill(x[:, :5], a)
    m.prefill(x[:, :5], b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        static.copy_(x[:, 5:6])
        m.decode(static, a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = m.decode(static, a)
    torch.cuda.current_stream().wait_stream(side)
    m.decode(x[:, 5:6], b)
    for i in range(6, 40):
        static.copy_(x[:, i:i + 1])
        graph.replay()
        assert torch.equal(y, m.decode(x[:, i:i + 1], b)), i
    assert torch.equal(a.length, b.length) and torch.equal(a.pool, b.pool) and torch.equal(a.table, b.table)


def test_prompts_after_replays():
    """Entries that a graph's replays stored count, for a prompt outside and for one that is replayed itself."""
    m = make_module()
    x = torch.randn(2, 40, 256, device="cuda").bfloat16()
    want = m.prefill(x, m.new_cache(2, 64, page_size=16))
    c = m.new_cache(2, 64, page_size=16)
    static, prompt = x[:, 5:6].clone(), x[:, 10:20].clone()
    m.prefill(x[:, :4], c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        static.copy_(x[:, 4:5])
        m.decode(static, c)
        one, ten = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(one, stream=side):
            m.decode(static, c)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(5, 10):
        static.copy_(x[:, i:i + 1])
        one.replay()
    got = [m.prefill(prompt, c)]
    assert c.length.tolist() == [20, 20] and c.bound == 20
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(ten, stream=side):
        y = m.prefill(prompt, c)
    torch.cuda.current_stream().wait_stream(side)
    for i in (20, 30):
        prompt.copy_(x[:, i:i + 10])
        ten.replay()
        got.append(y.clone())
    # both sides round to bf16 once per projection and output, as above
    for i, z in enumerate(got):
        assert (z.float() - want[:, 10 * i + 10:10 * i + 20].float()).abs().max() < 6e-2, i
    assert c.recount() == 40 and c.position.tolist() == [40, 40]


def test_an_append_of_other_shapes_takes_no_page():
    c = ra.RaPagedCache(2, 2, 64, 64, page_size=16)
    for shape in ((3, 20, 6 * 64), (2, 20, 6 * 128), (1, 20, 6 * 64)):
        with pytest.raises(ValueError, match="batch size"):
            c.append(torch.zeros(shape, device="cuda"), 2, norm="none")
    with pytest.raises(ValueError):
        c.append(torch.zeros(2, 20, 6 * 64, device="cuda"), 2, norm="none", count=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (c.uses == 0).all() and (c.table == -1).all() and c.bound == 0


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(2)
    sets = []
    for s in range(2):
        pool, table, n = filled(g, [600 - 7 * b for b in range(20)], 2, 16, 128, 40)
        q = torch.randn(20, 8, 128, generator=g).bfloat16().cuda()
        sets.append((q, pool, table, n))
    want = [ra.ra_attention_decode_paged(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[s].append(ra.ra_attention_decode_paged(*sets[s]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[s]) for s in range(2) for o in got[s])


def test_every_call_after_joined_streams_and_copies_in_a_graph():
    """The calls start early behind a kernel of the same stream; behind a copy, a set or an event of another stream, in
    a graph and outside, they wait for all of it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, H, D, page, N = 3, 2, 64, 16, 40
    k0, v0 = (torch.randn(B, H, N, D, generator=g, device="cuda") for _ in range(2))
    q0 = torch.randn(B, 4, D, generator=g, device="cuda")

    def state():
        return dict(k=torch.zeros_like(k0), v=torch.zeros_like(v0), q=torch.zeros_like(q0),
                    pool=torch.full((30, H, 2, page, 36), 255, dtype=torch.uint8, device="cuda"),
                    table=torch.full((B, 4), -1, dtype=torch.int32, device="cuda"), uses=torch.zeros(30, dtype=torch.int32, device="cuda"),
                    length=torch.zeros(B, dtype=torch.int32, device="cuda"), parent=torch.zeros(B, dtype=torch.int32, device="cuda"),
                    big=torch.zeros(1 << 24, device="cuda"))

    def work(s, stream, other):
        """Every call right behind something that is not one of the library's kernels."""
        out = []
        def join():                                # a slow kernel on another stream, then a copy and a set on this one
            other.wait_stream(stream)
            with torch.cuda.stream(other):
                s["big"].add_(1.0).mul_(1.0)
                s["k"].copy_(k0)
                s["v"].copy_(v0)
            stream.wait_stream(other)
        s["length"].zero_()
        join()
        granted = ra.ra_page_reserve(s["pool"], s["table"], s["length"], s["uses"], N)
        join()
        out += ra.ra_page_write(s["k"], s["v"], s["pool"], s["table"], s["length"], count=granted, held=True)
        s["length"].fill_(N)
        out += ra.ra_page_read(s["pool"], s["table"], s["length"], N, dtype=torch.float32)
        s["q"].copy_(q0)
        out.append(ra.ra_attention_decode_paged(s["q"], s["pool"], s["table"], s["length"]))
        s["parent"].copy_(torch.arange(B, device="cuda", dtype=torch.int32).flip(0))
        join()
        ra.ra_page_fork(s["table"], s["length"], s["uses"], s["parent"])
        join()
        small = torch.zeros(12, H, 2, page, 36, dtype=torch.uint8, device="cuda")
        out += ra.ra_page_compact(s["pool"], s["table"], s["uses"], small)
        out.append(ra.ra_attention_decode_paged(s["q"], small, out[-3], s["length"]))
        s["parent"].fill_(-1)
        ra.ra_page_fork(s["table"], s["length"], s["uses"], s["parent"])
        return out + [small, s["uses"].clone()]

    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = state(), state()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        want = work(a, main, other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        got = work(b, main, other)
    for _ in range(3):
        for t in got:
            t.zero_()
        b["k"].zero_()
        b["q"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    z = torch.matmul(q0.view(B, H, 2, D), want[0].transpose(-1, -2)) / 8.0
    u = ((z.amax(-1, keepdim=True) - z) / 16.0).clamp(max=1.0)
    p = ((1 - u) / (1 + u)) ** 8
    o = torch.matmul(p / p.sum(-1, keepdim=True), want[1]).view(B, 4, D)
    # fp32 on both sides, matmuls of torch possibly with fewer bits: far from what a missing wait would give
    assert (want[4] - o).abs().max() < 2e-2
