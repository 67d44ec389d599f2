"""GPU parity of ra_attention_decode and ra_cache_evict against the float64 oracle, and the serving path run
as a whole.

Tolerances of the decode.  Score error: delta = scale (D + 2) 2^-23 max_j sum_d |q_d k_jd| per row (as in
parity.py).  phi changes by at most delta relative to its row's maximum 1 (|d phi / d Delta| <= 1), and
forming it takes a difference, a sum, a reciprocal and four products, 2^-22 relative at most each
(approximate reciprocal), eight-fold by the power: 64 * 2^-23.  So every weight p_j is off by at most
(2 delta + 64 * 2^-23) (p_j + 1/s), s the row's sum of phi; summed over the row's values that is e_O =
(2 delta + 64 * 2^-23) (sum_j p_j |v_j| + sum over the support of |v_j| / s).  bf16 values add the
rounding of each weight, 2^-8 p_j |v_j|, and of the output, 2^-8 |O|."""
import numpy as np
import pytest
import torch

from oracle import ra_serving as S
import rational_softmax_attention_gb300 as ra

pytestmark = pytest.mark.gpu


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def inputs(B, Hq, Hkv, C, P, D, dtype, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, Hq, D, generator=g) * sigma).to(dtype)
    k = (torch.randn(B, Hkv, C, D, generator=g) * sigma).to(dtype)
    v = torch.randn(B, Hkv, C, D, generator=g).to(dtype)
    pk = (torch.randn(Hkv, P, D, generator=g) * sigma).to(dtype) if P else None
    pv = torch.randn(Hkv, P, D, generator=g).to(dtype) if P else None
    return q, k, v, pk, pv


def check_decode(q, k, v, length, pk, pv, scale=None, tracked=True, poison=True):
    """Runs the call with the cache's unused slots poisoned, checks o and the weights; returns o."""
    B, Hq, D = q.shape
    Hkv, C = k.shape[1:3]
    G = Hq // Hkv
    n = torch.as_tensor(length, dtype=torch.int32)
    kp, vp = k.clone(), v.clone()
    if poison:
        for b, m in enumerate(n.clamp(0, C).tolist()):
            kp[b, :, m:], vp[b, :, m:] = float("nan"), float("inf")
    weight = torch.full((B, Hkv, C), 0.25, device="cuda") if tracked else None
    cu = [None if t is None else t.cuda() for t in (pk, pv)]
    o = ra.ra_attention_decode(q.cuda(), kp.cuda(), vp.cuda(), n.cuda(), prefix_k=cu[0], prefix_v=cu[1], scale=scale,
                               weight=weight)
    torch.cuda.synchronize()
    assert o.dtype == q.dtype and o.shape == q.shape
    O, W, spread, sums = S.attention_decode(f64(q), f64(k), f64(v), n.tolist(), f64(pk), f64(pv), scale)
    sc = D ** -0.5 if not scale else scale
    delta = np.zeros((B, Hq))
    reach = np.zeros((B, Hq))
    for b in range(B):
        m = min(max(int(n[b]), 0), C)
        for h in range(Hq):
            keys, vals = f64(k[b, h // G, :m]), f64(v[b, h // G, :m])
            if pk is not None:
                keys, vals = np.concatenate([f64(pk[h // G]), keys]), np.concatenate([f64(pv[h // G]), vals])
            if len(keys):
                qa = np.abs(f64(q[b, h]))
                delta[b, h] = sc * (D + 2) * 2.0 ** -23 * (np.abs(keys) @ qa).max()
                z = keys @ f64(q[b, h]) * sc
                reach[b, h] = np.abs(vals[z.max() - z < 16.0 + 1e-3]).max() * np.count_nonzero(z.max() - z < 16.0 + 1e-3)
    e = 2 * delta + 64 * 2.0 ** -23
    inv = np.where(sums > 0, 1.0 / np.where(sums > 0, sums, 1.0), 0.0)
    half = torch.finfo(q.dtype).eps / 2
    bound = half * np.abs(O) + e[..., None] * (spread + (reach * inv)[..., None]) + 1e-30
    if q.dtype == torch.bfloat16:
        bound += half * spread
    err = np.abs(f64(o) - O)
    assert np.all(err <= bound), f"o beyond its bound by {np.max(err - bound):.3e}"
    if tracked:
        got = f64(weight) - 0.25
        wb = (e * inv).reshape(B, Hkv, G).sum(-1)[..., None] + e.reshape(B, Hkv, G).max(-1)[..., None] * W + 2.0 ** -24
        wb = wb + 2.0 ** -24 * (np.abs(W) + 0.25)
        assert np.all(np.abs(got - W) <= wb), f"weights beyond their bound by {np.max(np.abs(got - W) - wb):.3e}"
        for b, m in enumerate(n.clamp(0, C).tolist()):
            assert np.all(got[b, :, m:] == 0)
    return o


CASES = [  # B, Hq, Hkv, C, P, D, sigma, lengths
    (1, 1, 1, 1, 0, 64, 1.0, [1]),
    (1, 16, 16, 512, 0, 128, 1.0, [300]),
    (2, 4, 2, 40, 0, 64, 1.0, [0, 33]),                    # a sequence without any key
    (3, 6, 2, 129, 1, 128, 1.0, [0, 128, 129]),            # a prefix of one key
    (3, 8, 1, 300, 257, 64, 2.0, [300, 1, 31]),
    (2, 20, 1, 700, 0, 128, 1.0, [700, 513]),              # more query heads than a block of rows
    (5, 12, 4, 1003, 777, 64, 1.0, [1003, 0, 5, 512, 256]),
    (9, 16, 8, 65, 1300, 128, 3.0, [65, 64, 63, 33, 32, 31, 1, 0, 2]),
    (40, 4, 2, 48, 600, 64, 1.0, list(range(40))),         # rows of many sequences against the prefix
    (1, 5, 5, 4999, 0, 64, 3.0, [4990]),
    (2, 2, 1, 16, 2, 128, 1.0, [-3, 99]),                  # lengths outside the cache
    # many rows per shared key
    (33, 1, 1, 3, 1, 64, 1.0, [i % 4 for i in range(33)]),
    (70, 8, 2, 20, 129, 128, 1.0, [i % 21 for i in range(70)]),        # 280 rows: a second row pair of 24
    (100, 3, 1, 40, 2500, 128, 2.0, [i % 41 for i in range(100)]),     # three heads per key head, 300 rows
    (128, 2, 2, 9, 1024, 64, 1.0, [i % 10 for i in range(128)]),       # exactly one row tile
    (150, 4, 1, 5, 1000, 64, 3.0, [i % 6 for i in range(150)]),        # 600 rows
    (36, 8, 8, 700, 2900, 128, 3.0, [700 - i for i in range(36)]),
    (600, 2, 1, 5, 300, 64, 1.0, [i % 6 for i in range(600)]),         # more than 512 sequences
    (1, 1024, 1, 70, 40, 64, 1.0, [69]),                   # as many query heads per key head as there may be
    (8192, 1, 1, 3, 130, 64, 1.0, [i % 4 for i in range(8192)]),       # and as many sequences
    # the shared keys on the tensor cores (bf16, more than 3648 blocks of 16 rows by 16 keys)
    (33, 1, 1, 3, 20001, 64, 1.0, [i % 4 for i in range(33)]),
    (70, 8, 2, 20, 1700, 128, 1.0, [i % 21 for i in range(70)]),
    (100, 3, 1, 40, 3333, 128, 2.0, [i % 41 for i in range(100)]),
    (128, 2, 2, 9, 3712, 64, 1.0, [i % 10 for i in range(128)]),       # exactly one row tile
    (150, 4, 1, 5, 1600, 64, 3.0, [i % 6 for i in range(150)]),
    (600, 2, 1, 5, 800, 64, 1.0, [i % 6 for i in range(600)]),
    # short sequences in a large cache, one or more of them long
    (64, 8, 4, 6000, 0, 64, 1.0, [1 + i % 7 for i in range(64)]),
    (64, 8, 4, 3000, 5, 128, 1.0, [3000 if i == 9 else i % 5 for i in range(64)]),
    (3, 4, 2, 9000, 0, 64, 1.0, [2, 9000, 17]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode_matches_the_oracle(case, dtype):
    B, Hq, Hkv, C, P, D, sigma, lengths = case
    check_decode(*inputs(B, Hq, Hkv, C, P, D, dtype, seed=C + P, sigma=sigma)[:3], lengths,
                 *inputs(B, Hq, Hkv, C, P, D, dtype, seed=C + P, sigma=sigma)[3:])


@pytest.mark.parametrize("case", [(4, 16, 16, 700, 0, 128), (16, 16, 4, 700, 0, 64), (4, 64, 4, 500, 300, 128),
                                  (8, 48, 2, 300, 0, 64), (33, 4, 4, 40, 1500, 64), (32, 32, 8, 100, 1000, 128)], ids=str)
def test_decode_bf16_errors_are_the_outputs_own_rounding(case):
    """Up to 128 rows per shared key head the weights go into the products as two bf16 each (2^-15 lost), so what is
    off is the rounding of the output: uniform within half a step of each element, whose mean square
    follows from the exact outputs.  15% above its root leaves room for the sample (8192 elements or
    more: 1.3% for one standard deviation) and the scores' fp32 sums; weights of one bf16 would add as
    much again as the output's rounding, in all 41%."""
    B, Hq, Hkv, C, P, D = case
    q, k, v, pk, pv = inputs(B, Hq, Hkv, C, P, D, torch.bfloat16, seed=C + D)
    o = check_decode(q, k, v, [C - b for b in range(B)], pk, pv)
    O = S.attention_decode(f64(q), f64(k), f64(v), [C - b for b in range(B)], f64(pk), f64(pv))[0]
    half = 2.0 ** (np.floor(np.log2(np.abs(O))) - 8)
    assert np.sqrt(np.mean((f64(o) - O) ** 2)) <= 1.15 * np.sqrt(np.mean(half ** 2) / 3)


@pytest.mark.parametrize("D", [16, 32])
def test_decode_small_heads_fp32(D):
    q, k, v, pk, pv = inputs(3, 6, 3, 77, 50, D, torch.float32, seed=D)
    check_decode(q, k, v, [77, 10, 0], pk, pv, scale=0.3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_scores_beyond_the_support_skip_their_values(dtype):
    """Wide scores: most blocks have no key within 16 of the maximum, and one key alone decides some rows."""
    q, k, v, pk, pv = inputs(2, 4, 2, 2000, 600, 64, dtype, seed=21, sigma=1.0)
    q *= 8
    k[:, :, 1234] = q[:, ::2] * 2
    check_decode(q, k, v, [2000, 1500], pk, pv)
    o = check_decode(q, k, v, [1235, 1235], None, None)
    assert torch.allclose(o[:, ::2].float().cpu(), v[:, :, 1234].float(), atol=2e-2)


def test_decode_masked_neighbours_do_not_change_a_bit():
    q, k, v, pk, pv = inputs(3, 8, 2, 400, 300, 128, torch.bfloat16, seed=22)
    a = check_decode(q, k, v, [400, 7, 129], pk, pv, poison=True)
    b = check_decode(q, k, v, [400, 7, 129], pk, pv, poison=False, tracked=False)
    assert torch.equal(a, b)


def test_decode_is_the_attention_call():
    """One query row of ra_attention over the same keys, within both sides' bf16 rounding."""
    q, k, v, pk, pv = inputs(2, 3, 3, 500, 300, 128, torch.bfloat16, seed=23)
    o = ra.ra_attention_decode(q.cuda(), k.cuda(), v.cuda(), torch.full((2,), 500, dtype=torch.int32, device="cuda"),
                               prefix_k=pk.cuda(), prefix_v=pv.cuda())
    keys = torch.cat([pk.expand(2, -1, -1, -1), k], 2).cuda()
    vals = torch.cat([pv.expand(2, -1, -1, -1), v], 2).cuda()
    want = ra.ra_attention(q.cuda().unsqueeze(2), keys, vals)[:, :, 0]
    _, _, spread, _ = S.attention_decode(f64(q), f64(k), f64(v), [500, 500], f64(pk), f64(pv))
    bound = 2.0 ** -8 * (2 * np.abs(f64(want)) + spread * (1 + 2.0 ** -3)) + 1e-4 * spread
    assert np.all(np.abs(f64(o) - f64(want)) <= bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_repeats_streams_and_graphs_agree(dtype):
    """Bit-identical across calls, on a side stream, and replayed from two captured graphs in turn with other
    lengths in the same buffers."""
    q, k, v, pk, pv = (t.cuda() for t in inputs(4, 8, 4, 600, 500, 64, dtype, seed=24))
    n1, n2 = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([600, 3, 250, 0], [1, 600, 600, 77]))
    n = n1.clone()

    def call(w):
        return ra.ra_attention_decode(q, k, v, n, prefix_k=pk, prefix_v=pv, weight=w)
    ref = {}
    for name, x in (("1", n1), ("2", n2)):
        n.copy_(x)
        w = torch.zeros(4, 4, 600, device="cuda")
        ref[name] = call(w), w
        w2 = torch.zeros_like(w)
        assert torch.equal(call(w2), ref[name][0]) and torch.equal(w, w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w2 = torch.zeros_like(w)
        assert torch.equal(call(w2), ref["2"][0]) and torch.equal(w2, ref["2"][1])
    side.synchronize()
    graphs = []
    for _ in range(2):
        wg = torch.zeros_like(w)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            og = call(wg)
        graphs.append((g, og, wg))
    for name, x in (("1", n1), ("2", n2), ("1", n1)):
        n.copy_(x)
        for g, og, wg in graphs:
            wg.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, og, wg in graphs:
            assert torch.equal(og, ref[name][0]) and torch.equal(wg, ref[name][1])


def test_decode_calls_on_two_streams():
    """Calls that run at the same time, each in its own workspace, with and without the tensor cores' part."""
    sets = [tuple(t.cuda() for t in inputs(48, 8, 4, 300, 2600, 64, torch.bfloat16, seed=27)),
            tuple(t.cuda() for t in inputs(70, 4, 2, 200, 3400, 128, torch.bfloat16, seed=28)),
            tuple(t.cuda() for t in inputs(6, 4, 4, 900, 100, 64, torch.float32, seed=29))]
    lengths = [torch.arange(q.shape[0], dtype=torch.int32, device="cuda") * 4 % k.shape[2] for q, k, *_ in sets]

    def call(i):
        q, k, v, pk, pv = sets[i]
        return ra.ra_attention_decode(q, k, v, lengths[i], prefix_k=pk, prefix_v=pv)
    want = [call(i) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, call(i)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got) and ra.device_status() == "RA_OK"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_nan_stays_in_its_rows(dtype):
    q, k, v, _, _ = inputs(3, 4, 2, 200, 0, 64, dtype, seed=30)
    n = torch.tensor([200, 150, 0], dtype=torch.int32, device="cuda")
    want = ra.ra_attention_decode(q.cuda(), k.cuda(), v.cuda(), n)
    q[0, 1] = float("nan")              # a query
    k[1, 0, 17, 3] = float("nan")       # a key of two queries
    got = ra.ra_attention_decode(q.cuda(), k.cuda(), v.cuda(), n)
    bad = torch.zeros(3, 4, dtype=torch.bool)
    bad[0, 1] = bad[1, 0] = bad[1, 1] = True
    assert torch.isnan(got[bad.cuda()]).all() and torch.equal(got[~bad.cuda()], want[~bad.cuda()])


@pytest.mark.parametrize("bad,good", [(0, 8), (8, 0), (3, 11)])
def test_decode_nan_in_one_head_does_not_drop_anothers_values(bad, good):
    """Two heads that the same lanes hold, one NaN; the other alone has weight in a block of keys."""
    H, C, D = 16, 100, 64
    q, k = torch.zeros(1, H, D), torch.zeros(1, 1, C, D)
    q[:, :, 0] = 32.0
    q[0, good, 0], q[0, good, 1] = 0.0, 32.0
    k[0, 0, 3, 0] = k[0, 0, 85, 1] = 8.0        # scores of 32 against 0: key 3 for all heads, key 85 for `good`
    q[0, bad] = float("nan")
    v = torch.randn(1, 1, C, D, generator=torch.Generator().manual_seed(31)).bfloat16()
    o = ra.ra_attention_decode(q.bfloat16().cuda(), k.bfloat16().cuda(), v.cuda(),
                               torch.full((1,), C, dtype=torch.int32, device="cuda")).cpu()
    want = v[0, :, 3].expand(H, D).clone()
    want[good] = v[0, 0, 85]
    assert torch.isnan(o[0, bad]).all()
    keep = [h for h in range(H) if h != bad]
    assert torch.equal(o[0, keep], want[keep])


# own keys of up to 8 rows and of more, a short prefix, the tensor cores with one row tile and with several
@pytest.mark.parametrize("case", [(2, 4, 2, 50, 0, 64), (2, 16, 1, 50, 0, 128), (3, 4, 2, 20, 40, 64),
                                  (40, 2, 1, 20, 21000, 64), (70, 8, 2, 20, 1700, 128)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_infinite_values(case, dtype):
    """Every key has weight, those of the maxima exactly 1: an infinite value of any key makes its dimension
    infinite in every row that reads it, with its sign, and nothing else changes."""
    B, Hq, Hkv, C, P, D = case
    q, k, v, pk, pv = inputs(B, Hq, Hkv, C, P, D, dtype, seed=33, sigma=0.5)
    n = torch.full((B,), C, dtype=torch.int32, device="cuda")

    def call():
        how = {} if pk is None else dict(prefix_k=pk.cuda(), prefix_v=pv.cuda())
        return ra.ra_attention_decode(q.cuda(), k.cuda(), v.cuda(), n, **how)
    want = call()
    best = (k[0, 0].double() @ q[0, 0].double()).argmax()          # of the first row, among its own keys
    v[:, :, best, 5], v[:, :, 7, 6] = float("inf"), float("-inf")
    want[..., 5], want[..., 6] = float("inf"), float("-inf")
    if P:
        rest = (pk[0].double() @ q[0, 0].double()).argmax()
        pv[:, rest, 9] = float("inf")
        want[..., 9] = float("inf")
    assert torch.equal(call(), want)


def test_a_cache_beyond_32_bit_offsets():
    """More than 2^31 elements before the second sequence, and 2^31 scores: append, decode and evict
    find the entries at the far ends.  One key lies so far above the others that it decides alone."""
    C, D, Hq = (1 << 24) + 64, 128, 64
    k = torch.zeros(2, 1, C, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    qkv = torch.randn(2, 1, (Hq + 2) * D, device="cuda").bfloat16()
    qkv[:, :, :Hq * D] = 2.0
    qkv[:, :, Hq * D:Hq * D + D] = 2.0               # score 4 * 128 / sqrt(128) = 45 against 0
    n = torch.tensor([C - 1, 39], dtype=torch.int32, device="cuda")
    q = ra.ra_cache_append(qkv, k, v, n, Hq, 1, norm="none")
    n += 1
    new = qkv[:, 0, (Hq + 1) * D:]
    assert torch.equal(v[0, 0, C - 1], new[0]) and torch.equal(v[1, 0, 39], new[1])
    weight = torch.zeros(2, 1, C, device="cuda")
    o = ra.ra_attention_decode(q[:, :, 0].contiguous(), k, v, n, weight=weight)
    assert torch.equal(o, new.unsqueeze(1).expand_as(o))
    assert weight[0, 0, C - 1] == Hq and weight[1, 0, 39] == Hq and weight.sum() == 2 * Hq
    weight[0, 0, 7], weight[0, 0, C - 2], weight[1, 0, 5] = 3.0, 2.0, 1.0
    k[1, 0, 5] = 0.5
    ko, vo, wo, m, index = ra.ra_cache_evict(k, v, weight, n, 3, recent=1)
    assert index.tolist() == [[[7, C - 2, C - 1]], [[0, 5, 39]]] and m.tolist() == [3, 3]
    assert torch.equal(vo[:, 0, 2], new) and torch.equal(ko[1, 0, 1], k[1, 0, 5]) and wo[0, 0].tolist() == [3, 2, Hq]


def test_decode_shared_keys_beyond_the_support():
    """Row tiles whose every shared weight is 0 (a far larger own score), mixed with others."""
    q, k, v, pk, pv = inputs(64, 4, 2, 6, 4000, 128, torch.bfloat16, seed=25)
    k[:32, :, 2] = q[:32, ::2] * 8                # own scores of about 90 for half of the heads
    check_decode(q, k, v, [6] * 32 + [0] * 32, pk, pv)
    k[:, :, 2] = (q[:, ::2] + q[:, 1::2]) * 8     # and for all rows of all sequences
    o = check_decode(q, k, v, [6] * 64, pk, pv)
    assert torch.isfinite(o.float()).all()


def test_decode_wait_timeout_is_reported_and_the_context_survives():
    q, k, v, pk, pv = inputs(40, 4, 2, 16, 6000, 64, torch.bfloat16, seed=26)
    args = [t.cuda() for t in (q, k, v)] + [torch.full((40,), 16, dtype=torch.int32, device="cuda")]
    how = dict(prefix_k=pk.cuda(), prefix_v=pv.cuda())
    assert ra.device_status() == "RA_OK"
    ra.set_wait_limit_ns(2_000_000)
    ra.debug_force_timeout(True)
    try:
        ra.ra_attention_decode(*args, **how)
        torch.cuda.synchronize()
        status = ra.device_status()
    finally:
        ra.debug_force_timeout(False)
        ra.set_wait_limit_ns(0)
    assert status == "RA_ERR_TIMEOUT"
    check_decode(q, k, v, [16] * 40, pk, pv)
    assert ra.device_status() == "RA_OK"


def test_decode_refusals():
    q, k, v, pk, pv = (t.cuda() for t in inputs(2, 4, 2, 8, 4, 64, torch.bfloat16, seed=1))
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    bad = [(q, k, v.float(), n, {}), (q, k, v[:, :, :7], n, {}), (q, k, v, n.long(), {}), (q, k, v, n[:1], {}),
           (q[:, :3].contiguous(), k, v, n, {}), (q, k, v, n, dict(prefix_k=pk)),
           (q, k, v, n, dict(prefix_k=pk, prefix_v=pv[:, :3])), (q, k, v, n, dict(weight=torch.zeros(2, 2, 7, device="cuda"))),
           (q, k, v, n.cpu(), {}), (q.transpose(0, 1), k, v, n, {})]
    for a, b, c, m, how in bad:
        with pytest.raises(ValueError):
            ra.ra_attention_decode(a, b, c, m, **how)
    q, k, v, _, _ = (t if t is None else t.cuda() for t in inputs(1, 1, 1, 8, 0, 32, torch.bfloat16, seed=1))
    with pytest.raises(ra.RaError) as e:
        ra.ra_attention_decode(q, k, v, n[:1].contiguous())
    assert e.value.code == 2
    # an empty prefix is none
    q, k, v, _, _ = (t if t is None else t.cuda() for t in inputs(1, 2, 1, 8, 0, 64, torch.bfloat16, seed=1))
    e = torch.empty(1, 0, 64, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(ra.ra_attention_decode(q, k, v, n[:1].contiguous(), prefix_k=e, prefix_v=e),
                       ra.ra_attention_decode(q, k, v, n[:1].contiguous()))


# ---- eviction: choices and copies, so everything is exact ------------------------------------------
EVICT = [  # B, H, C, C_out, keep, recent, lengths
    (1, 1, 1, 1, 1, 0, [1]),
    (2, 3, 64, 40, 16, 4, [64, 10]),
    (3, 1, 1000, 300, 300, 0, [1000, 0, 301]),
    (2, 2, 5000, 2100, 2049, 2049, [5000, 2050]),
    (4, 2, 2500, 1024, 1024, 64, [2500, 1025, 1024, 1023]),
    (1, 2, 40000, 777, 777, 100, [39999]),
    (2, 1, 300, 300, 299, 1, [-5, 999]),
]


def evict_case(B, H, C, Co, keep, recent, lengths, D, dtype, weights, seed=0):
    g = torch.Generator().manual_seed(seed + C)
    k, v = (torch.randn(B, H, C, D, generator=g).to(dtype) for _ in range(2))
    w = {"spread": lambda: torch.rand(B, H, C, generator=g) ** 8,
         "ties": lambda: torch.randint(0, 4, (B, H, C), generator=g).float(),
         "equal": lambda: torch.full((B, H, C), 0.5),
         "signed": lambda: torch.randint(-2, 3, (B, H, C), generator=g).float()
         * torch.where(torch.rand(B, H, C, generator=g) < 0.5, -1.0, 1.0),
         "special": lambda: torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e-42, 2.0])[
             torch.randint(0, 7, (B, H, C), generator=g)]}[weights]()
    n = torch.tensor(lengths, dtype=torch.int32)
    out = tuple(torch.full(s, 9.0, dtype=t).cuda() for s, t in
                (((B, H, Co, D), dtype), ((B, H, Co, D), dtype), ((B, H, Co), torch.float32)))
    ko, vo, wo, no, index = ra.ra_cache_evict(k.cuda(), v.cuda(), w.cuda(), n.cuda(), keep, recent=recent, out=out)
    torch.cuda.synchronize()
    I, N = S.cache_evict(w.numpy(), lengths, keep, recent)
    assert np.array_equal(index.cpu().numpy(), I) and np.array_equal(no.cpu().numpy(), N)
    assert no.dtype == torch.int32 and index.dtype == torch.int32
    for b in range(B):
        m = int(N[b])
        for h in range(H):
            at = torch.as_tensor(I[b, h, :m])
            assert torch.equal(ko[b, h, :m].cpu(), k[b, h, at]) and torch.equal(vo[b, h, :m].cpu(), v[b, h, at])
            assert torch.equal(wo[b, h, :m].cpu().view(torch.int32), w[b, h, at].view(torch.int32))
    for t, full in zip(out, (9.0,) * 3):      # behind the new length: as they were
        for b in range(B):
            assert bool((t[b, :, int(N[b]):] == full).all())


@pytest.mark.parametrize("weights", ["spread", "ties", "equal", "signed", "special"])
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict_matches_the_oracle(case, weights):
    evict_case(*case, 64, torch.bfloat16, weights)


@pytest.mark.parametrize("D,dtype", [(16, torch.float32), (128, torch.float32), (24, torch.bfloat16), (128, torch.bfloat16)])
def test_evict_row_sizes(D, dtype):
    evict_case(2, 2, 1500, 600, 512, 33, [1500, 700], D, dtype, "spread")


def test_evict_stream_and_graph():
    k, v = (torch.randn(2, 2, 900, 64, device="cuda") for _ in range(2))
    w, n = torch.rand(2, 2, 900, device="cuda"), torch.tensor([900, 300], dtype=torch.int32, device="cuda")
    ref = ra.ra_cache_evict(k, v, w, n, 256, recent=16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ra.ra_cache_evict(k, v, w, n, 256, recent=16)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cap = ra.ra_cache_evict(k, v, w, n, 256, recent=16)
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, got, cap):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_evict_refusals():
    k = torch.zeros(1, 1, 8, 64, device="cuda")
    v, w, n = k.clone(), torch.zeros(1, 1, 8, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    out = (torch.zeros_like(k), torch.zeros_like(k), torch.zeros_like(w))
    for keep, how in ((0, {}), (4, dict(recent=5)), (4, dict(recent=-1)), (9, dict(out=out)),
                      (4, dict(out=(out[0], out[1].bfloat16(), out[2])))):
        with pytest.raises(ValueError):
            ra.ra_cache_evict(k, v, w, n, keep, **how)
    with pytest.raises(ra.RaError) as e:
        ra.ra_cache_evict(k, v, w, n, 4, out=(k, out[1], out[2]))
    assert e.value.code == 1
    with pytest.raises(ValueError):
        ra.ra_cache_evict(k, v, w.double(), n, 4)


# ---- the path as a whole ------------------------------------------------------------------------------
def module(dim=256, heads=2, dtype=torch.bfloat16, **how):
    torch.manual_seed(7)
    m = ra.RaAttention(dim, num_heads=heads, qk_norm=True, causal=True, **how).to(device="cuda", dtype=dtype)
    with torch.no_grad():
        for ln in (m.q_norm, m.k_norm):
            ln.weight.uniform_(0.5, 1.5)
            ln.bias.uniform_(-0.2, 0.2)
    return m


# bf16: q, k, v, O and y are rounded (2^-8 each) on both sides, of values up to about 4
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-4), (torch.bfloat16, 6e-2)])
@pytest.mark.parametrize("how", [dict(rope_sections=(64,)), dict(rope_sections=(16, 24, 24), rope_interleaved=True), {}],
                         ids=str)
def test_prefill_and_decode_are_the_forward(how, dtype, tol):
    """A prompt, then single tokens, against one causal forward of the whole sequence."""
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        m = module(dtype=dtype, **how)
        x = torch.randn(3, 45, 256, device="cuda").to(dtype)
        want = m(x).detach()
        cache = m.new_cache(3, 45)
        y = [m.prefill(x[:, :37], cache)]
        for i in range(37, 45):
            y.append(m.decode(x[:, i:i + 1], cache))
        assert cache.length.tolist() == [45] * 3 and cache.position.tolist() == [45] * 3
        assert (torch.cat(y, 1).float() - want.float()).abs().max() <= tol
        with pytest.raises(ValueError, match="no room"):
            m.decode(x[:, :1], cache)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = old


def test_a_shared_prefix_is_the_long_prompt():
    m = module(rope_sections=(64,))
    doc, x = torch.randn(1, 150, 256, device="cuda").bfloat16(), torch.randn(3, 20, 256, device="cuda").bfloat16()
    want = m(torch.cat([doc.expand(3, -1, -1), x], 1))[:, 150:].detach()
    one = m.new_cache(1, 150)
    m.prefill(doc, one)
    cache = m.new_cache(3, 30, prefix=(one.k[0], one.v[0]))
    y = [m.prefill(x[:, :12], cache)]
    y += [m.decode(x[:, i:i + 1], cache) for i in range(12, 20)]
    assert cache.position.tolist() == [170] * 3 and cache.length.tolist() == [20] * 3
    assert (torch.cat(y, 1).float() - want.float()).abs().max() <= 6e-2


def test_ragged_prompts_and_eviction_in_a_generation():
    """A padded batch of prompts, tokens with tracked weights, eviction, more tokens: against the operators'
    oracles fed with the cache's own contents."""
    m = module(rope_sections=(32,))
    x = torch.randn(2, 40, 256, device="cuda").bfloat16()
    count = torch.tensor([30, 17], dtype=torch.int32, device="cuda")
    cache = m.new_cache(2, 48, track_weight=True)
    m.prefill(x, cache, count=count)
    assert cache.length.tolist() == [30, 17] and cache.position.tolist() == [30, 17]
    for i in range(6):
        m.decode(x[:, i:i + 1], cache)
    total = cache.weight.sum(-1)
    assert torch.allclose(total, torch.full_like(total, 6.0), atol=1e-4)      # six queries, one head each
    k, v, w, n = (t.clone() for t in (cache.k, cache.v, cache.weight, cache.length))
    assert n.tolist() == [36, 23]
    before = cache.evict(16, recent=4)
    assert before[0].shape == cache.k.shape
    I, N = S.cache_evict(w.cpu().numpy(), n.tolist(), 16, 4)
    assert cache.length.tolist() == N.tolist() and cache.position.tolist() == [36, 23] and cache.bound == 16
    for b in range(2):
        for h in range(2):
            at = torch.as_tensor(I[b, h, :int(N[b])]).cuda()
            assert torch.equal(cache.k[b, h, :len(at)], k[b, h, at]) and torch.equal(cache.v[b, h, :len(at)], v[b, h, at])
    assert not cache.weight[:, :, 16:].any()
    y = m.decode(x[:, :1], cache)
    assert cache.length.tolist() == [17, 17] and torch.isfinite(y.float()).all()
    again = cache.evict(16, recent=4, spare=before)
    assert again[0].shape == cache.k.shape and cache.length.tolist() == [16, 16]


def test_ragged_appends_until_the_cache_is_full():
    """Padded appends go on while every sequence has room, whatever the padding adds up to; their entries stand
    one after the other."""
    cache = ra.RaCache(2, 1, 16, 64, dtype=torch.float32)
    want = [[], []]
    for i, count in enumerate(([4, 1], [0, 3], [4, 4], [4, 0], [4, 4], [0, 4])):
        qkv = torch.randn(2, 4, 3 * 64, device="cuda")
        cache.append(qkv, 1, count=torch.tensor(count, dtype=torch.int32, device="cuda"), norm="none")
        for b in range(2):
            want[b].append(qkv[b, :count[b], 64:128])
    assert cache.length.tolist() == [16, 16]
    for b in range(2):
        assert torch.equal(cache.k[b, 0], torch.cat(want[b]))
    with pytest.raises(ValueError, match="no room"):
        cache.append(qkv, 1, count=torch.tensor([1, 0], dtype=torch.int32, device="cuda"), norm="none")


def test_decode_step_in_a_graph():
    """The module's single-token step captured once and replayed: lengths and positions advance on the device."""
    m = module(rope_sections=(64,))
    x = torch.randn(2, 30, 256, device="cuda").bfloat16()
    eager, captured = m.new_cache(2, 30, track_weight=True), m.new_cache(2, 30, track_weight=True)
    for c in (eager, captured):
        m.prefill(x[:, :10], c)
    want = [m.decode(x[:, i:i + 1], eager) for i in range(10, 20)]
    token = x[:, 10:11].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [m.decode(token, captured).clone()]
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = m.decode(token, captured)
    for i in range(11, 20):
        token.copy_(x[:, i:i + 1])
        g.replay()
        got.append(y.clone())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert torch.equal(eager.weight, captured.weight) and captured.length.tolist() == [20, 20]


@pytest.mark.parametrize("how", [dict(rope_sections=(64,)), {}], ids=str)
def test_module_under_autocast(how):
    """fp32 parameters under bf16 autocast: the forward, its gradients, a prompt and single tokens are those of the bf16
    module (parameters that bf16 holds: the same products, and norms of the same rows, whose results may
    differ by a rounding, as in the runs above)."""
    m = module(dtype=torch.bfloat16, **how)
    wide = module(dtype=torch.float32, **how)
    wide.load_state_dict({n: t.float() for n, t in m.state_dict().items()})
    x = torch.randn(2, 24, 256, device="cuda").bfloat16()
    want, got = m(x), None
    want.float().sum().backward()
    with torch.autocast("cuda", dtype=torch.bfloat16):
        got = wide(x.float())
        assert got.dtype == torch.bfloat16 and (got.float() - want.float()).abs().max() <= 6e-2
        cache = wide.new_cache(2, 24, dtype=torch.bfloat16)
        y = [wide.prefill(x[:, :20].float(), cache)] + [wide.decode(x[:, i:i + 1].float(), cache) for i in range(20, 24)]
        assert (torch.cat(y, 1).float() - want.float()).abs().max() <= 6e-2
        with pytest.raises(ValueError, match="dtype"):
            wide.prefill(x.float(), wide.new_cache(2, 24))
    got.float().sum().backward()
    for (n, a), (_, b) in zip(m.named_parameters(), wide.named_parameters()):
        assert b.grad.dtype == torch.float32 and torch.isfinite(b.grad).all(), n


def test_module_gradients_with_rotation():
    """fp32 gradients of a rotated, normalised module against differences of its own forward in 64-bit sums."""
    m = module(dim=64, heads=2, dtype=torch.float32, rope_sections=(8, 8))
    x = torch.randn(2, 9, 64, device="cuda").requires_grad_(True)
    dy = torch.randn(2, 9, 64, device="cuda")
    pos = torch.stack([torch.arange(9), torch.arange(9) // 3]).view(2, 1, 9).cuda()
    m(x, positions=pos).backward(dy)
    e = 1e-2
    for t in (x, m.q_norm.weight, m.k_norm.weight, m.k_norm.bias, m.qkv.weight):
        u = torch.randn_like(t)
        u /= u.norm()
        with torch.no_grad():
            f = []
            for s in (e, -e):
                t += s * u
                f.append((m(x, positions=pos).double() * dy.double()).sum().item())
                t -= s * u
        want = (t.grad.double() * u.double()).sum().item()
        # central difference: e^2 / 6 times the third derivative, and fp32 noise of 1e-5 over 2 e
        assert abs((f[0] - f[1]) / (2 * e) - want) <= 5e-3 * (1 + abs(want)), (t.shape, f, want)
