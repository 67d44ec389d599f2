"""GPU parity of ra_qk_norm_rope (forward, backward, cache append) against the float64 oracle on the
same rounded inputs.

Tolerances.  Output rounding: half a step, finfo.eps / 2 of the value (bf16 2^-8, fp32 2^-24).
Arithmetic: fp32.  A normalised value passes about 20 roundings (two sums over D of at most 4 + 5 levels,
mean, square root, products) of 2^-24, the rotation two products, a sum, and a cosine and sine within
2 ulp of an angle within 2^-22 turns of the exact one: together below 64 * 2^-24 of the largest
value in the row.  A row gradient passes the same twice: 128 * 2^-24, of the row's largest possible
value r * max|g w| * 3.  A parameter gradient over n rows: (16 + log2 n) * 4 roundings of 2^-24 of the
sum of the terms' absolute values at most."""
import numpy as np
import pytest
import torch

from oracle import ra_serving as S
import rational_softmax_attention_gb300 as ra

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(B, N, Hq, Hkv, D, dtype, norm, bias, sections, interleaved, seed, start=0, shared_pos=False):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(B, N, (Hq + 2 * Hkv) * D, generator=g) * 1.5 + 0.2).to(dtype)
    params = {"q_weight": None, "q_bias": None, "k_weight": None, "k_bias": None}
    if norm != "none":
        params["q_weight"], params["k_weight"] = ((torch.rand(D, generator=g) + 0.5).to(dtype) for _ in range(2))
    if bias:
        params["q_bias"], params["k_bias"] = ((torch.randn(D, generator=g) * 0.2).to(dtype) for _ in range(2))
    how = {"norm": norm, "interleaved": interleaved, "sections": sections, "frequencies": None, "positions": None}
    if sections:
        how["frequencies"] = ra.ra_rope_frequencies(sections, device="cpu")
        shape = (1, 1, N) if shared_pos else (len(sections), B, N)
        how["positions"] = (torch.randint(0, 5000, shape, generator=g) + start).to(torch.int32)
    return qkv, params, how


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


def oracle_how(params, how):
    return dict(norm=how["norm"], params=tuple(f64(params[n]) for n in ("q_weight", "q_bias", "k_weight", "k_bias")),
                frequencies=f64(how["frequencies"]), sections=how["sections"],
                positions=None if how["positions"] is None else how["positions"].numpy(),
                interleaved=how["interleaved"])


def check_rows(got, want, dtype, what):
    assert got.dtype == dtype
    got = f64(got)
    bound = half_step(dtype) * np.abs(want) + 64 * U32 * np.abs(want).max(-1, keepdims=True)
    worst = np.max(np.abs(got - want) - bound)
    assert worst <= 0, f"{what}: beyond the bound by {worst:.3e}"


CASES = [  # B, N, Hq, Hkv, D, norm, bias, sections, interleaved
    (2, 128, 12, 12, 64, "layer", True, (32,), False),
    (1, 1, 1, 1, 64, "rms", False, (8, 24), False),
    (3, 37, 6, 2, 128, "rms", False, (16, 24, 24), True),
    (2, 19, 5, 1, 128, "layer", False, (10, 3, 2, 1), False),
    (1, 67, 3, 3, 16, "layer", True, (8,), False),
    (2, 33, 4, 2, 32, "none", False, (5, 2), True),
    (2, 50, 7, 1, 64, "layer", True, None, False),
    (1, 700, 16, 8, 128, "none", False, (64,), False),
    (4, 1500, 2, 1, 16, "rms", False, (1, 1), True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward_match_the_oracle(case, dtype):
    B, N, Hq, Hkv, D, norm, bias, sections, inter = case
    qkv, params, how = make(B, N, Hq, Hkv, D, dtype, norm, bias, sections, inter, seed=N + D)
    q, k, v = ra.ra_qk_norm_rope(qkv.cuda(), Hq, Hkv, **cuda(params), **cuda(how))
    torch.cuda.synchronize()
    oh = oracle_how(params, how)
    Q, K, V = S.qk_norm_rope(f64(qkv), Hq, Hkv, **oh)
    check_rows(q, Q, dtype, "q")
    check_rows(k, K, dtype, "k")
    assert np.array_equal(f64(v), V)

    g = torch.Generator().manual_seed(5)
    d = [torch.randn(B, h, N, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv)]
    got = ra.ra_qk_norm_rope_backward(qkv.cuda(), *(t.cuda() for t in d), Hq, Hkv, **cuda(params), **cuda(how))
    torch.cuda.synchronize()
    DX, DP = S.qk_norm_rope_bwd(f64(qkv), *(f64(t) for t in d), Hq, Hkv, **oh)
    dx = f64(got[0]).reshape(B, N, -1, D)
    DX = DX.reshape(B, N, -1, D)
    if norm == "none":
        scale = np.ones(DX.shape[:-1] + (1,))
    else:
        _, r = S._norm(f64(qkv).reshape(B, N, -1, D)[:, :, :Hq + Hkv], norm, 1e-5)
        scale = np.concatenate([r, np.ones((B, N, Hkv, 1))], 2) * 1.5
    dmax = np.concatenate([np.abs(f64(t)).max(-1, keepdims=True).transpose(0, 2, 1, 3) for t in d], 2) * np.sqrt(2)
    assert np.all(np.abs(dx - DX) <= half_step(dtype) * np.abs(DX) + 128 * U32 * 3 * scale * dmax)
    assert np.array_equal(dx[:, :, Hq + Hkv:], DX[:, :, Hq + Hkv:])
    names = ("q_weight", "q_bias", "k_weight", "k_bias")
    for i, name in enumerate(names):
        if params[name] is None:
            assert got[1 + i] is None
            continue
        rows = B * N * (Hq if i < 2 else Hkv)
        # |g| <= sqrt(2) max|d|, |xhat| <= sqrt(D): the terms' sum, by its mean size
        size = rows * 1.5 * np.abs(f64(d[i // 2])).mean() * (2.0 if i % 2 == 0 else 1.0)
        assert got[1 + i].dtype == torch.float32
        err = np.abs(f64(got[1 + i]) - DP[i]).max()
        assert err <= (16 + np.log2(rows)) * 4 * U32 * size, (name, err)


# Long batches, whose CTAs take three tiles of tokens and more, so that both halves of the table of cosines and sines
# are written again, and whose last tile is ragged: forward tiles of 32 (bf16, one head), 16 and 8 tokens.
@pytest.mark.parametrize("case,dtype", [((1, 30011, 1, 1, 128, "layer", True, (64,), False), torch.bfloat16),
                                        ((1, 9999, 5, 5, 32, "rms", False, (9, 5), True), torch.bfloat16),
                                        ((1, 5003, 4, 2, 128, "layer", True, (32, 16), False), torch.float32),
                                        ((3, 9001, 8, 1, 64, "none", False, (16,), False), torch.bfloat16)], ids=str)
def test_many_tiles_of_tokens_match_the_oracle(case, dtype):
    test_forward_and_backward_match_the_oracle(case, dtype)


@pytest.mark.parametrize("start", [(1 << 24) + 1, (1 << 31) - 6000, -(1 << 31)])
def test_far_positions_keep_their_angles(start):
    """Angles of positions that fp32 cannot hold, against 64 bits; positions shared by axes and batch."""
    qkv, params, how = make(2, 40, 2, 1, 64, torch.float32, "none", False, (16, 16), False, 3, start, True)
    q, k, _ = ra.ra_qk_norm_rope(qkv.cuda(), 2, 1, **cuda(params), **cuda(how))
    Q, K, _ = S.qk_norm_rope(f64(qkv), 2, 1, **oracle_how(params, how))
    # the frequency's two floats hold 48 bits: at 2^31 / (2 pi) turns 2^-49 of that more, 6e-7 turns
    more = 2 * np.pi * 2 ** 31 / (2 * np.pi) * 2.0 ** -48 * 2
    for got, want in ((q, Q), (k, K)):
        bound = (64 * U32 + more) * np.abs(want).max(-1, keepdims=True) * np.sqrt(2)
        assert np.all(np.abs(f64(got) - want) <= bound)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 24) + 1, (1 << 31) - 6000, -(1 << 31)])
def test_every_position_keeps_the_accuracy_of_a_near_one(start, inter):
    """The same bound at all int32 positions.  An angle within an eighth of a turn of a quarter: rounded once, pi / 4 *
    2^-24; cosine and sine within 2 ulp, 2 * 2^-24; two products and a sum, 2 * 2^-24: 5 * 2^-24 of |x0| + |x1|, which is
    10 of the row's largest.  The oracle's own angle is a rounded product, 2^-53 of it."""
    qkv, params, how = make(2, 300, 2, 1, 64, torch.float32, "none", False, (24, 8), inter, 19, start)
    how["frequencies"][24] = 1.0
    how["frequencies"][25] = -7.5              # more than a turn per position, and backwards
    q, k, _ = ra.ra_qk_norm_rope(qkv.cuda(), 2, 1, **cuda(params), **cuda(how))
    Q, K, _ = S.qk_norm_rope(f64(qkv), 2, 1, **oracle_how(params, how))
    angle = 7.5 * (abs(start) + 5000)
    for got, want in ((q, Q), (k, K)):
        most = np.abs(want).max(-1, keepdims=True) * np.sqrt(2)
        assert np.all(np.abs(f64(got) - want) <= (10 * U32 + 2.0 ** -53 * angle) * most)


def test_strided_projection_and_position_forms():
    """qkv as a slice of a wider row, misaligned slices, [N] and [B, N] and int64 positions: the same results."""
    B, N, Hq, Hkv, D = 2, 21, 3, 1, 64
    qkv, params, how = make(B, N, Hq, Hkv, D, torch.bfloat16, "layer", True, (32,), False, 8, 0, True)
    params, how = cuda(params), cuda(how)
    ref = ra.ra_qk_norm_rope(qkv.cuda(), Hq, Hkv, **params, **how)
    wide = torch.full((B, N + 3, qkv.shape[-1] + 72), float("nan"), dtype=qkv.dtype, device="cuda")
    for off in (8, 3):
        part = wide[:, 2:2 + N, off:off + qkv.shape[-1]]
        part.copy_(qkv)
        for a, b in zip(ref, ra.ra_qk_norm_rope(part, Hq, Hkv, **params, **how)):
            assert torch.equal(a, b)
    p = how.pop("positions")
    for form in (p.view(N), p.view(1, N).expand(B, N), p.view(N).long(), p.expand(1, B, N)):
        for a, b in zip(ref, ra.ra_qk_norm_rope(qkv.cuda(), Hq, Hkv, **params, **how, positions=form)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("N,count", [(1, None), (5, None), (6, [6, 0, 3])])
def test_append_writes_its_slots_and_nothing_else(N, count):
    B, Hq, Hkv, D, C = 3, 4, 2, 128, 24
    qkv, params, how = make(B, N, Hq, Hkv, D, torch.bfloat16, "rms", False, (64,), False, 11)
    params, how = cuda(params), cuda(how)
    q, k, v = ra.ra_qk_norm_rope(qkv.cuda(), Hq, Hkv, **params, **how)
    ck, cv = (torch.full((B, Hkv, C, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    length = torch.tensor([0, C - 2, 9], dtype=torch.int32, device="cuda")    # the second has room for two
    n = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
    got = ra.ra_cache_append(qkv.cuda(), ck, cv, length, Hq, Hkv, count=n, **params, **how)
    assert torch.equal(got, q) and length.tolist() == [0, C - 2, 9]
    wk, wv = torch.full_like(ck, 7.0), torch.full_like(cv, 7.0)
    for b, s in enumerate(length.tolist()):
        m = min(N if count is None else count[b], C - s)
        wk[b, :, s:s + m], wv[b, :, s:s + m] = k[b, :, :m], v[b, :, :m]
    assert torch.equal(ck, wk) and torch.equal(cv, wv)


def test_append_ignores_slots_outside_the_cache():
    qkv, params, how = make(3, 2, 1, 1, 64, torch.float32, "none", False, None, False, 12)
    ck, cv = torch.zeros(3, 1, 4, 64, device="cuda"), torch.zeros(3, 1, 4, 64, device="cuda")
    length = torch.tensor([-1, 4, (1 << 31) - 1], dtype=torch.int32, device="cuda")
    ra.ra_cache_append(qkv.cuda(), ck, cv, length, 1, 1, norm="none")
    assert torch.equal(ck[0, 0, 0], qkv[0, 1, 64:128].cuda()) and not ck[0, 0, 1:].any() and not ck[1:].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_autograd(dtype):
    """The autograd function gives the explicit backward's gradients, for the inputs that ask."""
    B, N, Hq, Hkv, D = 2, 30, 4, 2, 64
    qkv, params, how = make(B, N, Hq, Hkv, D, dtype, "layer", True, (16, 16), True, 13)
    params, how, qkv = cuda(params), cuda(how), qkv.cuda()
    d = [torch.randn(B, N, h, D, device="cuda").to(dtype).transpose(1, 2) for h in (Hq, Hkv, Hkv)]   # strided
    want = ra.ra_qk_norm_rope_backward(qkv, *(t.contiguous() for t in d), Hq, Hkv, **params, **how)
    x = qkv.clone().requires_grad_(True)
    p = {n: t.clone().requires_grad_(True) for n, t in params.items()}
    out = ra.ra_qk_norm_rope(x, Hq, Hkv, **p, **how)
    torch.autograd.backward(out, d)
    assert torch.equal(x.grad, want[0])
    for (n, t), w in zip(p.items(), want[1:]):
        assert t.grad.dtype == dtype and torch.equal(t.grad, w.to(dtype)), n
    y = qkv.clone().requires_grad_(True)
    q, _, _ = ra.ra_qk_norm_rope(y, Hq, Hkv, **params, **how)
    q.sum().backward()                                   # k and v take no part
    assert not y.grad.view(B, N, -1, D)[:, :, Hq:].any()


def test_bit_identical_on_streams_and_in_a_graph():
    B, N, Hq, Hkv, D = 2, 900, 4, 4, 128
    qkv, params, how = make(B, N, Hq, Hkv, D, torch.bfloat16, "layer", True, (64,), False, 14)
    params, how, x = cuda(params), cuda(how), qkv.cuda()
    d = [torch.randn(B, h, N, D, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv)]

    def both():
        return (*ra.ra_qk_norm_rope(x, Hq, Hkv, **params, **how),
                *ra.ra_qk_norm_rope_backward(x, *d, Hq, Hkv, **params, **how))
    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cap = both()
    for _ in range(2):
        for t in cap:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, got, cap):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_autograd_takes_any_view_once_and_in_a_graph():
    """Gradients that start at an odd address, a second derivative (refused), and a backward pass captured with its
    forward (of a leaf without a live eager graph: torch ties a leaf's accumulation to the stream of
    its first graph, and a capture cannot wait for another stream, whatever the operators)."""
    B, N, Hq, Hkv, D = 2, 50, 2, 1, 64
    qkv, params, how = make(B, N, Hq, Hkv, D, torch.bfloat16, "layer", True, (32,), False, 15)
    params, how, x = cuda(params), cuda(how), qkv.cuda()
    d = [torch.randn(B, h, N, D, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv)]
    want = ra.ra_qk_norm_rope_backward(x, *d, Hq, Hkv, **params, **how)[0]
    odd = [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view_as(t).copy_(t) for t in d]
    y = x.clone().requires_grad_(True)
    out = ra.ra_qk_norm_rope(y, Hq, Hkv, **params, **how)
    assert torch.equal(torch.autograd.grad(out, y, odd, retain_graph=True)[0], want)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g, = torch.autograd.grad(out, y, [t.requires_grad_(True) for t in d], create_graph=True)
        g.float().sum().backward()
    d = [t.detach() for t in d]
    y = x.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(ra.ra_qk_norm_rope(y, Hq, Hkv, **params, **how), y, d)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got, = torch.autograd.grad(ra.ra_qk_norm_rope(y, Hq, Hkv, **params, **how), y, d)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite(value, norm, dtype):
    """A NaN makes its whole row NaN, and an infinity what the definition gives for it (NaN where it stands and in its
    partner; zeros, or with a mean NaN, elsewhere); the other rows do not change a bit.  The weights' gradients
    are NaN in every column that the definition gives as NaN, and the others' rows of dqkv stay."""
    B, N, Hq, Hkv, D = 2, 37, 3, 2, 64
    qkv, params, how = make(B, N, Hq, Hkv, D, dtype, norm, False, (24,), False, 16)
    d = [torch.randn(B, h, N, D, generator=torch.Generator().manual_seed(6)).to(dtype).cuda() for h in (Hq, Hkv, Hkv)]

    def both():
        args = cuda(params), cuda(how)
        return ra.ra_qk_norm_rope(qkv.cuda(), Hq, Hkv, **args[0], **args[1]), \
            ra.ra_qk_norm_rope_backward(qkv.cuda(), *d, Hq, Hkv, **args[0], **args[1])
    clean, clean_b = both()
    rows = qkv.view(B, N, Hq + 2 * Hkv, D)
    rows[1, 5, 2, 11] = value              # query head 2 of a token
    rows[0, 36, Hq, 63] = value            # key head 0 of another, in a dimension that is not turned
    got, got_b = both()
    oh = oracle_how(params, how)
    with np.errstate(all="ignore"):
        want = S.qk_norm_rope(f64(qkv), Hq, Hkv, **oh)
        DX, DP = S.qk_norm_rope_bwd(f64(qkv), *(f64(t) for t in d), Hq, Hkv, **oh)
    for g, c, w, at in ((got[0], clean[0], want[0], (1, 2, 5)), (got[1], clean[1], want[1], (0, 0, 36))):
        row = f64(g)[at]
        assert np.array_equal(np.isnan(row), np.isnan(w[at])) and np.isnan(row).any()
        assert np.array_equal(row[~np.isnan(row)], np.zeros(np.count_nonzero(~np.isnan(row))))
        if value != value:
            assert np.isnan(row).all()
        g[at] = c[at]
        assert torch.equal(g, c)
    assert torch.equal(got[2], clean[2])
    dx, c = (t.view(B, N, -1, D).clone() for t in (got_b[0], clean_b[0]))
    for at in ((1, 5, 2), (0, 36, Hq)):
        assert np.array_equal(np.isnan(f64(dx)[at]), np.isnan(DX.reshape(B, N, -1, D)[at]))
        dx[at] = c[at]
    assert torch.equal(dx, c)
    for i in (0, 2):                       # the weights; without biases there are no others
        assert np.array_equal(np.isnan(f64(got_b[1 + i])), np.isnan(DP[i])) and np.isnan(DP[i]).any()


def _fill_shared_memory_with_nan():
    """Leaves NaN in the SMs' shared memory: a decode whose keys are all NaN stages them there on every SM."""
    q = torch.full((64, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    k = torch.full((64, 8, 600, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ra.ra_attention_decode(q, k, k, torch.full((64,), 600, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype,N", [(torch.bfloat16, 333), (torch.bfloat16, 1217), (torch.float32, 333)])
def test_parameter_gradients_of_a_ragged_last_tile(dtype, N):
    """The last tile of tokens has places without a token (one head of 128: tiles of 4 and more), whose sines and
    cosines nobody forms: whatever shared memory held before, they add nothing to the weights' gradients."""
    qkv, params, how = make(1, N, 1, 1, 128, dtype, "rms", False, (64,), False, 17)
    params, how, x = cuda(params), cuda(how), qkv.cuda()
    d = [torch.randn(1, 1, N, 128, device="cuda").to(dtype) for _ in range(3)]
    oh = oracle_how({n: None if t is None else t.cpu() for n, t in params.items()},
                    dict(how, positions=how["positions"].cpu()))
    _, DP = S.qk_norm_rope_bwd(f64(qkv), *(f64(t) for t in d), 1, 1, **oh)
    for _ in range(3):
        _fill_shared_memory_with_nan()
        got = ra.ra_qk_norm_rope_backward(x, *d, 1, 1, **params, **how)
        for i in (0, 2):
            size = N * 1.5 * d[i // 2].abs().float().mean().item() * 2.0
            assert np.abs(f64(got[1 + i]) - DP[i]).max() <= (16 + np.log2(N)) * 4 * U32 * size


def test_parameter_gradients_are_added_in_short_chains():
    """The biases' gradients, sums of exact terms of unit variance over 80000 rows.  Rounding a sum S is off by 0.42 *
    2^-24 |S| in the mean square (uniform within half a step, over mantissas); so adding k equal parts of a
    sum one after the other costs 0.42 * 2^-24 sqrt(k / 2) of it, and by halves 0.42 * 2^-24 sqrt(log2 k).  A lane
    adds about 5.4 rows, a CTA 8 sums one after the other and 16 by halves, the whole 2 and 64 by halves:
    0.42 * sqrt(2.7 + 4 + 4 + 1 + 6) = 1.8 of 2^-24; with the CTA's 128 one after the other it would be 3.6.  256
    samples: 4.4% for one standard deviation; a third more is allowed."""
    N, H, D, total = 20000, 4, 16, []
    w = torch.ones(D, device="cuda")
    for seed in range(8):
        g = torch.Generator(device="cuda").manual_seed(seed)
        qkv = torch.randn(1, N, 3 * H * D, device="cuda", generator=g)
        d = [torch.randn(1, H, N, D, device="cuda", generator=g) for _ in range(3)]
        got = ra.ra_qk_norm_rope_backward(qkv, *d, H, H, norm="layer", q_weight=w, q_bias=w, k_weight=w, k_bias=w)
        total += [got[2].double() - d[0].double().sum((0, 1, 2)), got[4].double() - d[1].double().sum((0, 1, 2))]
    rms = torch.cat(total).square().mean().sqrt().item() / (N * H) ** 0.5
    assert rms <= 1.8 * 1.33 * U32, rms / U32


def test_a_tangent_is_refused_with_and_without_an_input_that_asks_for_a_gradient():
    from torch.autograd import forward_ad
    x, w = torch.randn(1, 2, 3 * 64, device="cuda"), torch.ones(64, device="cuda")
    for weight in (w, w.clone().requires_grad_(True)):
        with forward_ad.dual_level(), pytest.raises(NotImplementedError):   # the second: torch's own refusal
            ra.ra_qk_norm_rope(forward_ad.make_dual(x, torch.ones_like(x)), 1, 1, norm="rms", q_weight=weight, k_weight=w)


def test_refusals():
    x = torch.zeros(1, 2, 3 * 64, device="cuda")
    w, f = torch.ones(64, device="cuda"), ra.ra_rope_frequencies((32,))
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [dict(norm="batch"), dict(norm="layer"), dict(norm="rms", q_weight=w, k_weight=w, q_bias=w),
           dict(norm="none", q_weight=w), dict(norm="none", sections=(32,)),
           dict(norm="none", sections=(32,), frequencies=f.float(), positions=pos),
           dict(norm="none", sections=(33,), frequencies=f, positions=pos),
           dict(norm="none", sections=(32,), frequencies=f, positions=pos.cpu()),
           dict(norm="none", sections=(32,), frequencies=f, positions=pos.float()),
           dict(norm="none", sections=(32,), frequencies=f, positions=pos[:1]),
           dict(norm="none", sections=(32,), frequencies=f, positions=pos.view(1, 1, 2).expand(3, 1, 2)),
           dict(norm="none", frequencies=f), dict(norm="layer", q_weight=w.bfloat16(), k_weight=w.bfloat16())]
    for how in bad:
        with pytest.raises(ValueError):
            ra.ra_qk_norm_rope(x, 1, 1, **how)
    with pytest.raises(ra.RaError) as e:
        ra.ra_qk_norm_rope(x, 1, 1, norm="none", sections=(4,), frequencies=f[:4].contiguous(), positions=pos)
    assert e.value.code == 2
    with pytest.raises(TypeError):
        ra.ra_qk_norm_rope(x.half(), 1, 1, norm="none")
    with pytest.raises(ValueError):
        ra.ra_qk_norm_rope(x, 3, 1, norm="none")      # 192 elements are not 5 heads
    c = torch.zeros(1, 1, 4, 64, device="cuda")
    with pytest.raises(ValueError):
        ra.ra_cache_append(x, c, c.bfloat16(), pos[:1], 1, 1, norm="none")
    with pytest.raises(ValueError):
        ra.ra_cache_append(x, c, c, pos[:1].long(), 1, 1, norm="none")
