"""RaAttention on a paged cache: prompts that continue a cache after replays, and the module's outputs against 64 bits on the
values that the cache holds.

Bound of an output y = W o + b: o is a row's attention, rounded to bf16 (half a step, 2^-8 |o|), from weights that the
tensor-core call rounds to bf16 (2^-8 sum_j p_j |v_j| =: 2^-8 S).  These errors of the columns c differ from one another, so by Hoeffding's
inequality |sum_c W_c e_c| <= 6 sqrt(sum_c (W_c b_c)^2), b_c = 2^-8 (|o_c| + S_c), but for 2 exp(-18) of the outputs; and
half a step of y.  At these sizes about 0.012, where a lost entry and a mask that is off by one give several times as much, which the
test states of its own reference."""
import pytest
import torch

import rational_softmax_attention_gb300 as ra

pytestmark = pytest.mark.gpu


def make_module(dtype=torch.bfloat16, dim=256, heads=4):
    torch.manual_seed(0)
    return ra.RaAttention(dim, num_heads=heads, qk_norm=True, causal=True, rope_sections=(32,), device="cuda", dtype=dtype)


def reference(m, x, first, k, v, seen):
    """(y, bound) in 64 bits: x [B, N, dim] from position `first` on, against k, v [B, H, C, D], where seen [N, C]."""
    B, N, _ = x.shape
    with torch.no_grad():
        qkv = m.qkv(x)
        positions = (first + torch.arange(N, device="cuda", dtype=torch.int32)).expand(B, N).contiguous()
        q = ra.ra_qk_norm_rope(qkv, m.num_heads, **m._how(positions, qkv.dtype))[0].double()
        z = (q @ k.double().transpose(-1, -2)) * m.head_dim ** -0.5
        z = z.masked_fill(~seen, -torch.inf)
        u = ((z.amax(-1, keepdim=True) - z) / 16.0).clamp(max=1.0)
        p = ((1.0 - u) / (1.0 + u)) ** 8
        p = p / p.sum(-1, keepdim=True)
        o, S = ((p @ t).transpose(1, 2).reshape(B, N, -1) for t in (v.double(), v.double().abs()))
        W = m.proj.weight.double()
        y = o @ W.T + (0.0 if m.proj.bias is None else m.proj.bias.double())
        b = 2.0 ** -8 * (o.abs() + S)
        return y, 6.0 * ((b * b) @ (W * W).T).sqrt() + 2.0 ** -8 * y.abs()


def test_continued_prompts_and_tokens_against_64_bits():
    """A prompt forked into four, continued over a shared page's border, then single tokens: the mask and the copied page."""
    m = make_module()
    first, then, steps = 50, 21, 14
    x = torch.randn(4, first + then + steps, 256, device="cuda").bfloat16()
    x[:, :first] = x[:1, :first]
    c = m.new_cache(4, 96, page_size=16)
    y = m.prefill(x[:, :first], c, count=torch.tensor([first, 0, 0, 0], dtype=torch.int32, device="cuda"))
    c.fork(torch.zeros(4, dtype=torch.int32, device="cuda"))
    got = {(0, first): y[:1], (first, then): m.prefill(x[:, first:first + then], c)}
    for i in range(first + then, first + then + steps):
        got[i, 1] = m.decode(x[:, i:i + 1], c)
    slot, shows = torch.arange(c.capacity, device="cuda"), {}
    for (at, n), y in got.items():
        B = y.shape[0]
        # a prompt attends to the values that the cache gives in bf16, a token to those that it holds
        k, v = (t[:B] for t in ra.ra_page_read(c.pool, c.table, c.length, c.capacity, dtype=torch.bfloat16 if n > 1 else torch.float32))
        row = at + torch.arange(n, device="cuda").view(n, 1)
        want, bound = reference(m, x[:B, at:at + n], at, k, v, slot <= row)
        worst = ((y.double() - want).abs() / bound).max().item()
        assert worst <= 1.0, (at, n, worst)
        if at:   # what mistakes would give, in the reference alone
            for name, seen in (("mask", slot < row), ("lost", (slot <= row) & (slot != first - 1))):
                wrong = ((reference(m, x[:B, at:at + n], at, k, v, seen)[0] - want).abs() / bound).max().item()
                shows[name, n] = max(shows.get((name, n), 0.0), wrong)
    assert min(shows.values()) > 1.5, shows


@pytest.mark.parametrize("captured", ["token", "prompt"])
def test_a_prompt_after_a_freed_cache_and_replays(captured):
    """What a graph's replays have stored since a cache was emptied counts for the next prompt."""
    m = make_module()
    x = torch.randn(2, 30, 256, device="cuda").bfloat16()
    c, plain = (m.new_cache(2, 64, page_size=16) for _ in range(2))
    call, n = (m.decode, 1) if captured == "token" else (m.prefill, 5)
    static = x[:, :n].clone()
    m.prefill(static, c)
    c.free([0, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = call(static, c)
    torch.cuda.current_stream().wait_stream(side)
    c.free([0, 1])
    graph.replay()
    assert torch.equal(y, call(static, plain)) and c.length.tolist() == [n, n]
    assert torch.equal(m.prefill(x[:, n:20], c), m.prefill(x[:, n:20], plain))
    assert c.length.tolist() == [20, 20] and c.bound == 20
    assert torch.equal(c.pool, plain.pool)


def test_a_cache_emptied_by_a_fork_takes_prompts():
    """In fp32 too, where only an empty cache does: the lengths decide, not the host's count."""
    m = make_module(torch.float32)
    x = torch.randn(2, 9, 256, device="cuda")
    c = m.new_cache(2, 16, page_size=16)
    want = m.prefill(x, c)
    with pytest.raises(NotImplementedError, match="bf16"):
        m.prefill(x[:, :2], c)
    c.fork(torch.full((2,), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(m.prefill(x, c), want) and c.length.tolist() == [9, 9]


def test_a_compacted_cache_goes_on_in_a_pool_with_room():
    """compact() keeps no free page: tokens fit up to the page's border; compact(more) makes room."""
    m = make_module()
    x = torch.randn(2, 40, 256, device="cuda").bfloat16()
    c, plain = (m.new_cache(2, 64, page_size=16) for _ in range(2))
    for cache in (c, plain):
        m.prefill(x[:, :30], cache)
    c.compact()
    assert c.pages == 4 and (c.uses == 1).all()
    for i in (30, 31):
        assert torch.equal(m.decode(x[:, i:i + 1], c), m.decode(x[:, i:i + 1], plain))
    with pytest.raises(ValueError, match="0 free pages of 4: 2 are needed"):
        m.decode(x[:, 32:33], c)
    c.compact(6)
    for i in range(32, 40):
        assert torch.equal(m.decode(x[:, i:i + 1], c), m.decode(x[:, i:i + 1], plain))
