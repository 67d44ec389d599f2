"""RaAttention on a paged cache: prompts that continue a cache after replays."""
import pytest
import torch

import rational_softmax_attention_gb300 as ra

pytestmark = pytest.mark.gpu


def make_module(dtype=torch.bfloat16, dim=256, heads=4):
    torch.manual_seed(0)
    return ra.RaAttention(dim, num_heads=heads, qk_norm=True, causal=True, rope_sections=(32,), device="cuda", dtype=dtype)


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
