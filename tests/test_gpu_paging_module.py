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
