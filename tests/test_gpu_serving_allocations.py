"""Outputs and workspaces of the serving calls are tensors that torch's modes see, like those of any other call."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import rational_softmax_attention_gb300 as ra

pytestmark = pytest.mark.gpu


class Allocations(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.shapes.append(tuple(out.shape))
        return out


def calls():
    pool, table = ra.ra_page_pool(4, 2, 64, 16), torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    n, uses = torch.full((2,), 20, dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    qkv, k = torch.randn(2, 5, 6 * 64, device="cuda"), torch.randn(2, 2, 5, 64, device="cuda")
    q, cache = torch.randn(2, 4, 64, device="cuda"), torch.randn(2, 2, 32, 64, device="cuda")
    out = torch.zeros_like(pool)
    return {"norm_rope": (lambda: ra.ra_qk_norm_rope(qkv, 2, norm="none"), 3),
            "decode": (lambda: ra.ra_attention_decode(q, cache, cache, n), 2),
            "write": (lambda: ra.ra_page_write(k, k, pool, table, held=True), 2),
            "read": (lambda: ra.ra_page_read(pool, table, n, 20), 2),
            "decode_paged": (lambda: ra.ra_attention_decode_paged(q, pool, table, n), 2),
            "reserve": (lambda: ra.ra_page_reserve(pool, table, n, uses, 3), 2),
            "compact": (lambda: ra.ra_page_compact(pool, table, uses, out), 4)}


@pytest.mark.parametrize("name", ["norm_rope", "decode", "write", "read", "decode_paged", "reserve", "compact"])
def test_modes_see_what_a_call_allocates(name):
    call, tensors = calls()[name]
    plain = call()
    with Allocations() as seen:
        got = call()
    assert len(seen.shapes) >= tensors
    for a, b in zip(*((x if isinstance(x, (tuple, list)) else (x,)) for x in (got, plain))):
        assert torch.equal(a, b) and tuple(a.shape) in seen.shapes


def test_results_do_not_depend_on_what_was_there():
    """With deterministic algorithms on, torch fills what it allocates."""
    made = {name: call for name, (call, _) in calls().items() if name != "reserve"}   # which changes its own inputs
    want = {name: call() for name, call in made.items()}
    torch.use_deterministic_algorithms(True)
    try:
        got = {name: call() for name, call in made.items()}
    finally:
        torch.use_deterministic_algorithms(False)
    for name in made:
        for a, b in zip(*((x if isinstance(x, (tuple, list)) else (x,)) for x in (got[name], want[name]))):
            assert torch.equal(a, b), name
