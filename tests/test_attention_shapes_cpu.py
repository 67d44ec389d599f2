"""ra_attention refuses tensors whose shapes or dtypes do not go together before anything is launched: the kernels
take B, H and the dtype from q and read k, v, the mask, the statistics and the workspace by them.  No GPU: the
checks come before the one that refuses CPU tensors, whose message says "CUDA"."""
import pytest
import torch

import rational_softmax_attention_gb300 as ra
from rational_softmax_attention_gb300 import build as ra_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    ra_build.build()
    return ra.lib()


def qkv(B=2, H=4, NQ=6, NK=9, D=64, dtype=torch.bfloat16):
    return (torch.zeros(B, H, NQ, D, dtype=dtype), torch.zeros(B, H, NK, D, dtype=dtype),
            torch.zeros(B, H, NK, D, dtype=dtype))


def packed(L, B, H, n_q, n_k, MB, MH):
    return (torch.zeros(MB * MH, n_q, L.ra_attention_mask_words(n_k), dtype=torch.int32),
            torch.zeros(MB * MH, n_k, L.ra_attention_mask_words(n_q), dtype=torch.int32), MB, MH)


def test_shapes_that_go_together_reach_the_cuda_check(lib):
    q, k, v = qkv()
    for call in (ra.ra_attention, ra.ra_attention_forward):
        with pytest.raises(ValueError, match="CUDA"):
            call(q, k, v)


@pytest.mark.parametrize("call", [ra.ra_attention, ra.ra_attention_forward])
def test_keys_and_values_unlike_the_queries_are_refused(call):
    q, k, v = qkv()
    few = [t[:, :2].contiguous() for t in (k, v)]                 # two key heads for four query heads
    bad = [(q, *few), (q, k, few[1]), (q, few[0], v), (q, k[:1], v[:1]), (q, k[..., :32], v[..., :32]),
           (q, k, v[:, :, :8]), (q, k, v[..., :32]), (q[0], k[0], v[0]), (q, k[:, :, :, None], v)]
    for a, b, c in bad:
        with pytest.raises(ValueError, match="heads"):
            call(a, b, c)
    for a, b, c in ((q, k.float(), v), (q, k, v.float()), (q.float(), k, v)):
        with pytest.raises(ValueError, match="must be torch"):
            call(a, b, c)


def test_a_mask_of_other_sizes_is_refused(lib):
    q, k, v = qkv()
    good = packed(lib, 2, 4, 6, 9, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_attention_forward(q, k, v, mask=good)
    for bad in (packed(lib, 2, 4, 5, 9, 2, 1), packed(lib, 2, 4, 6, 200, 1, 1), packed(lib, 2, 4, 6, 9, 3, 1),
                (*packed(lib, 2, 4, 6, 9, 1, 1)[:2], 2, 4)):
        with pytest.raises(ValueError, match="pack_attn_mask"):
            ra.ra_attention_forward(q, k, v, mask=bad)
    with pytest.raises(ValueError, match="mask_q"):
        ra.ra_attention_forward(q, k, v, mask=(good[0].float(), *good[1:]))


def test_the_backward_checks_what_the_forward_gave(lib):
    q, k, v = qkv()
    rows = torch.zeros(2, 4, 6)
    args = dict(o=q.float(), dout=q, row_m=rows, row_s=rows, row_arg=rows.int())

    def call(**other):
        a = dict(args, **other)
        keys = a.pop("k", k), a.pop("v", v)
        extra = {n: a.pop(n) for n in ("workspace",) if n in a}
        return ra.ra_attention_backward(q, *keys, a["o"], a["dout"], a["row_m"], a["row_s"], a["row_arg"], **extra)
    with pytest.raises(ValueError, match="CUDA"):
        call()
    for other, what in ((dict(k=k[:, :2], v=v[:, :2]), "heads"), (dict(o=q[:, :, :5]), "o and dout"),
                        (dict(dout=q[:, :2]), "o and dout"), (dict(dout=q.float()), "dout"),
                        (dict(row_m=rows[:1]), "row_m"), (dict(row_s=rows.double()), "row_s"),
                        (dict(row_arg=rows.long()), "row_arg"),
                        (dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace")):
        with pytest.raises(ValueError, match=what):
            call(**other)
