"""Refusals of the position and serving operators: the C ABI's host-side validation and the binding's
checks.  No GPU: every call here returns or raises before it would touch the device."""
import ctypes

import pytest
import torch

import rational_softmax_attention_gb300 as ra
from rational_softmax_attention_gb300 import build as ra_build

FAKE = ctypes.c_void_p(1 << 20)       # never dereferenced: every call below fails validation first
OTHER = [ctypes.c_void_p((1 << 20) + (i << 12)) for i in range(1, 8)]
MISALIGNED = ctypes.c_void_p((1 << 20) + 4)
ARG, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    ra_build.build()
    return ra.lib()


def _sections(s):
    return (ctypes.c_int32 * len(s))(*s) if s else None


def _norm_rope(lib, bwd=False, qkv=FAKE, bs=768, ts=192, qw=FAKE, qb=None, kw=FAKE, kb=None, norm=2, eps=1e-5,
               freq=FAKE, pos=FAKE, sections=(32,), axes=None, inter=0, out=FAKE, start=None, count=None, cap=0, B=2,
               N=4, Hq=1, Hkv=1, D=64, dt=1, ws=FAKE):
    lead = (qkv, bs, ts, qw, qb, kw, kb, norm, eps, freq, pos, 0, 0, _sections(sections),
            len(sections) if axes is None else axes, inter)
    if bwd:
        return lib.ra_qk_norm_rope_bwd(*lead, FAKE, FAKE, FAKE, out, FAKE, ws, B, N, Hq, Hkv, D, dt, None)
    return lib.ra_qk_norm_rope_fwd(*lead, out, FAKE, FAKE, start, count, cap, B, N, Hq, Hkv, D, dt, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_rope_validation(lib, bwd):
    bad = [dict(qkv=None), dict(qkv=MISALIGNED), dict(out=None), dict(out=MISALIGNED), dict(B=0), dict(N=0),
           dict(Hq=0), dict(Hkv=-1), dict(D=0), dict(dt=3), dict(norm=3), dict(norm=0), dict(qw=None), dict(kw=None),
           dict(qb=FAKE), dict(norm=1, qb=MISALIGNED), dict(eps=-1.0), dict(eps=float("nan")), dict(bs=4), dict(ts=7),
           dict(sections=(0, 8)), dict(sections=(33,)), dict(sections=(), axes=1), dict(sections=(8,), axes=-1),
           dict(freq=None), dict(pos=None), dict(B=1 << 20, N=1 << 20), dict(sections=((1 << 31) - 1,) * 4)]
    for how in bad:
        assert _norm_rope(lib, bwd, **how) == ARG, how
    unsupported = [dict(D=48, sections=(8,)), dict(D=256), dict(sections=(4,)), dict(sections=(1, 2, 2, 1, 2))]
    for how in unsupported:
        assert _norm_rope(lib, bwd, **how) == UNSUPPORTED, how


def test_norm_rope_own_arguments(lib):
    assert _norm_rope(lib, start=FAKE, cap=0) == ARG                # a cache needs a capacity
    assert _norm_rope(lib, cap=16) == ARG                           # and a capacity a cache
    assert _norm_rope(lib, count=FAKE) == ARG
    assert _norm_rope(lib, start=FAKE, cap=1 << 31 - 1, B=4, N=1) == ARG
    assert _norm_rope(lib, bwd=True, ws=None) == ARG
    assert lib.ra_qk_norm_rope_bwd_workspace_size(48) == 0
    assert lib.ra_qk_norm_rope_bwd_workspace_size(64) % (2 * 64 * 4) == 0


def _decode(lib, q=FAKE, length=FAKE, pk=None, pv=None, o=FAKE, weight=None, ws=FAKE, B=2, Hq=4, Hkv=2, C=16, P=0,
            D=64, scale=0.0, dt=1):
    return lib.ra_attention_decode(q, FAKE, FAKE, length, pk, pv, o, weight, ws, B, Hq, Hkv, C, P, D, scale, dt, None)


def test_decode_validation(lib):
    bad = [dict(q=None), dict(q=MISALIGNED), dict(length=None), dict(o=None), dict(ws=None), dict(ws=MISALIGNED),
           dict(B=0), dict(Hq=0), dict(Hkv=0), dict(C=0), dict(P=-1), dict(D=0), dict(Hq=3), dict(dt=2), dict(P=4),
           dict(P=4, pk=FAKE), dict(pk=FAKE, pv=FAKE), dict(P=4, pk=MISALIGNED, pv=FAKE), dict(scale=float("inf")),
           dict(weight=ctypes.c_void_p((1 << 20) + 2)), dict(length=ctypes.c_void_p((1 << 20) + 1)),
           dict(B=1 << 12, Hkv=1 << 12, Hq=1 << 12, C=1 << 10), dict(Hkv=1 << 16, Hq=1 << 16, P=1 << 16)]
    for how in bad:
        assert _decode(lib, **how) == ARG, how
    for how in [dict(D=48), dict(D=32), dict(D=256), dict(D=48, dt=0), dict(B=8193), dict(Hkv=1, Hq=1025)]:
        assert _decode(lib, **how) == UNSUPPORTED, how


def test_decode_workspace_size(lib):
    size = lib.ra_attention_decode_workspace_size
    assert size(2, 4, 2, 16, 0, 64, 1) > 0 and size(2, 3, 2, 16, 0, 64, 1) == 0 and size(2, 4, 2, 0, 0, 64, 1) == 0
    assert size(8193, 4, 2, 16, 0, 64, 1) == 0
    # more keys never need less
    assert size(2, 4, 2, 70000, 0, 64, 1) >= size(2, 4, 2, 1000, 0, 64, 1)
    assert size(2, 4, 2, 1000, 70000, 64, 1) >= size(2, 4, 2, 1000, 0, 64, 1)


def _evict(lib, k=FAKE, ko=OTHER[0], vo=OTHER[1], v=OTHER[2], w=OTHER[3], wo=OTHER[4], n=OTHER[5], no=OTHER[6],
           index=FAKE, B=2, H=2, C=64, Co=32, D=64, keep=16, recent=4, dt=1):
    return lib.ra_cache_evict(k, v, w, n, ko, vo, wo, no, index, B, H, C, Co, D, keep, recent, dt, None)


def test_evict_validation(lib):
    bad = [dict(k=None), dict(k=MISALIGNED), dict(ko=FAKE), dict(vo=OTHER[2]), dict(ko=OTHER[1]), dict(wo=OTHER[3]),
           dict(no=OTHER[5]), dict(index=None), dict(B=0), dict(H=0), dict(C=0), dict(Co=0), dict(D=0), dict(keep=0),
           dict(keep=33), dict(recent=17), dict(recent=-1), dict(dt=9), dict(C=1 << 30), dict(Co=1 << 30),
           dict(B=1, H=1, C=(1 << 31) - 1), dict(B=1, H=1, Co=(1 << 31) - 1)]
    for how in bad:
        assert _evict(lib, **how) == ARG, how
    assert _evict(lib, D=20) == UNSUPPORTED


def test_binding_refuses_before_the_library_is_called():
    x = torch.zeros(2, 4, 192, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_qk_norm_rope(x, 1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_attention_decode(x[:, :1, :64].contiguous(), torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_cache_evict(torch.zeros(2, 1, 8, 64), None, None, None, 4)
    with pytest.raises(ValueError):
        ra.ra_rope_frequencies((4, 0), device="cpu")


def test_frequencies():
    f = ra.ra_rope_frequencies((3, 1), theta=100.0, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, 100.0 ** (-torch.arange(4).double() / 4))
    f = ra.ra_rope_frequencies((2, 2), theta=100.0, per_axis=True, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 1.0, 0.1], dtype=torch.float64))


def test_cache_host_side_checks():
    c = ra.RaCache(2, 1, 8, 64, device="cpu", track_weight=False)
    assert c.capacity == 8 and c.prefix_length == 0
    c.require_room(8)
    c.advance(5)
    assert c.length.tolist() == [5, 5] and c.position.tolist() == [5, 5]
    c.advance(2, torch.tensor([1, 2], dtype=torch.int32))
    assert c.length.tolist() == [6, 7] and c.bound == 7
    with pytest.raises(ValueError, match="no room"):
        c.require_room(2)
    with pytest.raises(ValueError, match="track_weight"):
        c.evict(4)
    p = torch.zeros(1, 3, 64, dtype=torch.bfloat16)
    assert ra.RaCache(2, 1, 8, 64, device="cpu", prefix=(p, p)).position.tolist() == [3, 3]
    for bad in (torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.zeros(1, 3, 64)):
        with pytest.raises(ValueError, match="prefix"):
            ra.RaCache(2, 1, 8, 64, device="cpu", prefix=(bad, bad))
    with pytest.raises(ValueError):
        ra.RaCache(2, 0, 8, 64, device="cpu")


def test_module_host_side_checks():
    with pytest.raises(ValueError, match="rope_sections"):
        ra.RaAttention(64, num_heads=2, rope_sections=(17,))
    m = ra.RaAttention(64, num_heads=2)
    x = torch.zeros(1, 1, 64)
    with pytest.raises(ValueError, match="positions"):
        m(x, positions=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="causal"):
        m.decode(x, m.new_cache(1, 4))
    m = ra.RaAttention(64, num_heads=2, causal=True)
    with pytest.raises(ValueError, match="one token"):
        m.decode(torch.zeros(1, 2, 64), m.new_cache(1, 4))
    with pytest.raises(ValueError, match="no room"):
        m.prefill(torch.zeros(1, 5, 64), m.new_cache(1, 4))
    with pytest.raises(ValueError, match="batch size"):
        m.prefill(torch.zeros(1, 3, 64), m.new_cache(2, 4))
    with pytest.raises(ValueError, match="dtype"):
        m.prefill(torch.zeros(1, 3, 64), ra.RaCache(1, 2, 4, 32, device="cpu"))


def test_counts_beyond_the_call_are_not_counted():
    """Tokens that an append does not write do not lengthen the cache."""
    c = ra.RaCache(3, 1, 8, 64, device="cpu")
    c.advance(2, torch.tensor([5, -1, 1], dtype=torch.int32))
    assert c.length.tolist() == [2, 0, 1] and c.position.tolist() == [2, 0, 1] and c.bound == 2


def test_native_binding_refuses_what_is_no_tensor_or_size(lib):
    x, k = torch.zeros(2, 4, 192), torch.zeros(2, 1, 8, 64)
    for bad in ((None, k, k, k), ([1.0], k, k, k), (x, "k", k, k)):
        with pytest.raises(TypeError, match="tensor"):
            ra.ra_attention_decode(*bad)
    calls = pytest.importorskip("rational_softmax_attention_gb300._calls")
    with pytest.raises(TypeError, match="arguments"):
        calls.attention_decode(x)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_rope_refuses_a_token_beyond_32_bit_offsets(lib, bwd):
    """The kernels form offsets within a token, head * D up to 256 heads past the last, in 32 bits."""
    for Hq, Hkv, D in ((1 << 24, 1, 128), (1, 1 << 23, 128), (1 << 25, 1, 64), (((1 << 31) - 1) // 128 - 2, 1, 128)):
        assert (Hq + 2 * Hkv + 256) * D >= 1 << 31
        assert _norm_rope(lib, bwd, B=1, N=1, Hq=Hq, Hkv=Hkv, D=D, ts=0, bs=0) == ARG, (Hq, Hkv, D)


@pytest.mark.parametrize("which", ["qkv", "q_weight", "k_bias", "dk"])
def test_forward_mode_derivatives_are_refused(lib, which):
    """A tensor with a tangent has requires_grad False; its tangent would be dropped silently.  The refusal comes
    before the one of CPU tensors."""
    from torch.autograd import forward_ad
    x, w, d = torch.zeros(2, 4, 192), torch.ones(64), torch.zeros(2, 1, 4, 64)
    with forward_ad.dual_level():
        t = {"qkv": x, "q_weight": w, "k_bias": w, "dk": d}
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        how = dict(q_weight=t["q_weight"], k_weight=w, q_bias=w, k_bias=t["k_bias"])
        with pytest.raises(NotImplementedError, match="forward-mode"):
            if which == "dk":
                ra.ra_qk_norm_rope_backward(t["qkv"], d, t["dk"], d, 1, 1, **how)
            else:
                ra.ra_qk_norm_rope(t["qkv"], 1, 1, **how)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_qk_norm_rope(x, 1, 1, **dict(how, q_weight=w, k_bias=w))


def test_a_module_first_called_in_inference_mode_can_be_trained():
    """Its frequencies are made on the first call and saved for the backward of later ones, which torch allows
    only of tensors made outside inference mode."""
    m = ra.RaAttention(64, num_heads=2, rope_sections=(16,))
    with torch.inference_mode():
        how = m._how(torch.arange(3, dtype=torch.int32))
    assert not how["frequencies"].is_inference() and m._how(None)["frequencies"] is how["frequencies"]


def test_module_refuses_rotations_that_no_call_takes():
    """What the kernels do not take is refused when the module is made, not at its first forward."""
    for dim, heads, how in ((64, 2, dict(rope_sections=(4,))), (64, 2, dict(rope_sections=(8, 3))),
                            (96, 2, dict(rope_sections=(8,))), (512, 2, dict(rope_sections=(64,))),
                            (64, 2, dict(rope_sections=(2, 2, 2, 1, 1)))):
        with pytest.raises(ValueError, match="rope_sections"):
            ra.RaAttention(dim, num_heads=heads, **how)
    ra.RaAttention(64, num_heads=2, rope_sections=(3, 2), rope_interleaved=True)
    ra.RaAttention(64, num_heads=2, rope_sections=(3, 5))


def test_padding_does_not_fill_a_cache():
    """A ragged batch's padded tokens are not entries: what counts is whether each sequence has room."""
    c = ra.RaCache(2, 1, 8, 64, device="cpu")
    for _ in range(3):                       # 4 padded tokens a time, 2 and 1 of them real
        n = torch.tensor([2, 1], dtype=torch.int32)
        c.require_room(4, n)
        c.advance(4, n)
    assert c.length.tolist() == [6, 3] and c.bound <= 8
    c.require_room(2)
    assert c.bound == 6
    c.require_room(4, torch.tensor([2, 4], dtype=torch.int32))
    for tokens, n in ((3, None), (4, [3, 0]), (9, [0, 6])):
        with pytest.raises(ValueError, match="no room"):
            c.require_room(tokens, None if n is None else torch.tensor(n, dtype=torch.int32))
    assert c.bound == 6
