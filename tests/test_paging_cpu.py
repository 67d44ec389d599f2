"""Refusals of the paged cache: the C ABI's host-side validation, the binding's checks and the cache's own.  No GPU:
every call here returns or raises before it would touch the device."""
import ctypes

import pytest
import torch

import rational_softmax_attention_gb300 as ra
from rational_softmax_attention_gb300 import build as ra_build

FAKE = ctypes.c_void_p(1 << 20)       # never dereferenced: every call below fails validation first
OTHER = [ctypes.c_void_p((1 << 20) + (i << 12)) for i in range(1, 8)]
MISALIGNED, ODD = ctypes.c_void_p((1 << 20) + 4), ctypes.c_void_p((1 << 20) + 1)
ARG, UNSUPPORTED = 1, 2
MAX = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    ra_build.build()
    return ra.lib()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def _rows(lib, write, k=FAKE, v=FAKE, ks=strides(256, 128, 64), vs=strides(256, 128, 64), pool=FAKE, stride=1 << 16, table=FAKE,
          start=None, limit=None, kh=None, vh=None, B=2, N=2, H=2, D=64, pages=4, page=16, M=3, dt=1):
    if write:
        return lib.ra_page_write(k, v, ks, vs, pool, stride, table, start, limit, kh, vh, B, N, H, D, pages, page, M, dt, None)
    return lib.ra_page_read(pool, stride, table, start, limit, k, v, B, N, H, D, pages, page, M, dt, None)


@pytest.mark.parametrize("write", [True, False])
def test_rows_validation(lib, write):
    bad = [dict(k=None), dict(v=None), dict(k=MISALIGNED), dict(pool=None), dict(pool=MISALIGNED), dict(stride=8), dict(stride=16),
           dict(stride=-(1 << 16)), dict(table=None), dict(table=ODD), dict(start=ODD), dict(limit=ODD), dict(B=0), dict(N=0),
           dict(H=0), dict(D=0), dict(pages=0), dict(page=0), dict(M=0), dict(M=-1), dict(dt=2), dict(M=1 << 28), dict(B=1 << 30, M=3),
           dict(B=1 << 16, N=1 << 14), dict(H=1 << 24), dict(N=MAX)]
    if write:
        bad += [dict(ks=None), dict(vs=strides(256, 128, 60)), dict(ks=strides(4, 128, 64)), dict(kh=FAKE), dict(kh=FAKE, vh=MISALIGNED)]
    for how in bad:
        assert _rows(lib, write, **how) == ARG, how
    for how in (dict(D=32), dict(D=96), dict(D=256), dict(page=8), dict(page=48), dict(page=512)):
        assert _rows(lib, write, **how) == UNSUPPORTED, how


def _decode(lib, q=FAKE, pool=FAKE, stride=1 << 16, table=FAKE, length=FAKE, o=FAKE, ws=FAKE, B=2, Hq=4, H=2, D=64, pages=4, page=16,
            M=3, scale=0.0, dt=1):
    return lib.ra_attention_decode_paged(q, pool, stride, table, length, o, ws, B, Hq, H, D, pages, page, M, scale, dt, None)


def test_decode_validation(lib):
    for how in [dict(q=None), dict(q=MISALIGNED), dict(pool=None), dict(pool=MISALIGNED), dict(stride=24), dict(stride=16), dict(table=None),
                dict(table=ODD), dict(length=None), dict(length=ODD), dict(o=None), dict(o=MISALIGNED), dict(ws=None), dict(ws=MISALIGNED),
                dict(B=0), dict(Hq=0), dict(H=0), dict(D=0), dict(pages=0), dict(page=0), dict(M=0), dict(Hq=3), dict(scale=float("inf")),
                dict(dt=7), dict(M=1 << 27), dict(B=1 << 16, Hq=1 << 16)]:
        assert _decode(lib, **how) == ARG, how
    for how in [dict(D=32), dict(D=256), dict(page=24), dict(B=8193), dict(H=1, Hq=1025)]:
        assert _decode(lib, **how) == UNSUPPORTED, how
    size = lib.ra_attention_decode_paged_workspace_size
    assert size(2, 4, 2, 3, 16, 64) > 0
    assert [size(*s) for s in ((2, 3, 2, 3, 16, 64), (2, 4, 2, 0, 16, 64), (8193, 4, 2, 3, 16, 64), (2, 4, 2, 3, 20, 64),
                               (2, 4, 2, 3, 16, 80), (8192, 64, 64, 1 << 20, 256, 64))] == [0] * 6
    assert size(2, 4, 2, 5000, 16, 64) >= size(2, 4, 2, 300, 16, 64)


def test_table_validation(lib):
    def fork(table=FAKE, length=FAKE, uses=FAKE, parent=FAKE, B=2, M=3, pages=4):
        return lib.ra_page_fork(table, length, uses, parent, B, M, pages, None)
    for how in [dict(table=None), dict(length=None), dict(uses=None), dict(parent=None), dict(parent=ODD), dict(B=0), dict(M=0), dict(pages=0),
                dict(B=8000, M=1 << 20)]:
        assert fork(**how) == ARG, how
    assert fork(B=8193) == UNSUPPORTED

    def reserve(pool=FAKE, stride=1 << 16, page_bytes=1 << 12, table=FAKE, length=FAKE, uses=FAKE, count=None, granted=FAKE, ws=FAKE, B=2, M=3,
                tokens=5, pages=4, page=16):
        return lib.ra_page_reserve(pool, stride, page_bytes, table, length, uses, count, granted, ws, B, M, tokens, pages, page, None)
    for how in [dict(pool=None), dict(pool=MISALIGNED), dict(stride=100), dict(stride=2048), dict(page_bytes=0), dict(page_bytes=40), dict(table=None),
                dict(length=None), dict(uses=None), dict(count=ODD), dict(granted=None), dict(ws=None), dict(ws=MISALIGNED), dict(B=0), dict(M=0),
                dict(tokens=0), dict(pages=0), dict(page=0), dict(M=1 << 28), dict(tokens=MAX), dict(B=1 << 20, tokens=1 << 20), dict(B=1 << 30)]:
        assert reserve(**how) == ARG, how
    assert reserve(page=24) == UNSUPPORTED
    size = lib.ra_page_reserve_workspace_size
    assert size(2, 5, 16) > 0 and [size(0, 5, 16), size(2, 0, 16), size(2, 5, 17), size(1 << 20, 1 << 20, 16), size(2, MAX, 16)] == [0] * 5

    def compact(pool=FAKE, stride=1 << 16, table=OTHER[0], uses=OTHER[1], out=OTHER[2], out_stride=1 << 16, t=OTHER[3], u=OTHER[4], live=OTHER[5],
                ws=FAKE, page_bytes=1 << 12, B=2, M=3, pages=4, pages_out=4):
        return lib.ra_page_compact(pool, stride, table, uses, out, out_stride, t, u, live, ws, page_bytes, B, M, pages, pages_out, None)
    for how in [dict(pool=None), dict(pool=MISALIGNED), dict(stride=8), dict(out_stride=16), dict(table=None), dict(uses=None), dict(out=None), dict(t=None),
                dict(u=None), dict(live=None), dict(live=ODD), dict(ws=None), dict(page_bytes=8), dict(B=0), dict(M=0), dict(pages=0), dict(pages_out=0),
                dict(out=FAKE), dict(t=OTHER[0]), dict(u=OTHER[1]), dict(B=1 << 16, M=1 << 16)]:
        assert compact(**how) == ARG, how
    assert lib.ra_page_compact_workspace_size(0) == 0 and lib.ra_page_compact_workspace_size(100) >= 800


def test_binding_refuses_before_the_library_is_called():
    pool, table = ra.ra_page_pool(4, 2, 64, 16, device="cpu"), torch.zeros(2, 3, dtype=torch.int32)
    assert pool.shape == (4, 2, 2, 16, 36) and ra.ra_page_pool(1, 1, 128, device="cpu").shape == (1, 1, 2, 64, 72)
    k, n = torch.zeros(2, 2, 5, 64), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ra.ra_page_write(k, k, pool, table), lambda: ra.ra_page_read(pool, table, n, 4),
                 lambda: ra.ra_attention_decode_paged(k[:, :, 0].contiguous(), pool, table, n), lambda: ra.ra_page_fork(table, n, n, n),
                 lambda: ra.ra_page_reserve(pool, table, n, n, 1), lambda: ra.ra_page_compact(pool, table, n, pool)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: ra.ra_page_write(None, k, pool, table), lambda: ra.ra_page_read([1], table, n, 4),
                 lambda: ra.ra_page_fork(table.tolist(), n, n, n)):
        with pytest.raises(TypeError, match="tensor"):
            call()
    with pytest.raises(TypeError, match="dtype"):
        ra.ra_page_read(pool, table, n, 4, dtype=torch.float16)
    for bad in ((4, 2, 96, 16), (4, 2, 64, 24), (0, 2, 64, 16), (4, 0, 64, 16)):
        with pytest.raises(ValueError):
            ra.ra_page_pool(*bad, device="cpu")


def test_cache_and_module_refuse_on_the_host():
    with pytest.raises(ValueError, match="head_dim"):
        ra.RaPagedCache(2, 2, 64, 32, device="cpu")
    for size in (0, 10):
        with pytest.raises(ValueError, match="page_size"):
            ra.RaPagedCache(2, 2, 64, 64, page_size=size, device="cpu")
    with pytest.raises(ValueError, match="at least 1"):
        ra.RaPagedCache(0, 2, 64, 64, device="cpu")
    with pytest.raises(TypeError, match="dtype"):
        ra.RaPagedCache(2, 2, 64, 64, device="cpu", dtype=torch.float16)
    m = ra.RaAttention(128, num_heads=2, causal=True)
    for how in (dict(page_size=16, track_weight=True), dict(page_size=16, prefix=(None, None)), dict(pages=3)):
        with pytest.raises(ValueError):
            m.new_cache(1, 4, **how)
    c = m.new_cache(2, 40, page_size=16)
    assert c.capacity == 48 and c.pages == 6 and c.head_dim == 64 and c.num_kv_heads == 2 and c.page_size == 16
    for x, cache, match in ((torch.zeros(1, 3, 128), c, "batch size"), (torch.zeros(2, 49, 128), c, "no room"),
                            (torch.zeros(2, 3, 128), ra.RaPagedCache(2, 2, 40, 128, device="cpu"), "head dim"),
                            (torch.zeros(2, 3, 128), ra.RaPagedCache(2, 2, 40, 64, device="cpu"), "dtype")):
        with pytest.raises(ValueError, match=match):
            m.prefill(x, cache)
    c.bound = 3
    with pytest.raises(NotImplementedError, match="bf16"):
        m.prefill(torch.zeros(2, 3, 128), c)
    with pytest.raises(ValueError, match="causal"):
        ra.RaAttention(128, num_heads=2).prefill(torch.zeros(2, 3, 128), c)


def test_room_is_counted_in_entries_and_pages():
    """The host's bound first; where it leaves a doubt, the table itself."""
    c = ra.RaPagedCache(3, 1, 64, 64, page_size=16, pages=5, device="cpu")
    c.require_room(16)                              # a page each
    with pytest.raises(ValueError, match="5 free pages of 5: 6"):
        c.require_room(17)
    c.require_room(17, torch.tensor([17, 1, 2], dtype=torch.int32))
    with pytest.raises(ValueError, match="no room"):
        c.require_room(65, torch.tensor([65, 0, 0], dtype=torch.int32))
    # sequence 0 holds 30 entries, 1 shares its pages, 2 is empty
    c.table[0, :2] = c.table[1, :2] = torch.tensor([0, 3], dtype=torch.int32)
    c.uses[0] = c.uses[3] = 2
    c.length[:2] = 30
    c.bound, c.shared = 30, True
    c.require_room(1)                               # a copy for each sharer and a page: 3 of 3
    with pytest.raises(ValueError, match="3 free pages of 5: 5"):
        c.require_room(3)
    c.require_room(3, torch.tensor([0, 2, 3], dtype=torch.int32))
    c.uses[3] = 1
    c.table[1, 1] = 4
    c.uses[4] = 1
    c.require_room(2)
    assert c.bound == 30


def test_a_scale_that_is_not_finite_is_refused(lib):
    """NaN too, which is not above 0 either and would pass for the default."""
    for scale in (float("nan"), float("-inf"), float("inf")):
        assert _decode(lib, scale=scale) == ARG, scale
