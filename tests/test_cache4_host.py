"""What the cache held in 4 bits, attention over it and the pages of a cache refuse
before any GPU call."""
import ctypes
import math

import pytest

import gptq_bit_weight_amd as q4

S = ctypes.c_int64 * 3


def _cache(**kw):
    from gptq_bit_weight_amd.attention import _Cache4
    # 4 pages of 2 heads of 16 rows of 64 values: 32 bytes of codes and 8 of scales a row
    c = _Cache4(1 << 20, 2 << 20, 3 << 20, 4 << 20, S(1024, 512, 32), S(1024, 512, 32), S(256, 128, 8), S(256, 128, 8), 4, 2, 16, 64, 32)
    for k, v in kw.items():
        setattr(c, k, S(*v) if k.endswith("stride") else v)
    return c


BAD_CACHES = [
    (dict(k=None), 1), (dict(v_scale=None), 1), (dict(pages=0), 1), (dict(kv_heads=0), 1), (dict(page_size=-1), 1), (dict(dim=0), 1),
    (dict(pages=1 << 20, page_size=1 << 12), 2), (dict(dim=48), 2), (dict(dim=288, group=32), 2), (dict(group=16), 2), (dict(group=0), 2),
    (dict(group=128), 2), (dict(group=48), 2), (dict(dim=96, group=64), 2), (dict(k_stride=(1024, 512, 40)), 2), (dict(v_stride=(1032, 512, 32)), 2),
    (dict(v_stride=(-1024, 512, 32)), 2), (dict(k_scale_stride=(256, 130, 8)), 2), (dict(v_scale_stride=(256, 128, -8)), 2),
    (dict(k_stride=(1024, 512, 1 << 27)), 2), (dict(v_scale_stride=(1024, 512, 1 << 27)), 2), (dict(k=(1 << 20) + 8), 2),
    (dict(v_scale=(4 << 20) + 2), 2)]


@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_caches(cache, status):
    lib = q4.load_library()
    c = _cache(**cache)
    ref = ctypes.byref(c)
    assert lib.q4_check_cache4(ref) == status and lib.q4_last_error()
    assert _append(lib, c) == status
    assert _read(lib, c) == status
    assert _attend(lib, c) == status
    assert lib.q4_attend4_workspace(ref, 4) == 0


def test_a_cache():
    assert q4.load_library().q4_check_cache4(ctypes.byref(_cache())) == 0


def _append(lib, c, **kw):
    a = dict(k=8 << 20, k_token=128, k_head=64, v=9 << 20, v_token=128, v_head=64, slots=10 << 20, slot_bits=64, tokens=6, rotary=None,
             positions=None, position_bits=64, q=None, q_token=256, q_head=64, q_out=None, o_token=256, o_head=64, heads=0, bf16=0)
    a.update(kw)
    return lib.q4_cache4_append(None if c is None else ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(slot_bits=16), 1), (dict(tokens=-1), 1), (dict(heads=-1), 1),
    (dict(k_token=-128), 2), (dict(v_head=1 << 31), 2), (dict(k_token=1 << 31), 2), (dict(q=11 << 20, q_out=12 << 20, heads=4), 1),
    (dict(k=1 << 20), 1), (dict(v=(4 << 20) + 512), 1), (dict(slots=(2 << 20) + 4000), 1), (dict(slots=(3 << 20) - 48 + 8), 1)])
def test_append_refuses(kw, status):
    lib = q4.load_library()
    assert _append(lib, _cache(), **kw) == status and lib.q4_last_error()


def test_append_of_nothing():
    lib = q4.load_library()
    assert _append(lib, _cache(), tokens=0, k=None) == 0
    assert _append(lib, None) == 1


def _read(lib, c, **kw):
    a = dict(slots=10 << 20, slot_bits=32, tokens=6, k=8 << 20, k_token=128, k_head=64, v=9 << 20, v_token=128, v_head=64)
    a.update(kw)
    return lib.q4_cache4_read(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(slot_bits=8), 1), (dict(tokens=-1), 1), (dict(tokens=1 << 28), 2),
    (dict(v=8 << 20), 1), (dict(k=2 << 20), 1), (dict(v=3 << 20), 1), (dict(slots=8 << 20), 1)])
def test_read_refuses(kw, status):
    lib = q4.load_library()
    assert _read(lib, _cache(), **kw) == status and lib.q4_last_error()
    assert _read(lib, _cache(), tokens=0) == 0


def _attend(lib, c, **kw):
    a = dict(q=8 << 20, q_token=512, q_head=64, heads=8, tokens=3, starts=10 << 20, lengths=11 << 20, table=12 << 20, width=2, stride=2,
             requests=2, window=0, sinks=0, scale=0.125, out=9 << 20, o_token=512, o_head=64, ws=None, ws_bytes=0, bf16=0)
    a.update(kw)
    return lib.q4_attend4(ctypes.byref(c), *a.values(), None)


REFUSED = [
    (dict(heads=0), 1), (dict(heads=7), 1), (dict(tokens=-1), 1), (dict(requests=-1), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
    (dict(scale=math.nan), 1), (dict(scale=-math.inf), 1), (dict(q=None), 1), (dict(starts=None), 1), (dict(lengths=None), 1),
    (dict(table=None), 1), (dict(out=None), 1), (dict(width=0), 1), (dict(stride=1), 1), (dict(stride=1 << 31), 1), (dict(q=(8 << 20) + 8), 2),
    (dict(q_token=508), 2), (dict(q_head=-64), 2), (dict(tokens=1 << 30), 2), (dict(out=(9 << 20) + 1), 2), (dict(out=8 << 20), 1)]


@pytest.mark.parametrize("kw,status", REFUSED + [(dict(out=x << 20), 1) for x in (1, 2, 3, 4, 10, 11, 12)])
def test_attend4_refuses(kw, status):
    lib = q4.load_library()
    assert _attend(lib, _cache(), **kw) == status and lib.q4_last_error()


def test_attend4_of_nothing():
    lib = q4.load_library()
    assert _attend(lib, _cache(), tokens=0) == 0
    assert _attend(lib, _cache(), requests=0) == 0


@pytest.mark.parametrize("kw,status", REFUSED + [(dict(out=x << 20), 1) for x in (1, 2, 10, 11, 12)])
def test_attend_with_sinks_refuses(kw, status):
    from gptq_bit_weight_amd.attention import _Cache
    lib = q4.load_library()
    c = _Cache(1 << 20, 2 << 20, S(2048, 1024, 64), S(2048, 1024, 64), 4, 2, 16, 64, 0)
    a = dict(q=8 << 20, q_token=512, q_head=64, heads=8, tokens=3, starts=10 << 20, lengths=11 << 20, table=12 << 20, width=2, stride=2,
             requests=2, window=5, sinks=3, scale=0.125, out=9 << 20, o_token=512, o_head=64, ws=None, ws_bytes=0)
    a.update(kw)
    assert lib.q4_attend_ex(ctypes.byref(c), *a.values(), None) == status and lib.q4_last_error()


# ------------------------------------------------------------------- pages ---

def _pool(**kw):
    from gptq_bit_weight_amd.attention import _Pool
    p = _Pool()
    for i, at in enumerate((1 << 20, 2 << 20)):
        x = p.plane[i]
        x.at, x.page, x.head, x.row, x.heads, x.rows, x.bytes = at, 4096, 2048, 128, 2, 16, 128
    p.planes, p.pages = 2, 8
    for k, v in kw.items():
        setattr(p if k in ("planes", "pages") else p.plane[1], k, v)
    return p


BAD_POOLS = [(dict(planes=0), 1), (dict(planes=5), 1), (dict(pages=0), 1), (dict(at=None), 1), (dict(page=-1), 1), (dict(head=-1), 1),
             (dict(row=-1), 1), (dict(heads=0), 1), (dict(rows=0), 1), (dict(bytes=0), 1), (dict(rows=1 << 20, bytes=1 << 20), 2),
             (dict(rows=1 << 15, bytes=(1 << 14) + 1), 2)]


def _copy(lib, pool, src=8 << 20, src_bits=32, dst=9 << 20, dst_bits=64, n=4):
    return lib.q4_copy_pages(None if pool is None else ctypes.byref(pool), src, src_bits, dst, dst_bits, n, None)


@pytest.mark.parametrize("pool,status", BAD_POOLS)
def test_pools(pool, status):
    lib = q4.load_library()
    assert _copy(lib, _pool(**pool)) == status and lib.q4_last_error()
    pages, ref = _books()
    if "pages" not in pool:
        assert lib.q4_pages_fork(ref, ctypes.byref(_pool(**pool)), 8 << 20, 32, 9 << 20, 32, 2, 10 << 20, None) == status
        assert lib.q4_pages_compact(ref, ctypes.byref(_pool(**pool)), 10 << 20, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(src_bits=16), 1), (dict(dst_bits=0), 1), (dict(n=(1 << 30) + 1), 2),
    (dict(n=1 << 30), 2), (dict(src=(1 << 20) + 4096), 1), (dict(dst=(2 << 20) - 8), 1)])
def test_copy_refuses(kw, status):
    lib = q4.load_library()
    if kw == dict(n=1 << 30):
        kw = dict(n=1 << 30, src=1 << 40, dst=1 << 41)
    assert _copy(lib, _pool(), **kw) == status and lib.q4_last_error()
    assert _copy(lib, _pool(), src=None, dst=None, n=0) == 0
    assert _copy(lib, None) == 1


def _books(**kw):
    from gptq_bit_weight_amd.pages import _Pages
    a = dict(table=16 << 20, lengths=17 << 20, counts=18 << 20, work=19 << 20, requests=3, width=5, pages=8, page_size=16)
    a.update(kw)
    b = _Pages(*a.values())
    return b, ctypes.byref(b)


@pytest.mark.parametrize("books,status", [
    (dict(table=None), 1), (dict(lengths=None), 1), (dict(counts=None), 1), (dict(work=None), 1), (dict(requests=0), 1), (dict(width=0), 1),
    (dict(pages=0), 1), (dict(page_size=0), 1), (dict(requests=1 << 16, width=1 << 15), 2), (dict(width=1 << 16, page_size=1 << 15), 2),
    (dict(pages=1 << 20, page_size=1 << 11), 2)])
def test_books(books, status):
    lib = q4.load_library()
    b, ref = _books(**books)
    pool = _pool(pages=b.pages if b.pages > 0 else 1)
    assert lib.q4_pages_extend(ref, 8 << 20, 4, 9 << 20, None) == status and lib.q4_last_error()
    assert lib.q4_pages_fork(ref, ctypes.byref(pool), 8 << 20, 32, 9 << 20, 32, 2, 10 << 20, None) == status
    assert lib.q4_pages_free(ref, 8 << 20, 32, 2, None) == status
    assert lib.q4_pages_trim(ref, 4, 0, None) == status
    assert lib.q4_pages_compact(ref, ctypes.byref(pool), 10 << 20, None) == status


def test_pages_calls_refuse():
    lib = q4.load_library()
    _, ref = _books()
    pool, other = ctypes.byref(_pool()), ctypes.byref(_pool(pages=9))
    for status, st in [
            (1, lib.q4_pages_extend(ref, 8 << 20, -1, 9 << 20, None)), (1, lib.q4_pages_extend(ref, None, 1, 9 << 20, None)),
            (1, lib.q4_pages_extend(ref, 8 << 20, 1, None, None)), (2, lib.q4_pages_extend(ref, 8 << 20, (1 << 30) + 1, 9 << 20, None)),
            (1, lib.q4_pages_fork(ref, other, 8 << 20, 32, 9 << 20, 32, 2, 10 << 20, None)),
            (1, lib.q4_pages_fork(ref, pool, 8 << 20, 32, 9 << 20, 32, -1, 10 << 20, None)),
            (1, lib.q4_pages_fork(ref, pool, None, 32, 9 << 20, 32, 2, 10 << 20, None)),
            (1, lib.q4_pages_fork(ref, pool, 8 << 20, 32, 9 << 20, 8, 2, 10 << 20, None)),
            (1, lib.q4_pages_fork(ref, pool, 8 << 20, 32, 9 << 20, 32, 2, None, None)),
            (1, lib.q4_pages_free(ref, None, 32, 1, None)), (1, lib.q4_pages_free(ref, 8 << 20, 33, 1, None)),
            (1, lib.q4_pages_free(ref, 8 << 20, 32, -1, None)), (1, lib.q4_pages_trim(ref, 0, 0, None)), (1, lib.q4_pages_trim(ref, 3, -1, None)),
            (1, lib.q4_pages_compact(ref, other, 10 << 20, None)), (1, lib.q4_pages_compact(ref, pool, None, None))]:
        assert st == status
    assert lib.q4_pages_extend(ref, None, 0, None, None) == 0
    assert lib.q4_pages_fork(ref, pool, None, 32, None, 32, 0, None, None) == 0
    assert lib.q4_pages_free(ref, None, 32, 0, None) == 0
    assert lib.q4_pages_workspace(0, 4) == 0 and lib.q4_pages_workspace(4, 0) == 0
    assert lib.q4_pages_workspace(3, 8) == lib.q4_pages_workspace(8, 3) == 4 * (16 + 2 * 8)


def test_python_refuses_before_the_gpu():
    import torch
    codes, scales = torch.zeros(2, 1, 16, 16, dtype=torch.uint8), torch.zeros(2, 1, 16, 1, 2, dtype=torch.float16)
    for args, kind in [
            ((None, codes, scales, scales), TypeError), ((codes.int(), codes, scales, scales), ValueError), ((codes, codes, scales.float(), scales), ValueError),
            ((codes[0], codes, scales, scales), ValueError), ((codes, codes, scales[..., :1], scales), ValueError),
            ((codes[:, :0], codes, scales, scales), ValueError), ((codes, codes, scales, scales), ValueError)]:
        with pytest.raises(kind):
            q4.PagedCache4(*args)
    for a in ((2, 1, 16, 33), (2, 1, 16, 0), (2, 1, 16, 48)):
        with pytest.raises(ValueError):
            q4.PagedCache4.empty(*a, device="cpu")


@pytest.mark.parametrize("cache,meets", [
    (dict(v=1 << 20), True), (dict(v=(1 << 20) + 16), True), (dict(k_scale=2 << 20), True), (dict(v_scale=(3 << 20) + 4), True),
    (dict(v=(1 << 20) + 4096), False), (dict(v_scale=(3 << 20) + 1024), False),
    # rows of keys and of values in turn
    (dict(k_stride=(2048, 1024, 64), v_stride=(2048, 1024, 64), v=(1 << 20) + 32), False),
    (dict(k_stride=(2048, 1024, 64), v_stride=(2048, 1024, 64), v=(1 << 20) + 16), True)])
def test_tensors_that_overlap(cache, meets):
    lib = q4.load_library()
    assert lib.q4_check_cache4(ctypes.byref(_cache(**cache))) == (1 if meets else 0)
