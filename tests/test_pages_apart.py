"""The books of a cache's pages, a call's indexes and its output lie apart: what overlaps is refused before
any GPU call. (Each call here is refused, for that or later on for its size: nothing is launched.)"""
import ctypes

import pytest

import gptq_bit_weight_amd as q4

MB = 1 << 20
# 3 requests of 5 pages, 8 pages of 16 rows: 60, 12 and 32 bytes, and 4 * (16 + 2 * 8) of scratch
TABLE, LENGTHS, COUNTS, WORK = 16 * MB, 17 * MB, 18 * MB, 19 * MB
ENDS = [(TABLE, 60), (LENGTHS, 12), (COUNTS, 32), (WORK, 128)]


def books(**kw):
    from gptq_bit_weight_amd.pages import _Pages
    a = dict(table=TABLE, lengths=LENGTHS, counts=COUNTS, work=WORK, requests=3, width=5, pages=8, page_size=16)
    a.update(kw)
    b = _Pages(*a.values())
    return b, ctypes.byref(b)


def pool(**kw):
    """Two planes of 8 pages of 2 heads of 16 rows of 128 bytes at 1 and 2 MiB."""
    from gptq_bit_weight_amd.attention import _Pool
    p = _Pool()
    for i in range(2):
        x = p.plane[i]
        x.at, x.page, x.head, x.row, x.heads, x.rows, x.bytes = (i + 1) * MB, 4096, 2048, 128, 2, 16, 128
    p.planes, p.pages = 2, kw.get("pages", 8)
    return ctypes.byref(p)


def refused(st, meets=True):
    assert st != 0
    assert (b"overlap" in q4.load_library().q4_last_error()) == meets and (st == 1 or not meets)


@pytest.mark.parametrize("at,size", ENDS)
@pytest.mark.parametrize("low", [False, True])
def test_indexes_and_outputs(at, size, low):
    lib, (_, ref) = q4.load_library(), books()
    edge = lambda n: at - n + 4 if low else at + size - 4       # noqa: E731 (n bytes that share four with the array)
    far = 8 * MB
    refused(lib.q4_pages_extend(ref, edge(16), 6, far, None))
    refused(lib.q4_pages_extend(ref, far, 6, edge(24), None))
    refused(lib.q4_pages_fork(ref, pool(), edge(8), 32, far, 32, 2, far + 64, None))
    refused(lib.q4_pages_fork(ref, pool(), far, 32, edge(16), 64, 2, far + 64, None))
    refused(lib.q4_pages_fork(ref, pool(), far, 32, far + 64, 32, 2, edge(16), None))
    refused(lib.q4_pages_free(ref, edge(8), 32, 2, None))
    refused(lib.q4_pages_free(ref, edge(16), 64, 2, None))
    refused(lib.q4_pages_compact(ref, pool(), edge(32), None))


@pytest.mark.parametrize("at", [MB, 2 * MB])
def test_what_lies_in_the_cache(at):
    lib, (_, ref), far = q4.load_library(), books(), 8 * MB
    for x in (at + 4096 * 3 + 64, at + 8 * 4096 - 4):
        refused(lib.q4_pages_fork(ref, pool(), x, 32, far, 32, 2, far + 64, None))
        refused(lib.q4_pages_fork(ref, pool(), far, 32, x, 32, 2, far + 64, None))
        refused(lib.q4_pages_fork(ref, pool(), far, 32, far + 64, 32, 2, x, None))
        refused(lib.q4_pages_compact(ref, pool(), x, None))
        for name in ("table", "lengths", "counts", "work"):
            inside = books(**{name: x})[1]
            refused(lib.q4_pages_fork(inside, pool(), far, 32, far + 64, 32, 2, far + 128, None))
            refused(lib.q4_pages_compact(inside, pool(), far, None))


def test_indexes_in_the_output():
    lib, (_, ref), far = q4.load_library(), books(), 8 * MB
    refused(lib.q4_pages_extend(ref, far, 6, far + 12, None))
    refused(lib.q4_pages_extend(ref, far + 20, 6, far, None))
    # (done has room for 2 n values)
    refused(lib.q4_pages_fork(ref, pool(), far + 12, 32, far + 64, 32, 2, far, None))
    refused(lib.q4_pages_fork(ref, pool(), far + 64, 32, far + 12, 32, 2, far, None))


@pytest.mark.parametrize("kw", [dict(lengths=TABLE), dict(lengths=TABLE + 56), dict(counts=LENGTHS + 8), dict(work=COUNTS - 124), dict(table=WORK + 124),
                                dict(work=LENGTHS - 124)])
def test_books_in_each_other(kw):
    lib, (_, ref), far = q4.load_library(), books(**kw), 8 * MB
    refused(lib.q4_pages_extend(ref, far, 6, far + 64, None))
    refused(lib.q4_pages_fork(ref, pool(), far, 32, far + 64, 32, 2, far + 128, None))
    refused(lib.q4_pages_free(ref, far, 32, 2, None))
    refused(lib.q4_pages_trim(ref, 3, 0, None))
    refused(lib.q4_pages_compact(ref, pool(), far, None))


def test_neighbours_are_not_refused():
    """Side by side is apart. (2^30 pairs of two pieces, or as many pages, are too many for a launch.)"""
    lib, n, far = q4.load_library(), 1 << 30, 1 << 43       # (2^30 pages of the cache end at 2^42)
    at = far // 2                       # (far from the cache, which begins at 1 MiB)
    _, ref = books(table=at, lengths=at + 60, counts=at + 72, work=at + 104)
    refused(lib.q4_pages_fork(ref, pool(), at + 232, 32, far, 32, n, 2 * far, None), False)
    refused(lib.q4_pages_fork(ref, pool(), far, 32, at - 4 * n, 32, n, 2 * far, None), False)
    refused(lib.q4_pages_fork(ref, pool(), far, 32, far, 64, n, far + 8 * n, None), False)
    refused(lib.q4_pages_fork(ref, pool(), far + 8 * n, 32, far - 4 * n, 32, n, far, None), False)
    _, wide = books(pages=n, page_size=1)
    refused(lib.q4_pages_compact(wide, pool(pages=n), far, None))       # (the cache reaches the books)
    _, wide = books(table=far, lengths=far + 60, counts=far + 72, work=far + 72 + 4 * n, pages=n, page_size=1)
    refused(lib.q4_pages_compact(wide, pool(pages=n), 2 * far, None), False)
