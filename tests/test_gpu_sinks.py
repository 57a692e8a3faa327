"""Attention with a window and sinks over the 16-bit cache, against the
definition in 64 bits (tolerances: test_gpu_attend.py)."""
import math

import pytest

from tests.cache4_util import attention, rows_of
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_attend import check, make

torch = torch_mod()
pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


def run(dt, H, kv, D, ps, news, lens, window, sinks, seed=0):
    import gptq_bit_weight_amd as q4
    announce(f"sinks {dt} H={H} kv={kv} D={D} ps={ps} news={news[:8]} lens={lens[:8]} window={window} sinks={sinks}")
    q, kc, vc, starts, lengths, table = make(dt, H, kv, D, ps, news, lens, seed)
    cache = q4.PagedCache(kc, vc)
    y = cache.attend(q, starts, lengths, table, window=window, sinks=sinks)
    k, v = (rows_of(x, table, lens) for x in (kc, vc))
    check(y, *attention(q, k, v, news, lens, window, sinks))
    # entries between the sinks and the window name no page, keys there are not finite
    if window:
        for b, (n, m) in enumerate(zip(news, lens)):
            lo = max(0, m - n - window + 1)
            for e in range(-(-sinks // ps), lo // ps):
                page = int(table[b, e])
                kc[page], vc[page] = math.nan, math.inf
                table[b, e] = -1
        assert torch.equal(y, cache.attend(q, starts, lengths, table, window=window, sinks=sinks))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 0), (2, 100), (31, 4), (32, 32), (33, 40), (64, 100), (100, 16), (1000, 4), (200, 64),
                                          (17, 1000), (60, 128)])
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64), (256, 32), (80, 16), (128, 9)])
def test_windows_and_sinks(dt, window, sinks, D, ps):
    run(dt, 4, 2, D, ps, [1, 1, 1, 1], [300, 5, 1333, 40], window, sinks, seed=window)
    run(dt, 4, 2, D, ps, [1, 1, 40, 7, 130], [300, 5, 333, 7, 450], window, sinks, seed=window)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D", [(16, 1, 128), (2, 2, 64), (4, 2, 256)])
def test_long(dt, H, kv, D):
    run(dt, H, kv, D, 64, [1], [40001], 20000, 70, seed=3)
    run(dt, H, kv, D, 16, [300, 1, 40], [9000, 4000, 60], 3000, 5, seed=4)
    run(dt, H, kv, D, 16, [700], [9000], 300, 200, seed=5)


def test_every_sink_and_window_near_the_edges():
    lens = list(range(1, 140, 3))
    for sinks in (1, 15, 16, 17, 33):
        run(F16, 4, 2, 64, 16, [1] * len(lens), lens, 17, sinks, seed=1)
        run(BF16, 4, 2, 128, 64, [min(m, 30) for m in lens], lens, 3, sinks, seed=2)
        run(BF16, 4, 2, 64, 7, [min(m, 30) for m in lens], lens, 20, sinks, seed=2)


def test_sinks_without_a_window_and_huge_ones():
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(F16, 4, 2, 64, 16, [1, 50], [90, 200])
    cache = q4.PagedCache(kc, vc)
    plain = cache.attend(q, starts, lengths, table)
    for w, s in ((0, 7), (2 ** 40, 7), (5, 2 ** 31 - 1), (1, 2 ** 40), (5, 200)):
        assert torch.equal(plain, cache.attend(q, starts, lengths, table, window=w, sinks=s)), (w, s)
    with pytest.raises(ValueError, match="negative"):
        cache.attend(q, starts, lengths, table, window=5, sinks=-1)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("news,lens", [([1, 1], [300, 130]), ([60, 9], [300, 130])])
def test_what_is_not_finite_reaches_only_those_who_see_it(dt, news, lens):
    """Keys and values between the sinks and the window, in tiles that hold visible ones too."""
    import gptq_bit_weight_amd as q4
    window, sinks, ps = 50, 5, 16
    q, kc, vc, starts, lengths, table = make(dt, 4, 2, 64, ps, news, lens, seed=4)
    cache = q4.PagedCache(kc, vc)
    for b, (n, m) in enumerate(zip(news, lens)):
        for j in range(sinks, m - n - window + 1):
            page, row = int(table[b, j // ps]), j % ps
            kc[page, :, row], vc[page, :, row] = math.nan, -math.inf
    got = cache.attend(q, starts, lengths, table, window=window, sinks=sinks)
    k, v = (rows_of(x, table, lens) for x in (kc, vc))
    check(got, *attention(q, k, v, news, lens, window, sinks))
    assert got.isfinite().all()
