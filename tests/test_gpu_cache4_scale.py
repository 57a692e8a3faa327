"""Attention over 4 bits where a row's power of two and the scale leave fp32's range together. The
tolerance is that of test_gpu_cache4.py: nothing of it hangs on the scale's size."""
import pytest

from tests.cache4_util import attention, rows_of
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_attend import check
from tests.test_gpu_cache4 import make, pools

torch = torch_mod()
pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16

# few rows, many, and as many as have the keys and values brought into binary16 first
CALLS = [([1, 1, 3], [300, 5, 70]), ([60, 9, 130], [300, 9, 400]), ([700], [900])]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


def compare(q, cache, starts, lengths, table, news, lens, scale, **kw):
    got = cache.attend(q, starts, lengths, table, scale=scale, **kw)
    k, v = (rows_of(x, table, lens) for x in pools(cache))
    check(got, *attention(q, k, v, news, lens, kw.get("window", 0), kw.get("sinks", 0), scale, F16))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news,lens", CALLS)
@pytest.mark.parametrize("ps", [16, 7])
def test_small_scales(dt, D, news, lens, ps):
    """Rows of zeros and of least values, whose scores are all but alike: a row is its values' mean."""
    announce(f"attend4 small scales {dt} D={D} news={news} ps={ps}")
    q, cache, *rest = make(dt, 8, 2, D, 32, ps, news, lens, seed=D)
    q[0] = 0
    q[-1, ::2] = 0
    q[1, 1] *= torch.finfo(dt).smallest_normal
    q[-1, 1] *= 2.0 ** -110 if dt is BF16 else 2.0 ** -14
    for scale in (1e-9, -1e-20, 2.0 ** -126, 1e-38):
        compare(q, cache, *rest, news, lens, scale)
        compare(q, cache, *rest, news, lens, scale, window=40, sinks=3)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("news,lens", CALLS)
def test_scores_of_zero_under_a_large_scale(dt, news, lens):
    """Large queries that meet only keys of zero."""
    announce(f"attend4 large scale {dt} news={news}")
    q, cache, starts, lengths, table = make(dt, 8, 2, 128, 32, 16, news, lens, seed=3)
    q[..., 32:] = 0
    q[..., :32] = q[..., :32].sign() * torch.finfo(dt).max / 4
    cache.k_scale[..., 0, :] = 0
    for scale in (2.0 ** 20, -2.0 ** 100, 3e38):
        compare(q, cache, starts, lengths, table, news, lens, scale)
        compare(q, cache, starts, lengths, table, news, lens, scale, window=40, sinks=3)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("news,lens", CALLS)
def test_the_largest_scale_over_16_bits(dt, news, lens):
    """Queries of zero: every score is 0, a row is its values' mean."""
    import gptq_bit_weight_amd as q4
    from tests.test_gpu_attend import reference
    announce(f"attend largest scale {dt} news={news}")
    q, cache4, starts, lengths, table = make(dt, 8, 2, 128, 32, 16, news, lens, seed=3)
    k, v = (x.nan_to_num(0.25).to(dt) for x in pools(cache4))
    q.zero_()
    for kw in (dict(), dict(window=40)):
        ref, tol = reference(q, k, v, news, lens, table.cpu(), scale=3e38, **kw)
        check(q4.PagedCache(k, v).attend(q, starts, lengths, table, scale=3e38, **kw), ref, tol)
