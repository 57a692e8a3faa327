"""Pages of a 4-bit cache that no token sees are not read where long chunks have their keys and values
brought into binary16: nothing of them is found in the call's workspace."""
import pytest

from tests.cache4_util import attention, rows_of
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_attend import check
from tests.test_gpu_cache4 import make, pools

torch = torch_mod()
pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
MARK = 28.40625         # what every value of an unseen page stands for; the others are other values


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("ps", [1, 7, 16, 64])
@pytest.mark.parametrize("news,lens,window,sinks", [
    ([700], [1500], 300, 0), ([700, 900], [1531, 1222], 170, 37), ([700], [1500], 333, 130), ([640], [3000], 1, 1), ([800, 700], [800, 2000], 100, 5),
    ([700], [710], 4000, 9)])
def test_unseen_pages(dt, ps, news, lens, window, sinks):
    import gptq_bit_weight_amd as q4
    announce(f"attend4 unseen pages {dt} ps={ps} news={news} lens={lens} window={window} sinks={sinks}")
    H, kv, D = 8, 2, 64
    lib = q4.load_library()
    q, cache, starts, lengths, table = make(dt, H, kv, D, 32, ps, news, lens, seed=ps + sinks)
    k, v = (rows_of(x, table, lens) for x in pools(cache))
    seen = torch.zeros(cache.pages, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(news, lens)):
        j = torch.arange(m)
        j = j[(j < sinks) | (j > m - n - window)]
        seen[table[b].cpu().long()[j // ps]] = True
    for x in (cache.k_scale, cache.v_scale):
        x[~seen.cuda()] = torch.tensor([0.0, MARK], dtype=F16, device="cuda")
    size = lib.q4_attend4_workspace_for(cache._ref, H, q.shape[0], len(news), table.shape[1])
    assert size > lib.q4_attend4_workspace(cache._ref, H)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    st = lib.q4_attend4(cache._ref, q.data_ptr(), q.stride(0), q.stride(1), H, q.shape[0], starts.data_ptr(), lengths.data_ptr(), table.data_ptr(),
                        table.shape[1], table.stride(0), len(news), window, sinks, D ** -0.5, out.data_ptr(), out.stride(0), out.stride(1),
                        ws.data_ptr(), size, int(dt is BF16), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    check(out, *attention(q, k, v, news, lens, window, sinks, None, F16))
    mark = int(torch.tensor(MARK, dtype=F16).view(torch.int16))
    # (eight values of a row and more, one after the other)
    held = (ws[:size // 16 * 16].view(torch.int16).view(-1, 8) == mark).all(-1)
    assert not held.any(), f"{int(held.sum())} pieces of unseen pages"
