"""An append to a 4-bit cache of tens of millions of tokens at once."""
import pytest

from tests.cache4_util import turned
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_cache4 import check_rows, gen

torch = torch_mod()
pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


@pytest.mark.parametrize("queries", [False, True])
def test_many_tokens(queries):
    import gptq_bit_weight_amd as q4
    T, kv, D, ps = 34_000_003, 1, 32, 64
    announce(f"append4 of {T} tokens queries={queries}")
    k = torch.randn(T, kv, D, generator=gen(1), device="cuda", dtype=F16)
    v = torch.randn(T, kv, D, generator=gen(2), device="cuda", dtype=F16)
    at = torch.tensor([0, 1, 2 ** 22 - 1, 2 ** 22, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, 22_369_622, 2 ** 25 - 1, 2 ** 25, 33_000_000, T - 2, T - 1], device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[at] = torch.arange(len(at), device="cuda", dtype=torch.int32) * 3
    positions = torch.arange(T, device="cuda", dtype=torch.int32)
    cache = q4.PagedCache4.empty(2, kv, ps, D)
    if not queries:
        cache.append(k, v, slots)
        check_rows(cache, slots[at], k[at], v[at])
        return
    rope = q4.Rotary(D)
    q = torch.randn(T, 1, D, generator=gen(3), device="cuda", dtype=F16)
    y = cache.append(k, v, slots, rotary=rope, positions=positions, q=q)
    check_rows(cache, slots[at], turned(k[at], positions[at], D, "half"), v[at])
    assert torch.equal(y, rope.rotate(q, positions))
