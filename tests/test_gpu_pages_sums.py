"""Requests whose length and new tokens together pass 2^31 get nothing, and hold nobody up."""
import pytest

from tests.gpu_util import announce, torch_mod

torch = torch_mod()
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


def test_length_and_tokens_past_31_bits():
    import gptq_bit_weight_amd as q4
    announce("extend by 2^30 tokens of a request that is full")
    ps = 1 << 26
    # (a page of 2^26 rows of 8 values of one head: 1 GiB)
    cache = q4.PagedCache(*torch.zeros(2, 2, 1, ps, 8, dtype=torch.float16, device="cuda"))
    p = q4.Pages(cache, 3, 16)
    p.lengths[1] = 1 << 30                      # its 16 pages name none: as after trim()
    slots = p.extend(torch.tensor([0, 2, (1 << 30) - 3, 1 << 30], dtype=torch.int32, device="cuda"), 1 << 30)
    assert slots[:2].tolist() == [0, 1] and slots[-3:].tolist() == [ps, ps + 1, ps + 2]
    assert int((slots >= 0).sum()) == 5 and p.lengths.tolist() == [2, 1 << 30, 3] and p.counts.tolist() == [1, 1]
