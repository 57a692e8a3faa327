"""Attention of more rows than one launch has workgroups for is refused."""
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


@pytest.mark.parametrize("four", [False, True])
def test_units(four):
    """2^21 tokens of 1024 heads of one request, by a stride of 0: 2^24 units of 128 rows, 2^32 lanes. (Refused by the host.)"""
    import gptq_bit_weight_amd as q4
    announce(f"attend 2^24 units four={four}")
    H, D = 1024, 32
    lib = q4.load_library()
    cache = q4.PagedCache4.empty(1, H, 16, D) if four else q4.PagedCache(*torch.zeros(2, 1, H, 16, D, dtype=torch.float16, device="cuda"))
    q, out = (torch.zeros(H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    need = (lib.q4_attend4_workspace if four else lib.q4_attend_workspace)(cache._ref, H)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")

    def call(tokens):
        starts, lengths = torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), torch.tensor([16], dtype=torch.int32, device="cuda")
        args = [cache._ref, q.data_ptr(), 0, D, H, tokens, starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), 1, 1, 1, 0]
        end = [D ** -0.5, out.data_ptr(), 0, D, ws.data_ptr(), need]
        s = torch.cuda.current_stream().cuda_stream
        return lib.q4_attend4(*args, 0, *end, 0, s) if four else lib.q4_attend(*args, *end, s)

    for tokens in (1 << 21, (1 << 21) + 12345):
        assert call(tokens) == 2 and b"2^24" in lib.q4_last_error()
