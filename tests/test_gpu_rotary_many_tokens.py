"""Rotations of, and appends of, more tokens than one launch has lanes for."""
import pytest

from tests.gpu_util import announce, torch_mod

torch = torch_mod()
pytestmark = pytest.mark.gpu
F16 = torch.float16
T, PART = 68_000_003, 1 << 23       # (4 tokens of a workgroup of 256: 2^32 lanes at 2^26 tokens)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


def values(seed, heads=1):
    return torch.randn(T, heads, 8, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=F16)


def parts():
    return [slice(i, min(i + PART, T)) for i in range(0, T, PART)]


@pytest.mark.parametrize("transpose", [False, True])
def test_rotate(transpose):
    import gptq_bit_weight_amd as q4
    announce(f"rotate {T} tokens transpose={transpose}")
    rope, x, positions = q4.Rotary(8), values(1), torch.arange(T, device="cuda")
    y = rope.rotate(x, positions, transpose=transpose)
    for s in parts():
        assert torch.equal(y[s], rope.rotate(x[s], positions[s], transpose=transpose)), s


def test_append():
    import gptq_bit_weight_amd as q4
    announce(f"append {T} tokens")
    rope, k, v, q, positions = q4.Rotary(8), values(1), values(2), values(3), torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.full((T,), -1, device="cuda")
    at = torch.tensor([0, 1, 2 ** 24, 2 ** 25 + 3, 2 ** 26 - 1, 2 ** 26, T - 1], device="cuda")
    slots[at] = torch.arange(len(at), device="cuda") * 5
    cache = q4.PagedCache(*torch.zeros(2, 3, 1, 16, 8, dtype=F16, device="cuda"))
    y = cache.append(k, v, slots, rotary=rope, positions=positions, q=q)
    for s in parts():
        assert torch.equal(y[s], rope.rotate(q[s], positions[s])), s
    rows = lambda t: t.transpose(1, 2).reshape(48, 1, 8)[slots[at]]      # noqa: E731
    assert torch.equal(rows(cache.k), rope.rotate(k[at], positions[at])) and torch.equal(rows(cache.v), v[at])
