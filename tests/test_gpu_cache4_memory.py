"""The scratch that long chunks over 4 bits are faster with: what a call does where there is no memory for it."""
import pytest

from tests.cache4_util import attention, rows_of
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_attend import check
from tests.test_gpu_cache4 import make, pools

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


def wide_call(dt, seed):
    """640 tokens over 1000 keys by a table of 131072 rows: 512 MiB of scratch."""
    H, kv, D, ps, news, lens = 32, 8, 128, 16, [640], [1000]
    q, cache, starts, lengths, table = make(dt, H, kv, D, 32, ps, news, lens, seed=seed)
    wide = torch.full((1, 131072 // ps), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    k, v = (rows_of(x, table, lens) for x in pools(cache))
    return (q, starts, lengths, wide), cache, attention(q, k, v, news, lens, 0, 0, None, F16)


@pytest.fixture
def little_memory():
    """No more than 256 MiB beyond what is in use."""
    from gptq_bit_weight_amd import attention
    attention._refused.clear()

    def limit():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        total = torch.cuda.get_device_properties(0).total_memory
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (256 << 20)) / total)
    yield limit
    torch.cuda.set_per_process_memory_fraction(1.0)
    attention._refused.clear()


@pytest.mark.parametrize("dt", [F16, BF16])
def test_no_memory_for_the_scratch(dt, little_memory):
    """Without it every workgroup unpacks for itself: the same result."""
    announce(f"attend4 long chunk without memory for its scratch {dt}")
    args, cache, want = wide_call(dt, 1)
    s = torch.cuda.Stream()                     # (a stream that holds none yet)
    s.wait_stream(torch.cuda.current_stream())
    little_memory()
    for _ in range(3):
        y = cache.attend(*args, stream=s)
        s.synchronize()
        check(y, *want)
    # a short call on that stream
    short = (args[0][:3], torch.tensor([0, 3], dtype=torch.int32, device="cuda")) + args[2:]
    torch.cuda.synchronize()
    a = cache.attend(*short, stream=s)
    s.synchronize()
    k, v = (rows_of(x, args[3], [1000]) for x in pools(cache))
    check(a, *attention(args[0][:3], k, v, [3], [1000], 0, 0, None, F16))


def test_a_size_without_memory_is_asked_for_once(little_memory, monkeypatch):
    from gptq_bit_weight_amd import attention
    announce("attend4 long chunk without memory, three times")
    args, cache, want = wide_call(F16, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    asked, new = [], attention._new_workspace
    monkeypatch.setattr(attention, "_new_workspace", lambda n, d: asked.append(n) or new(n, d))
    little_memory()
    for _ in range(3):
        y = cache.attend(*args, stream=s)
        s.synchronize()
        check(y, *want)
    assert len([n for n in asked if n > 512 << 20]) == 1


def test_a_large_scratch_is_not_held():
    """After the call its memory is the allocator's again; what a stream holds is 64 MiB more than any call needs, at most."""
    import gptq_bit_weight_amd as q4
    announce("attend4 long chunk: what a stream holds after it")
    args, cache, want = wide_call(BF16, 3)
    least = q4.load_library().q4_attend4_workspace(cache._ref, 32)
    narrow = args[:3] + (args[3][:, :2048 // 16].contiguous(),)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for call in (args, narrow, args, narrow):
        before = torch.cuda.memory_allocated()
        y = cache.attend(*call, stream=s)
        s.synchronize()
        check(y, *want)
        del y
        assert torch.cuda.memory_allocated() - before <= (least if call is args else least + (64 << 20)) + 4096
