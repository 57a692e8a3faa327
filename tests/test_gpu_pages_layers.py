"""Layers that share one table: heads of one pool, a cache on each layer's slice, books over the whole.
Every layer then holds and gives, bit for bit, what it would with a pool and books of its own."""
import pytest

from tests.gpu_util import announce, torch_mod

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def empty(four, pages, heads, ps, D):
    import gptq_bit_weight_amd as q4
    return q4.PagedCache4.empty(pages, heads, ps, D) if four else q4.PagedCache(*torch.zeros(2, pages, heads, ps, D, dtype=F16, device="cuda"))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("ps", [16, 5])
def test_layers(four, ps):
    import gptq_bit_weight_amd as q4
    announce(f"pages of three layers four={four} ps={ps}")
    L, kv, H, D, P, R, W = 3, 2, 4, 64, 60, 5, 12
    whole = empty(four, P, L * kv, ps, D)
    layers = [type(whole)(*(t[:, i * kv:(i + 1) * kv] for t in whole._tensors)) for i in range(L)]
    books = q4.Pages(whole, R, W)
    alone = [empty(four, P, kv, ps, D) for _ in range(L)]
    apart = [q4.Pages(c, R, W) for c in alone]
    rope, seed = q4.Rotary(D), [0]

    def both(f):
        first = f(books)
        rest = [f(p) for p in apart]
        assert first is None or all(torch.equal(first, x) for x in rest)
        return first

    def tokens(news):
        starts = ints([0] + torch.tensor(news).cumsum(0).tolist())
        T = sum(news)
        at = books.lengths.clone()
        slots = both(lambda p: p.extend(starts, T))
        of = torch.repeat_interleave(torch.arange(R), torch.tensor(news)).cuda()
        positions = (at[of] + torch.arange(T, device="cuda") - starts[of]).int()
        for a, b, x in zip(layers, alone, apart):
            g = torch.Generator(device="cuda").manual_seed(seed[0])
            seed[0] += 1
            q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").half() for h in (H, kv, kv))
            y = a.append(k, v, slots, rotary=rope, positions=positions, q=q)
            assert torch.equal(y, b.append(k, v, slots, rotary=rope, positions=positions, q=q))
            assert torch.equal(a.attend(y, starts, books.lengths, books.table, window=30, sinks=2),
                               b.attend(y, starts, x.lengths, x.table, window=30, sinks=2))

    tokens([20, 0, 7, 0, 3])
    assert both(lambda p: p.fork(ints([0, 2]), ints([1, 3]))).tolist() == [1, 1]
    tokens([1, 1, 9, 1, 1])
    both(lambda p: p.trim(30, 2))
    both(lambda p: p.free(ints([2])))
    both(lambda p: p.compact())
    tokens([3, 2, 18, 1, 1])
    for a, b in zip(layers, alone):
        for s, t in zip(a._tensors, b._tensors):
            used = books.counts > 0
            assert torch.equal(s[used], t[used])
