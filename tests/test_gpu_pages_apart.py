"""Books, indexes and outputs of Pages that lie in each other are refused; neighbours are not."""
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
def test_lists_that_are_the_books_or_the_cache(four):
    import gptq_bit_weight_amd as q4
    announce(f"pages: lists in the books, four={four}")
    cache = q4.PagedCache4.empty(9, 2, 16, 64) if four else q4.PagedCache(*torch.zeros(2, 9, 2, 16, 64, dtype=torch.float16, device="cuda"))
    p = q4.Pages(cache, 4, 5)
    near = torch.zeros(64, dtype=torch.int32, device="cuda")
    near[0:5] = torch.tensor([0, 20, 20, 20, 20])
    assert p.extend(near[:5], 20).tolist() == list(range(20))
    inside = cache.k.view(torch.int32).flatten()
    mine = [p.table[0], p.lengths, p.counts[:4]]
    before = [t.clone() for t in p._tensors[:3] + cache._tensors]
    for bad in mine:
        for call in (lambda: p.free(bad[:2]), lambda: p.fork(bad[:2], near[:2]), lambda: p.fork(near[:2], bad[:2])):
            with pytest.raises(ValueError, match="overlap"):
                call()
    for call in (lambda: p.fork(inside[:2], near[:2]), lambda: p.fork(near[:2], inside[:2]), lambda: p.extend(p.table.flatten()[:5], 3),
                 lambda: p.extend(p.counts[:5], 3)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    for t, b in zip(p._tensors[:3] + cache._tensors, before):
        assert torch.equal(t, b)
    # both lists one tensor, and lists side by side
    near[:4] = torch.tensor([0, 0, 1, 2])
    assert p.fork(near[1:2], near[2:3]).tolist() == [1] and p.fork(near[3:4], near[3:4]).tolist() == [1]
    p.free(near[2:3])
    assert p.lengths.tolist() == [20, 0, 0, 0] and p.counts.tolist() == [1, 1] + [0] * 7
