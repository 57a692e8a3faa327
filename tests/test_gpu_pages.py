"""Pages of a cache on the GPU: copies, and the books against the same steps one
after the other on the host. Everything is whole numbers: results are equal."""
import random

import pytest

from tests.gpu_util import announce, torch_mod
from tests.pages_sim import Sim

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def filled(cache, seed=1):
    """Every byte of the cache random; copies of its tensors."""
    for t in cache._tensors:
        n = t.element_size()
        raw = torch.randint(0, 256, (*t.shape, n), generator=gen(seed), device="cuda", dtype=torch.uint8)
        t.copy_(raw.view(t.dtype)[..., 0] if n > 1 else raw[..., 0])
    return [t.clone() for t in cache._tensors]


def bits(t):
    return t.contiguous().view(torch.uint8)


def caches(kind):
    import gptq_bit_weight_amd as q4
    P = 37
    if kind == "16 bits":
        return q4.PagedCache(torch.empty(P, 3, 16, 64, dtype=F16, device="cuda"), torch.empty(P, 3, 16, 64, dtype=F16, device="cuda"))
    if kind == "16 bits, large pages":
        return q4.PagedCache(*torch.empty(2, P, 8, 64, 128, dtype=torch.bfloat16, device="cuda"))
    if kind == "16 bits, odd sizes":
        return q4.PagedCache(torch.empty(P, 3, 5, 7, dtype=F16, device="cuda"), torch.empty(P, 3, 5, 7, dtype=F16, device="cuda"))
    if kind == "16 bits, strided":
        base = torch.zeros(2, 16, P, 3, 80, dtype=F16, device="cuda")
        return q4.PagedCache(base[0, ..., :64].permute(1, 2, 0, 3), base[1, ..., 1:65].permute(1, 2, 0, 3))
    if kind == "16 bits, rows apart":
        base = torch.zeros(2, P, 3, 16, 72, dtype=F16, device="cuda")
        return q4.PagedCache(base[0, ..., :64], base[1, ..., 8:])
    return q4.PagedCache4.empty(P, 3, 16, 96 if kind == "4 bits, groups of 32" else 128,
                                group=32 if kind == "4 bits, groups of 32" else 128)


KINDS = ["16 bits", "16 bits, large pages", "16 bits, odd sizes", "16 bits, strided", "16 bits, rows apart", "4 bits, groups of 32", "4 bits"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src_t,dst_t", [(torch.int32, torch.int32), (torch.int64, torch.int32), (torch.int32, torch.int64)])
def test_copy(kind, src_t, dst_t):
    announce(f"copy_pages {kind} {src_t} {dst_t}")
    cache = caches(kind)
    before = filled(cache)
    order = torch.randperm(cache.pages, generator=gen(2), device="cuda").tolist()
    dst, src = order[:15], [order[20 + i % 9] for i in range(15)]
    src[3], dst[7] = -1, cache.pages
    src[11] = cache.pages + 5
    dst[12] = -3
    cache.copy_pages(ints(src, src_t), ints(dst, dst_t))
    for t, b in zip(cache._tensors, before):
        for s, d in zip(src, dst):
            if 0 <= s < cache.pages and 0 <= d < cache.pages:
                b[d] = b[s]
        assert torch.equal(bits(t), bits(b))
    cache.copy_pages(ints([], src_t), ints([], dst_t))
    cache.copy_pages(ints([4], src_t), ints([4], dst_t))
    for t, b in zip(cache._tensors, before):
        assert torch.equal(bits(t), bits(b))


def test_copy_many_pages():
    import gptq_bit_weight_amd as q4
    announce("copy_pages, 3000 pairs")
    cache = q4.PagedCache(*torch.empty(2, 6001, 2, 16, 64, dtype=F16, device="cuda"))
    before = filled(cache)
    order = torch.randperm(6001, generator=gen(2), device="cuda")
    cache.copy_pages(order[:3000], order[3000:6000])
    for t, b in zip(cache._tensors, before):
        b[order[3000:6000]] = b[order[:3000]]
        assert torch.equal(bits(t), bits(b))


class Both:
    """A Pages and the host's books, one step at a time."""

    def __init__(self, cache, requests, width, wide):
        import gptq_bit_weight_amd as q4
        self.pages, self.cache = q4.Pages(cache, requests, width), cache
        self.sim = Sim(requests, width, cache.pages, cache.page_size)
        self.start = filled(cache)
        self.t = torch.int64 if wide else torch.int32

    def check(self, what):
        s, p = self.sim, self.pages
        assert p.counts.tolist() == s.counts, what
        assert p.lengths.tolist() == s.lengths, what
        assert p.table.tolist() == s.table, what
        used = [i for i in range(s.P) if s.counts[i] > 0]
        for t, b in zip(self.cache._tensors, self.start):
            assert torch.equal(bits(t[ints(used).long()]), bits(b[ints([s.data[i] for i in used]).long()])), what

    def extend(self, news):
        starts = [0]
        for n in news:
            starts.append(starts[-1] + n)
        got = self.pages.extend(ints(starts), starts[-1]).tolist()
        assert got == self.sim.extend(starts, starts[-1])
        self.check(f"extend {news}")
        return got

    def fork(self, a, b):
        assert self.pages.fork(ints(a, self.t), ints(b, self.t)).tolist() == self.sim.fork(a, b), (a, b)
        self.check(f"fork {a} {b}")

    def free(self, a):
        self.pages.free(ints(a, self.t))
        self.sim.free(a)
        self.check(f"free {a}")

    def trim(self, window, sinks):
        self.pages.trim(window, sinks)
        self.sim.trim(window, sinks)
        self.check(f"trim {window} {sinks}")

    def compact(self):
        assert self.pages.compact().tolist() == self.sim.compact()
        self.check("compact")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wide", [False, True])
def test_steps(kind, wide):
    announce(f"pages {kind} wide={wide}")
    x = Both(caches(kind), 9, 12, wide)
    ps = x.cache.page_size
    x.extend([0, 3, 2 * ps, 0, ps + 1, 5, 1, 0, 0])
    x.extend([1] * 7 + [0, 0])
    x.free([5, 5, -1, 9, 5, 8])
    x.fork([2, 4, 4, 1, 7, 0, 11, 3], [5, 7, 7, 2, 8, 8, 3, -1])
    x.extend([0, ps, 1, 0, 3 * ps, 2, 0, 1, 0])
    x.trim(ps, 1)
    x.trim(1, 0)
    x.compact()
    x.compact()
    x.fork([4], [8])
    x.free(list(range(9)))
    x.compact()


def test_no_pages_left():
    """Requests are served in their order until the free pages run out."""
    x = Both(caches("16 bits"), 6, 30, False)
    x.extend([16 * 10, 0, 16 * 20, 0, 0, 0])
    x.extend([0, 0, 1, 16 * 7, 5, 16])           # 31 used of 37: request 3 does not fit, nor do those after it
    x.extend([0, 0, 1, 3, 2, 1])
    x.extend([0, 0, 16 * 30, 3, 2, 1])           # request 2's row is too short; the others take nothing new
    x.fork([3, 3, 3, 0], [1, 1, 5, 1])
    x.extend([0, 16 * 2, 15, 14, 0, 16])
    x.free([2])
    x.extend([1, 1, 1, 1, 1, 1])
    x.compact()


def test_starts_that_make_no_sense():
    x = Both(caches("16 bits"), 5, 8, False)
    starts = [3, 1, 9, 4, 200, 7]
    got = x.pages.extend(ints(starts), 20).tolist()
    x.sim.extend(starts, 20)
    x.check("starts out of order")
    assert all(-1 <= s < x.cache.pages * 16 for s in got)


@pytest.mark.parametrize("seed", range(6))
def test_random_steps(seed):
    import gptq_bit_weight_amd as q4
    rng = random.Random(seed)
    R, ps = rng.choice([3, 40, 1500]), rng.choice([1, 3, 16])
    P = rng.choice([50, 700, 9000])
    announce(f"pages random steps seed={seed} R={R} ps={ps} P={P}")
    cache = q4.PagedCache(*torch.empty(2, P, 1, ps, 8, dtype=F16, device="cuda"))
    x = Both(cache, R, 60, seed % 2)
    for _ in range(14):
        step = rng.choice(["extend", "extend", "fork", "free", "trim", "compact"])
        if step == "extend":
            x.extend([rng.choice([0, 0, 1, 1, 2, rng.randint(0, 9 * ps)]) for _ in range(R)])
        elif step == "fork":
            n = rng.randint(1, 2 * R + 2)
            x.fork([rng.randint(-1, R) for _ in range(n)], [rng.randint(-1, R) for _ in range(n)])
        elif step == "free":
            x.free([rng.randint(-1, R) for _ in range(rng.randint(1, R))])
        elif step == "trim":
            x.trim(rng.randint(1, 20 * ps), rng.randint(0, 3 * ps))
        else:
            x.compact()


def test_a_long_prompt():
    import gptq_bit_weight_amd as q4
    cache = q4.PagedCache(*torch.empty(2, 5000, 1, 16, 8, dtype=F16, device="cuda"))
    x = Both(cache, 4, 4000, False)
    x.extend([3, 40001, 2, 16 * 400])
    x.free([1])
    x.extend([30000, 0, 1, 1])
    x.compact()


def test_captured_steps():
    """A serving step as one graph: room, write, attention, drop; replayed with eager work between."""
    import gptq_bit_weight_amd as q4
    announce("pages captured")
    R, kv, H, D, ps = 5, 2, 4, 64, 16

    def serving():
        cache = q4.PagedCache4.empty(40, kv, ps, D, group=32)
        return cache, q4.Pages(cache, R, 20)

    graphed, eager = serving(), serving()
    starts = torch.arange(R + 1, device="cuda", dtype=torch.int32)
    rope = q4.Rotary(D)
    k, v, q = torch.zeros(R, kv, D, dtype=F16, device="cuda"), torch.zeros(R, kv, D, dtype=F16, device="cuda"), torch.zeros(R, H, D, dtype=F16, device="cuda")
    parent, child = ints([0]), ints([4])

    def step(cache, pages):
        positions = pages.lengths.clone()
        slots = pages.extend(starts, R)
        y = cache.append(k, v, slots, rotary=rope, positions=positions, q=q)
        o = cache.attend(y, starts, pages.lengths, pages.table, window=40, sinks=3)
        pages.trim(40, 3)
        pages.free(child)
        pages.fork(parent, child)
        to = pages.compact()
        return o, slots, to

    def data(seed):
        for i, t in enumerate((k, v, q)):
            t.copy_(torch.randn(t.shape, generator=gen(10 * seed + i), device="cuda"))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        data(0)
        step(*eager)                                 # (warms the stream's workspaces up)
    torch.cuda.synchronize()
    eager = serving()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step(*graphed)
    for i in range(60):
        data(i)
        want = step(*eager)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i
        for a, b in zip(graphed[1]._tensors[:3] + graphed[0]._tensors, eager[1]._tensors[:3] + eager[0]._tensors):
            assert torch.equal(a, b), i
    assert graphed[1].lengths.tolist()[:4] == [60] * 4 and (graphed[1].counts > 0).sum() < 40


def test_another_stream_and_refusals():
    import gptq_bit_weight_amd as q4
    cache = caches("16 bits")
    pages = q4.Pages(cache, 3, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    slots = pages.extend(ints([0, 5, 5, 30]), 30, stream=s)
    done = pages.fork(ints([2]), ints([1]), stream=s)
    pages.free(ints([0]), stream=s)
    pages.trim(9, 0, stream=s)
    to = pages.compact(stream=s)
    cache.copy_pages(ints([0]), ints([36]), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert slots.tolist()[:5] == [0, 1, 2, 3, 4] and done.tolist() == [1] and pages.lengths.tolist() == [0, 25, 25]
    assert sorted(t for t in to.tolist() if t >= 0) == list(range(int((pages.counts > 0).sum())))
    for bad in (lambda: pages.fork(ints([0, 1]), ints([1])), lambda: pages.free(ints([[0]])), lambda: pages.free(ints([0]).cpu()),
                lambda: pages.free(ints([0]).float()), lambda: pages.trim(0), lambda: pages.trim(4, -1), lambda: pages.extend(ints([0, 1]), 1),
                lambda: pages.extend(ints([0, 1, 1, 1]), -1), lambda: cache.copy_pages(ints([0]), ints([0, 1])), lambda: q4.Pages(cache, 0, 3)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        q4.Pages(None, 1, 1)
    assert pages.extend(ints([0, 0, 0, 0]), 0).shape == (0,)
    assert pages.fork(ints([]), ints([])).shape == (0,)
    pages.free(ints([]))
    with torch.inference_mode():
        inner = q4.Pages(q4.PagedCache4.empty(3, 1, 16, 32), 2, 2)
        inner.extend(ints([0, 3, 4]), 4)
        inner.fork(ints([0]), ints([1]))
        inner.compact()
    with pytest.raises(ValueError, match="gradient"):
        grown = torch.zeros(3, 1, 16, 8, dtype=F16, device="cuda", requires_grad=True)
        q4.PagedCache(grown, grown.detach().clone()).copy_pages(ints([0]), ints([1]))
