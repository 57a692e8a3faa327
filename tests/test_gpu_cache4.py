"""The cache held in 4 bits on the GPU: codes against the definition in 64 bits,
exactly, and attention over what it stands for.

Tolerances of attention are those derived in test_gpu_attend.py, with the weights rounded
to binary16 whatever the type of the queries. Queries of bfloat16 become binary16 times a
power of two: exact for values above 2^-31 of their row's largest, which adds nothing above the 2^-18 there."""
import math

import pytest

from tests.cache4_util import attention, quantise, rows_of, turned, unpack, values
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_attend import check

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def same(a, b, what):
    eq = (a == b) | (a.isnan() & b.isnan())
    if not eq.all():
        i = tuple((~eq).nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int((~eq).sum())} of {eq.numel()} differ, first {i}: {a[i].item()} against {b[i].item()}")


def held(cache, slots, side):
    """Codes, steps, least values of rows `slots` as they lie in memory (float64)."""
    codes, scales = (cache.k, cache.k_scale) if side == "k" else (cache.v, cache.v_scale)
    page, row = slots.long() // cache.page_size, slots.long() % cache.page_size
    sc = scales[page, :, row].double()
    return unpack(codes[page, :, row]).double(), sc[..., 0], sc[..., 1]


def check_rows(cache, slots, k, v, what=""):
    for side, x in (("k", k), ("v", v)):
        want = quantise(x, cache.group)
        for a, b, name in zip(held(cache, slots, side), want, ("codes", "steps", "least values")):
            same(a, b, f"{what} {side} {name}")
    for x, y in zip(cache.read(slots), (k, v)):
        same(x.double(), values(*quantise(y, cache.group)), f"{what} read")


def tokens(dt, T, heads, D, seed, spread=1.0):
    return (torch.randn(T, heads, D, generator=gen(seed), device="cuda") * spread).to(dt)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D,G", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 64), (160, 32),
                                 (256, 256), (256, 32)])
@pytest.mark.parametrize("T,kv,ps", [(1, 1, 16), (7, 3, 5), (65, 2, 16), (1030, 8, 64)])
def test_codes(dt, D, G, T, kv, ps):
    import gptq_bit_weight_amd as q4
    announce(f"append4 {dt} D={D} G={G} T={T} kv={kv} ps={ps}")
    pages = -(-T // ps) + 2
    cache = q4.PagedCache4.empty(pages, kv, ps, D, group=G)
    k, v = tokens(dt, T, kv, D, T + D), tokens(dt, T, kv, D, T + G, 30.0)
    slots = torch.randperm(pages * ps, generator=gen(3), device="cuda")[:T]
    before = [t.clone() for t in cache._tensors]
    cache.append(k, v, slots)
    check_rows(cache, slots, k, v)
    # no other row is touched
    free = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    free[slots] = False
    for t, b in zip(cache._tensors, before):
        rows = free.view(pages, ps)[:, None].expand(pages, kv, ps)
        assert torch.equal(t[rows], b[rows])


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,G,rot", [(128, 32, 128), (64, 64, 32), (256, 128, 256), (96, 32, 48), (128, 128, 20), (32, 32, 30)])
def test_turned_keys(dt, layout, D, G, rot):
    """A key's codes are those of the definition in 64 bits; a query is turned as Rotary does."""
    import gptq_bit_weight_amd as q4
    announce(f"append4 rotary {dt} {layout} D={D} G={G} rot={rot}")
    T, kv, H, ps = 1203, 2, 6, 16
    fused = tokens(dt, T, (H + 2 * kv), D, D + rot)
    q, k, v = fused[:, :H], fused[:, H:H + kv], fused[:, H + kv:]
    positions = torch.randint(0, 200000, (T,), generator=gen(5), device="cuda")
    rope = q4.Rotary(D, rot, layout=layout)
    for T1 in (T, 5):
        cache = q4.PagedCache4.empty(-(-T // ps), kv, ps, D, group=G)
        slots = torch.randperm(T, generator=gen(6), device="cuda")[:T1].int()
        y = cache.append(k[:T1], v[:T1], slots, rotary=rope, positions=positions[:T1], q=q[:T1])
        assert torch.equal(y, rope.rotate(q[:T1], positions[:T1]))
        check_rows(cache, slots, turned(k[:T1], positions[:T1], rot, layout), v[:T1], f"T={T1}")
    # in place, and with values that lie on no 16 bytes
    odd = torch.empty(T * (H + 2 * kv) * (D + 1) + 1, dtype=dt, device="cuda")[1:].view(T, H + 2 * kv, D + 1)[..., :D]
    odd.copy_(fused)
    cache = q4.PagedCache4.empty(-(-T // ps), kv, ps, D, group=G)
    slots = torch.arange(T, device="cuda")
    y = cache.append(odd[:, H:H + kv], odd[:, H + kv:], slots, rotary=rope, positions=positions, q=odd[:, :H], q_out=odd[:, :H])
    assert y.data_ptr() == odd.data_ptr() and torch.equal(y, rope.rotate(q.contiguous(), positions))
    check_rows(cache, slots, turned(k, positions, rot, layout), v, "odd strides")


@pytest.mark.parametrize("dt", [F16, BF16])
def test_borders(dt):
    """Values half way between two codes, flat groups, subnormal steps, the largest values, and
    ones that are not finite."""
    import gptq_bit_weight_amd as q4
    announce(f"append4 borders {dt}")
    D, G = 64, 32
    rows = []
    half_steps = torch.arange(31) / 2.0                   # 0 .. 15 by halves: ties to even
    rows.append(torch.cat([half_steps, torch.tensor([15.0])]).repeat(2))
    rows.append(rows[0] * 2.0 ** -12 - 2.0 ** -10)
    rows.append(-rows[0] * 8)
    rows.append(torch.full((D,), 3.25))                   # one value: step 0
    rows.append(torch.full((D,), -0.0))
    rows.append(torch.linspace(0, 5, D) * 2.0 ** -24)     # steps below the least subnormal
    rows.append(torch.linspace(0, 40, D) * 2.0 ** -24)
    rows.append(torch.linspace(-65504, 65504, D))
    rows.append(torch.linspace(-7.5, 7.5, D).index_fill(0, torch.tensor([5]), 2.0 ** -20).index_fill(0, torch.tensor([6]), -(2.0 ** -20)))
    sym = torch.linspace(-7.5, 7.5, G)
    sym[3], sym[4], sym[5] = 2.0 ** -24, -(2.0 ** -24), 0.0
    rows.append(torch.cat([sym, sym * 4]))
    for bad in (math.inf, -math.inf, math.nan):
        r = torch.linspace(-1, 1, D)
        r[40] = bad
        rows.append(r)
    if dt is BF16:
        rows.append(torch.linspace(-1e38, 3e38, D))
        rows.append(torch.linspace(-1, 1, D) * 1e-30)
        rows.append(torch.linspace(-1, 1, D).index_fill(0, torch.tensor([7]), 1e-38))
    x = torch.stack(rows).to(dt).cuda()[:, None]
    T = x.shape[0]
    cache = q4.PagedCache4.empty(T, 1, 1, D, group=G)
    slots = torch.arange(T, device="cuda")
    cache.append(x, x.flip(0).contiguous(), slots)
    check_rows(cache, slots, x, x.flip(0))


def test_slots_outside_strides_and_streams():
    import gptq_bit_weight_amd as q4
    announce("append4 slots outside, strided caches, another stream")
    kv, ps, D, G, pages = 3, 16, 64, 32, 5
    base = torch.zeros(ps, pages, 2, kv, D // 2 + 16, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(pages, ps, kv, 2, D // G + 3, 2, dtype=F16, device="cuda")
    k, v = (base[:, :, i, :, :D // 2].permute(1, 2, 0, 3) for i in (0, 1))
    ks, vs = (scale[:, :, :, i, :D // G].permute(0, 2, 1, 3, 4) for i in (0, 1))
    cache = q4.PagedCache4(k, v, ks, vs)
    T = 40
    x, y = tokens(F16, T, kv, D, 1), tokens(F16, T, kv, D, 2)
    slots = torch.randperm(pages * ps, generator=gen(4), device="cuda")[:T]
    slots[[3, 17, 39]] = torch.tensor([-1, pages * ps, 2 ** 40], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache.append(x, y, slots, stream=s)
    a, b = cache.read(slots, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    on = torch.ones(T, dtype=torch.bool, device="cuda")
    on[[3, 17, 39]] = False
    check_rows(cache, slots[on], x[on], y[on])
    assert not a[~on].any() and not b[~on].any()
    written = torch.zeros(pages * ps, dtype=torch.bool, device="cuda")
    written[slots[on]] = True
    assert not ks.permute(0, 2, 1, 3, 4).reshape(pages * ps, -1)[~written].any()
    assert not base[..., D // 2:].any() and not scale[..., D // G:, :].any()
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    cache.append(x[:0], y[:0], empty)
    assert cache.read(empty)[0].shape == (0, kv, D)


# ---------------------------------------------------------------- attention ---

def make(dt, H, kv, D, G, ps, news, lens, seed=0, spread=1.0):
    """A cache whose rows no token wrote hold NaN, pages in random order."""
    import gptq_bit_weight_amd as q4
    g = gen(seed)
    need = [-(-m // ps) for m in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int().cpu()
    table = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32)
    cache = q4.PagedCache4.empty(pages, kv, ps, D, group=G)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        step = torch.rand(t.shape[:-1], generator=g, device="cuda") * 0.2 + 0.1
        t.copy_(torch.stack([step, step * (torch.rand(step.shape, generator=g, device="cuda") * 4 - 9.5)], -1))
    written = torch.zeros(pages, ps, dtype=torch.bool)
    at = 0
    for b, (n, m) in enumerate(zip(need, lens)):
        mine = order[at:at + n]
        table[b, :n] = mine
        at += n
        rows = torch.arange(m)
        written[mine.long()[rows // ps], rows % ps] = True
    dead = (~written).cuda()[:, None].expand(-1, kv, -1)
    cache.k_scale[dead] = math.nan
    cache.v_scale[dead] = math.nan
    q = (torch.randn(sum(news), H, D, generator=g, device="cuda") * spread).to(dt)
    starts = torch.tensor([0] + news).cumsum(0).int().cuda()
    return q, cache, starts, torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda()


def pools(cache):
    out = []
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        s = s.double()
        out.append(values(unpack(c).double(), s[..., 0], s[..., 1]))
    return out


def run(dt, H, kv, D, G, ps, news, lens, window=0, sinks=0, seed=0, spread=1.0, scale=None):
    announce(f"attend4 {dt} H={H} kv={kv} D={D} G={G} ps={ps} news={news[:8]} lens={lens[:8]} window={window} sinks={sinks}")
    q, cache, starts, lengths, table = make(dt, H, kv, D, G, ps, news, lens, seed, spread)
    y = cache.attend(q, starts, lengths, table, window=window, sinks=sinks, scale=scale)
    k, v = (rows_of(x, table, lens) for x in pools(cache))
    ref, tol = attention(q, k, v, news, lens, window, sinks, scale, F16)
    # (a query that is not finite has no softmax)
    none = ref.isnan()
    assert torch.equal(none, y.isnan()) and (not none.any() or not q.isfinite().all())
    check(torch.where(none, 0, y), torch.where(none, 0, ref), torch.where(none, 0, tol))
    return y


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D,G", [(4, 4, 128, 32), (8, 1, 64, 64), (6, 2, 256, 64), (16, 2, 128, 128), (7, 1, 128, 64), (3, 3, 64, 32),
                                      (16, 1, 256, 256), (4, 2, 256, 32), (4, 2, 96, 32), (4, 2, 32, 32), (5, 1, 160, 32), (2, 1, 192, 64)])
@pytest.mark.parametrize("ps", [16, 64, 5])
def test_single_tokens(dt, H, kv, D, G, ps):
    run(dt, H, kv, D, G, ps, [1] * 7, [1, 2, 31, 32, 33, 500, 1027], seed=D + ps)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D,G", [(4, 4, 64, 32), (8, 2, 128, 32), (12, 4, 128, 128), (4, 1, 256, 64), (5, 1, 96, 32), (4, 2, 192, 32)])
@pytest.mark.parametrize("news,lens", [
    ([64], [64]), ([128], [500]), ([257], [257]), ([1, 300, 17], [900, 300, 80]), ([65, 0, 2], [65, 40, 700]),
    ([600], [2000]), ([33] * 9, [33, 40, 65, 100, 129, 200, 300, 400, 1000])])
@pytest.mark.parametrize("ps", [16, 7])
def test_chunks(dt, H, kv, D, G, news, lens, ps):
    run(dt, H, kv, D, G, ps, news, lens, seed=sum(lens))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D", [(16, 1, 128), (2, 2, 64), (4, 2, 256)])
def test_long(dt, H, kv, D):
    run(dt, H, kv, D, 32, 64, [70], [12001], seed=3)
    run(dt, H, kv, D, 64, 16, [1], [40001], seed=5)
    run(dt, H, kv, D, 64, 16, [2, 1], [9001, 17], seed=6)
    run(dt, H, kv, D, 32, 32, [300, 1, 40], [9000, 4000, 60], window=3000, sinks=5, seed=4)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (31, 4), (32, 32), (33, 40), (64, 100), (100, 16), (1000, 4), (200, 64), (17, 1000)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 9])
def test_windows_and_sinks(dt, window, sinks, D, ps):
    run(dt, 4, 2, D, 32, ps, [1, 1, 1, 1], [300, 5, 1333, 40], window=window, sinks=sinks, seed=window)
    run(dt, 4, 2, D, 32, ps, [1, 1, 40, 7, 130], [300, 5, 333, 7, 450], window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("dt", [F16, BF16])
def test_sharp_flat_and_far(dt):
    run(dt, 4, 2, 128, 64, 16, [1, 100], [700, 400], spread=30.0, seed=8)
    run(dt, 4, 2, 128, 64, 16, [1, 100], [700, 400], spread=0.0, seed=9)
    run(dt, 4, 2, 128, 64, 16, [1, 100], [700, 400], scale=-0.3, seed=10)
    run(dt, 4, 2, 128, 64, 16, [1, 100], [700, 400], scale=0.0, seed=11)
    for few in ([1, 1], [1, 100]):
        run(dt, 4, 2, 128, 64, 16, few, [700, 400], spread=2.0 ** 15, scale=2.0 ** -18, seed=12)
        run(dt, 4, 2, 128, 64, 16, few, [700, 400], spread=2.0 ** 12, scale=2.0 ** -15, seed=12)
        run(dt, 4, 2, 128, 64, 16, few, [700, 400], spread=2.0 ** -12, scale=2.0 ** 9, seed=13)
        if dt is BF16:
            run(dt, 4, 2, 128, 64, 16, few, [700, 400], spread=2.0 ** 100, scale=2.0 ** -103, seed=14)
            run(dt, 4, 2, 128, 64, 16, few, [700, 400], spread=2.0 ** -100, scale=2.0 ** 97, seed=15)


def test_many_requests():
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(1, 700, (200,), generator=g).tolist()
    run(BF16, 8, 2, 128, 32, 16, [0 if i % 5 == 3 else 1 for i in range(200)], lens)
    run(F16, 4, 2, 64, 32, 16, [min(m, [0, 1, 3, 50][i % 4]) for i, m in enumerate(lens)], lens, window=90, sinks=3)
