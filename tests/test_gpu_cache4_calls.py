"""Calls of the cache held in 4 bits as programs make them: values that are not finite, tokens
that see nothing, pools past 32 bits, strides, streams, threads, captured graphs.

Results are compared with the definition in 64 bits (tolerances: test_gpu_cache4.py) or, bit for
bit, with another call of the same operator."""
import math
import threading

import pytest

from tests.cache4_util import attention, rows_of, turned
from tests.gpu_util import announce, torch_mod
from tests.test_gpu_attend import check
from tests.test_gpu_cache4 import check_rows, gen, make, pools, run, tokens

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


def seen_by(news, lens, window, sinks):
    """Per new token the visible keys of its request: bool [tokens of it, length] each."""
    out = []
    for n, m in zip(news, lens):
        i, j = torch.arange(m - n, m)[:, None], torch.arange(m)[None]
        see = j <= i
        if window:
            see = see & ((j > i - window) | (j < sinks))
        out.append(see)
    return out


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 64), (96, 32)])
@pytest.mark.parametrize("news,lens", [([1, 1, 3], [300, 130, 70]), ([60, 9, 130], [300, 130, 400])])
@pytest.mark.parametrize("window,sinks,ps", [(50, 5, 16), (0, 0, 16), (33, 0, 7)])
def test_what_is_not_finite_reaches_only_those_who_see_it(dt, D, G, news, lens, window, sinks, ps):
    """A key's group of NaN makes the rows that see it NaN as a whole, a value's its
    columns; whoever does not see them gets what it would without them."""
    H, kv = 4, 2
    announce(f"attend4 not finite {dt} D={D} G={G} news={news} window={window} sinks={sinks} ps={ps}")
    q, cache, starts, lengths, table = make(dt, H, kv, D, G, ps, news, lens, seed=D + ps)
    # the first new token of a request sees its own key and not the next one: keys about there, and about
    # the window's and the sinks' edges
    bad_k, bad_v = [], []
    for b, (n, m) in enumerate(zip(news, lens)):
        first = m - n
        for j in {first + 1, first + n // 2, first - window, first - window + 1, sinks, sinks + 1}:
            if 0 <= j < m:
                (bad_k if (j + b) % 3 == 0 else bad_v).append((b, j, (j + b) % kv, j % (D // G)))
    plain_k, plain_v = (rows_of(x, table, lens) for x in pools(cache))
    for t, bad in ((cache.k_scale, bad_k), (cache.v_scale, bad_v)):
        for b, j, h, g in bad:
            t[int(table[b, j // ps]), h, j % ps, g] = math.nan
    got = cache.attend(q, starts, lengths, table, window=window, sinks=sinks)
    ref, tol = attention(q, plain_k, plain_v, news, lens, window, sinks, None, F16)
    none = torch.zeros(q.shape, dtype=torch.bool)
    at, see = [0], seen_by(news, lens, window, sinks)
    for n in news:
        at.append(at[-1] + n)
    for b, j, h, g in bad_k:
        none[at[b]:at[b + 1], h * (H // kv):(h + 1) * (H // kv)] |= see[b][:, j, None, None]
    for b, j, h, g in bad_v:
        none[at[b]:at[b + 1], h * (H // kv):(h + 1) * (H // kv), g * G:(g + 1) * G] |= see[b][:, j, None, None]
    none = none.cuda()
    assert torch.equal(got.isnan(), none)
    check(torch.where(none, 0, got), torch.where(none, 0, ref), torch.where(none, 0, tol))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 16), (256, 7)])
def test_tokens_that_see_nothing(dt, D, ps):
    """More new tokens than cached ones: those before the first key give zeros."""
    run(dt, 4, 2, D, 32, ps, [1, 1, 1], [0, 1, 0], seed=1)
    run(dt, 4, 2, D, 32, ps, [5, 3, 2], [2, 0, 40], seed=2)
    run(dt, 4, 2, D, 32, ps, [130, 200, 40], [60, 0, 300], seed=3)
    run(dt, 4, 2, D, 32, ps, [130, 3, 40], [60, 0, 300], window=20, sinks=3, seed=4)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D,G", [(8, 2, 128, 64), (6, 2, 64, 32), (4, 1, 256, 32)])
@pytest.mark.parametrize("ps", [16, 11])
def test_between_few_rows_and_many(dt, H, kv, D, G, ps):
    """5 to 100 rows a request, on both sides of where one kernel takes over from the other."""
    for n in (3, 15, 16, 17, 24, 25):
        run(dt, H, kv, D, G, ps, [n] * 5, [n, 64, 100, 333, 1200], seed=n)
        run(dt, H, kv, D, G, ps, [n] * 5, [n, 64, 100, 333, 1200], window=70, sinks=20, seed=n)
    run(dt, H, kv, D, G, ps, [0, 90, 0, 1, 1, 0, 1], [40, 500, 0, 30, 2000, 7, 33], seed=7)


def test_no_tokens_and_no_requests():
    import gptq_bit_weight_amd as q4
    cache = q4.PagedCache4.empty(4, 2, 16, 64)
    q = tokens(F16, 3, 4, 64, 1)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    assert cache.attend(q[:0], torch.zeros(2, dtype=torch.int32, device="cuda"), zero, table).shape == (0, 4, 64)
    # rows behind the last sequence stay as they were
    out = torch.full_like(q, 7.0)
    cache.attend(q, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), zero, table, out=out)
    assert not out[0].any() and (out[1:] == 7).all()
    for types in ((F16, BF16), (BF16, F16), (torch.float32, torch.float32)):
        with pytest.raises(ValueError):
            cache.append(q[:, :2].to(types[0]), q[:, :2].to(types[1]), torch.arange(3, device="cuda"))
    with pytest.raises(ValueError):
        cache.attend(q.float(), torch.tensor([0, 3], dtype=torch.int32, device="cuda"), zero, table)
    with pytest.raises(ValueError):
        cache.attend(q, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), zero, table, out=q.to(BF16))
    with pytest.raises(ValueError):
        cache.attend(q, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), zero, table, window=4, sinks=-1)
    with pytest.raises(ValueError):
        cache.read(torch.zeros(2, 2, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_many_tokens_with_queries(dt, layout):
    """Queries beside many keys and values, bit for bit as Rotary turns them, in place too."""
    import gptq_bit_weight_amd as q4
    announce(f"append4 many queries {dt} {layout}")
    T, H, kv, D, ps = 3001, 8, 2, 128, 16
    q, k, v = tokens(dt, T, H, D, 1), tokens(dt, T, kv, D, 2), tokens(dt, T, kv, D, 3)
    positions = torch.randint(0, 100000, (T,), generator=gen(5), device="cuda", dtype=torch.int32)
    rope = q4.Rotary(D, 64, layout=layout)
    slots = torch.randperm(T, generator=gen(6), device="cuda")
    cache = q4.PagedCache4.empty(-(-T // ps), kv, ps, D, group=64)
    want = rope.rotate(q, positions)
    assert torch.equal(cache.append(k, v, slots, rotary=rope, positions=positions, q=q), want)
    check_rows(cache, slots, turned(k, positions, 64, layout), v)
    cache.append(k, v, slots, rotary=rope, positions=positions, q=q, q_out=q)
    assert torch.equal(q, want)


def spaced(cache, k_gap, v_gap):
    """The same cache with pages k_gap and v_gap bytes of codes and an eighth of that of scales apart."""
    import gptq_bit_weight_amd as q4
    out = []
    for t, step in ((cache.k, k_gap), (cache.v, v_gap), (cache.k_scale, k_gap // 16), (cache.v_scale, v_gap // 16)):
        span = (t.shape[0] - 1) * step + t[0].numel()
        mem = torch.empty(span, dtype=t.dtype, device="cuda")
        s = mem.as_strided(t.shape, (step,) + t[0].stride())
        s.copy_(t)
        out.append(s)
    return q4.PagedCache4(*out)


@pytest.mark.parametrize("k_gap,v_gap", [(1 << 20, 1 << 20), (3 << 30, 1 << 20), (1 << 20, 3 << 30), (1 << 20, 5 << 30)])
def test_offsets_past_32_bits(k_gap, v_gap):
    """Pages of keys or of values gigabytes apart (14 of them: to 42 GiB, where 32 bits count 16 bytes each, and to 70 GiB, where they
    do not) give what neighbouring ones do."""
    H, kv, D, G, ps = 8, 2, 128, 64, 16
    for dt, news, lens in ((F16, [1, 1], [100, 60]), (BF16, [100, 40], [100, 60])):
        announce(f"attend4 pages {k_gap} and {v_gap} bytes apart {dt} news={news}")
        q, cache, starts, lengths, table = make(dt, H, kv, D, G, ps, news, lens, seed=3)
        want = cache.attend(q, starts, lengths, table)
        far = spaced(cache, k_gap, v_gap)
        assert far.k.stride(0) == k_gap and far.v.stride(0) == v_gap
        got = far.attend(q, starts, lengths, table)
        # (where 32 bits do not suffice the keys are found one by one, by the same kernel: the sums are the same)
        assert torch.equal(got, want)
        slots = torch.arange(cache.pages * ps, device="cuda")
        for a, b in zip(far.read(slots), cache.read(slots)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        k, v = tokens(dt, 5, kv, D, 1), tokens(dt, 5, kv, D, 2)
        last = slots[-5:]
        far.append(k, v, last)
        check_rows(far, last, k, v)
        far.copy_pages(torch.tensor([cache.pages - 1], device="cuda"), torch.tensor([0], device="cuda"))
        assert torch.equal(far.k[0], far.k[-1]) and torch.equal(far.v_scale[0].view(torch.int16), far.v_scale[-1].view(torch.int16))
        del far
        torch.cuda.empty_cache()


@pytest.mark.parametrize("news,lens", [([1, 1], [700, 40]), ([100, 33], [300, 900])])
def test_strided_caches_and_queries(news, lens):
    import gptq_bit_weight_amd as q4
    H, kv, D, G, ps = 6, 3, 64, 32, 16
    announce(f"attend4 strides news={news}")
    q, cache, starts, lengths, table = make(F16, H, kv, D, G, ps, news, lens, seed=5)
    want = cache.attend(q, starts, lengths, table, window=90, sinks=2)
    codes = torch.zeros(ps, cache.pages, 2, kv, D // 2 + 16, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(cache.pages, ps, kv, 2, D // G + 3, 2, dtype=F16, device="cuda")
    k, v = (codes[:, :, i, :, :D // 2].permute(1, 2, 0, 3) for i in (0, 1))
    ks, vs = (scales[:, :, :, i, :D // G].permute(0, 2, 1, 3, 4) for i in (0, 1))
    for a, b in zip((k, v, ks, vs), cache._tensors):
        a.copy_(b)
    odd = q4.PagedCache4(k, v, ks, vs)
    wide = torch.zeros(H, q.shape[0], D + 8, dtype=F16, device="cuda")[..., :D].transpose(0, 1)
    wide.copy_(q)
    out = torch.full((q.shape[0], H, D + 1), 7.0, dtype=F16, device="cuda")
    tables = torch.full((len(lens), table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    tables[:, :table.shape[1]] = table
    odd.attend(wide, starts, lengths, tables[:, :table.shape[1]], window=90, sinks=2, out=out[..., :D])
    assert torch.equal(out[..., :D], want) and (out[..., D:] == 7).all()


def test_threads_and_streams():
    """Calls of several threads, each on its own stream and two on one, over one cache."""
    cases = []
    for i, (news, lens) in enumerate([([1] * 6, [900, 3, 50, 700, 2000, 33]), ([60, 3], [400, 700]), ([1], [6000]), ([200], [900])]):
        c = make((F16, BF16)[i % 2], 8, 2, 128, 64, 16, news, lens, seed=i)
        cases.append((c[1], (c[0],) + c[2:], c[1].attend(c[0], *c[2:])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    wrong = []

    def work(i):
        cache, args, want = cases[i]
        s = streams[min(i, 2)]
        got = [cache.attend(*args, stream=s) for _ in range(40)]
        s.synchronize()
        wrong.extend((i, k) for k, y in enumerate(got) if not torch.equal(y, want))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("news,lens", [([1] * 5, [900, 30, 50, 700, 2000]), ([80, 3], [400, 700]), ([1400], [1700])])
def test_two_captured_graphs(news, lens):
    """Two graphs of append and attend over caches of their own, replayed in turn while lengths grow on the
    device, against eager calls."""
    import gptq_bit_weight_amd as q4
    H, kv, D, G, ps = 8, 2, 128, 64, 16
    announce(f"attend4 captured news={news}")
    B, T = len(news), sum(news)
    rope = q4.Rotary(D, D)
    sides = []
    for i, dt in enumerate((F16, BF16, F16, BF16)):
        q, cache, starts, lengths, table = make(dt, H, kv, D, G, ps, news, [m + 40 for m in lens], seed=i % 2)
        lengths.copy_(torch.tensor(lens))
        cache.k_scale.nan_to_num_(0.5)
        cache.v_scale.nan_to_num_(0.5)
        k, v = tokens(dt, T, kv, D, 10 + i % 2), tokens(dt, T, kv, D, 20 + i % 2)
        row = torch.cat([torch.arange(n) - n for n in news]).cuda()
        of = torch.repeat_interleave(torch.arange(B), torch.tensor(news)).cuda()

        def step(q=q, cache=cache, starts=starts, lengths=lengths, table=table, k=k, v=v):
            at = lengths[of] + row
            slots = table[of, torch.div(at, ps, rounding_mode="floor")].long() * ps + at % ps
            turned_q = cache.append(k, v, slots, rotary=rope, positions=at, q=q)
            y = cache.attend(turned_q, starts, lengths, table, window=100, sinks=4)
            lengths += 1
            return y

        sides.append((step, cache))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        wants = [sides[0][0](), sides[1][0]()]
        first = [sides[2][0](), sides[3][0]()]          # (warms up; both sides are a step on)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(wants, first))
    graphs = []
    for step, _ in sides[2:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = step()
        graphs.append((g, y))
    for i in range(12):
        for k in (0, 1):
            want = sides[k][0]()
            graphs[k][0].replay()
            torch.cuda.synchronize()
            assert torch.equal(graphs[k][1], want), (i, k)
            for a, b in zip(sides[k][1]._tensors, sides[2 + k][1]._tensors):
                assert torch.equal(a, b), (i, k)


@pytest.mark.parametrize("ps", [1, 3, 512])
def test_pages_of_one_row_and_of_many(ps):
    run(F16, 4, 2, 64, 32, ps, [1, 1], [70, 515], seed=ps)
    run(BF16, 4, 2, 128, 128, ps, [90, 1], [300, 65], window=80, sinks=2, seed=ps)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D", [(17, 1, 64), (64, 1, 128), (65, 1, 64), (120, 1, 32), (80, 40, 64)])
def test_large_groups_and_many_heads(dt, H, kv, D):
    run(dt, H, kv, D, 32, 16, [1, 1, 2], [90, 700, 33], seed=H)


def test_thousands_of_requests():
    lens = [1 + (7 * i) % 90 for i in range(3000)]
    run(F16, 4, 2, 64, 64, 16, [1] * 3000, lens, seed=1)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("news,lens", [([1] * 20, [50 + i for i in range(20)]), ([70], [200])])
def test_queries_that_are_not_finite(dt, news, lens):
    """Such a token's heads are NaN, the others are what they are without it. (Not always to the bit: rows of one wave
    put a growth of their maxima off together, so a row's weights may be rounded at another power of its sum; the derived
    tolerance holds at any.)"""
    announce(f"attend4 queries not finite {dt} news={news[:3]}")
    q, cache, starts, lengths, table = make(dt, 4, 2, 128, 32, 16, news, lens, seed=4)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    k, v = (rows_of(x, table, lens) for x in pools(cache))
    ref, tol = attention(q, k, v, news, lens, 0, 0, None, F16)
    for i, x in ((0, math.inf), (3, -math.inf), (17, math.nan)):
        q[i, i % 4, 5] = x
        bad[i, i % 4] = True
    got = cache.attend(q, starts, lengths, table)
    assert not got[bad].isfinite().any()
    check(got[~bad], ref[~bad], tol[~bad])


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_read_by_either_index(index):
    import gptq_bit_weight_amd as q4
    announce(f"read4 {index}")
    cache = q4.PagedCache4.empty(5, 3, 7, 96)
    k, v = tokens(F16, 35, 3, 96, 1), tokens(F16, 35, 3, 96, 2)
    cache.append(k, v, torch.arange(35, device="cuda"))
    slots = torch.tensor([34, 0, -1, 35, 12, 12], dtype=index, device="cuda")
    a, b = cache.read(slots)
    whole = cache.read(torch.arange(35, device="cuda"))
    for x, y in zip((a, b), whole):
        assert torch.equal(x[[0, 1, 4, 5]], y[[34, 0, 12, 12]]) and not x[[2, 3]].any()


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,kv,D,G,ps", [(8, 2, 128, 32, 16), (16, 2, 64, 64, 7), (12, 3, 256, 128, 64), (8, 2, 96, 32, 1)])
@pytest.mark.parametrize("news,lens,window,sinks", [
    ([700], [900], 0, 0), ([1300, 0, 700], [1300, 50, 2500], 0, 0), ([900, 1100], [400, 1111], 0, 0), ([800], [3000], 300, 0),
    ([800, 1400], [3001, 2000], 170, 37), ([700], [0], 0, 0)])
def test_long_chunks(dt, H, kv, D, G, ps, news, lens, window, sinks):
    """Chunks whose keys and values are brought into binary16 once."""
    import ctypes
    import gptq_bit_weight_amd as q4
    from gptq_bit_weight_amd.attention import _Cache4
    assert sum(news) * H // kv >= 2560 * len(news)
    width = max(max(-(-m // ps) for m in lens), 1)
    c = _Cache4(*[1 << 20] * 4, *[(ctypes.c_int64 * 3)(0, 0, 0)] * 4, width * len(lens) + 3, kv, ps, D, G)
    lib = q4.load_library()
    full = lib.q4_attend4_workspace_for(ctypes.byref(c), H, sum(news), len(news), width)
    assert full > 4 * len(news) * kv * width * ps * D
    run(dt, H, kv, D, G, ps, news, lens, window=window, sinks=sinks, seed=D + len(news))


def test_long_chunks_in_less_memory():
    """With the least workspace every workgroup unpacks for itself: another order of the sums, the same bound."""
    import ctypes
    import gptq_bit_weight_amd as q4
    announce("attend4 long chunk, least workspace")
    H, kv, D, ps, news, lens = 8, 2, 128, 16, [1000, 700], [1300, 2000]
    lib = q4.load_library()
    for dt in (F16, BF16):
        q, cache, starts, lengths, table = make(dt, H, kv, D, 32, ps, news, lens, seed=9)
        least = lib.q4_attend4_workspace(cache._ref, H)
        full = lib.q4_attend4_workspace_for(cache._ref, H, sum(news), 2, table.shape[1])
        assert 0 < least < full
        # few rows, or more than 2^30 bytes: no more than the least
        assert lib.q4_attend4_workspace_for(cache._ref, H, 100, 2, table.shape[1]) == least
        assert lib.q4_attend4_workspace_for(cache._ref, H, 4000, 2, 1 << 20) == least
        assert lib.q4_attend4_workspace_for(cache._ref, H, 0, 0, 0) == least
        ws = torch.zeros(least, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        st = lib.q4_attend4(cache._ref, q.data_ptr(), q.stride(0), q.stride(1), H, q.shape[0], starts.data_ptr(), lengths.data_ptr(),
                            table.data_ptr(), table.shape[1], table.stride(0), 2, 0, 0, D ** -0.5, out.data_ptr(), out.stride(0), out.stride(1),
                            ws.data_ptr(), least, int(dt is BF16), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        k, v = (rows_of(x, table, lens) for x in pools(cache))
        ref, tol = attention(q, k, v, news, lens, 0, 0, None, F16)
        check(out, ref, tol)
        check(cache.attend(q, starts, lengths, table), ref, tol)


@pytest.mark.parametrize("dt", [F16, BF16])
def test_what_is_not_finite_in_long_chunks(dt):
    H, kv, D, G, ps, window, sinks = 8, 2, 64, 32, 16, 150, 5
    news, lens = [700, 900], [1000, 950]
    announce(f"attend4 long chunks not finite {dt}")
    q, cache, starts, lengths, table = make(dt, H, kv, D, G, ps, news, lens, seed=5)
    plain_k, plain_v = (rows_of(x, table, lens) for x in pools(cache))
    none = torch.zeros(q.shape, dtype=torch.bool)
    see, at = seen_by(news, lens, window, sinks), [0, 700, 1600]
    for b, j, h, g, t in ((0, 7, 0, 1, "k"), (0, 400, 1, 0, "v"), (0, 999, 0, 0, "v"), (1, 60, 1, 1, "k"), (1, 300, 0, 1, "v"), (1, 949, 1, 0, "k")):
        (cache.k_scale if t == "k" else cache.v_scale)[int(table[b, j // ps]), h, j % ps, g] = math.nan
        cols = slice(None) if t == "k" else slice(g * G, (g + 1) * G)
        none[at[b]:at[b + 1], h * (H // kv):(h + 1) * (H // kv), cols] |= see[b][:, j, None, None]
    got = cache.attend(q, starts, lengths, table, window=window, sinks=sinks)
    ref, tol = attention(q, plain_k, plain_v, news, lens, window, sinks, None, F16)
    none = none.cuda()
    assert torch.equal(got.isnan(), none)
    check(torch.where(none, 0, got), torch.where(none, 0, ref), torch.where(none, 0, tol))


@pytest.mark.parametrize("news,lens", [([1, 1], [900, 1300]), ([40, 30], [900, 1300]), ([700, 800], [1600, 2300])])
@pytest.mark.parametrize("ps", [16, 7])
def test_pages_between_sinks_and_window_are_not_named(news, lens, ps):
    """Entries of pages that no token sees name nothing, and the page that is read in their stead holds NaN."""
    H, kv, D, window, sinks = 8, 2, 64, 200, 9
    announce(f"attend4 pages not named news={news} ps={ps}")
    for dt in (F16, BF16):
        q, cache, starts, lengths, table = make(dt, H, kv, D, 32, ps, news, lens, seed=6)
        k, v = (rows_of(x, table, lens) for x in pools(cache))
        spare = cache.pages - 1
        free = [p for p in range(cache.pages) if not (table == p).any()][0]
        cache.copy_pages(torch.tensor([spare], device="cuda"), torch.tensor([free], device="cuda"))
        table[table == spare] = free
        cache.k_scale[spare], cache.v_scale[spare] = math.nan, math.nan
        for b, (n, m) in enumerate(zip(news, lens)):
            table[b, -(-sinks // ps):max(m - n - window + 1, 0) // ps] = -1
        got = cache.attend(q, starts, lengths, table, window=window, sinks=sinks)
        check(got, *attention(q, k, v, news, lens, window, sinks, None, F16))


def test_a_cache_of_one_tensor_twice():
    import gptq_bit_weight_amd as q4
    announce("cache4 of one tensor twice")
    c = q4.PagedCache4.empty(3, 2, 16, 64)
    with pytest.raises(ValueError, match="overlap"):
        q4.PagedCache4(c.k, c.k, c.k_scale, c.v_scale)
    with pytest.raises(ValueError, match="overlap"):
        q4.PagedCache4(c.k, c.v, c.v_scale, c.v_scale)
