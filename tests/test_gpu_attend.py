"""Attention of new tokens over the paged cache on the GPU, against the
definition in 64 bits.

Tolerance, derived. A weight w_j = exp(s_j - max) is off by its score's error,
twice over (its own and the sum's): a score is a fp32 sum of dim products, off
by at most (dim + 2) 2^-24 scale sum |q k|; the exponential, the running rescales
and the fp32 sums add a few 2^-24 each, together below 2^-18 (the longest sums
here have some ten thousand terms, summed in tiles of 32). Each weight is then
rounded once for the second product: eps / 2 of itself, or 2^-25 where it is
subnormal in binary16 (the largest weight is 1, so the sum is at least 1). The result is
rounded once: eps / 2. With A = sum w |v| / sum w:
  |y - ref| <= eps/2 |ref| + (eps/2 + 2 delta + 2^-18) A (1 + eps) + 2^-25 sum |v| / sum w + tiny
"""
import math

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


def reference(q, kc, vc, news, lens, table, window=0, scale=None):
    """(result, tolerance) in float64."""
    dt, D = q.dtype, q.shape[2]
    kv, ps = kc.shape[1], kc.shape[2]
    g = q.shape[1] // kv
    scale = D ** -0.5 if scale is None else scale
    half = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * half
    outs, tols, at = [], [], 0
    for b, (n, m) in enumerate(zip(news, lens)):
        if n == 0:
            continue
        qq = q[at:at + n].double()
        at += n
        if m == 0:
            outs.append(torch.zeros_like(qq))
            tols.append(torch.zeros_like(qq))
            continue
        need = -(-m // ps)
        pages = table[b, :need].long().to(kc.device)
        k, v = (c[pages].transpose(0, 1).reshape(kv, -1, D)[:, :m].double() for c in (kc, vc))
        i, j = torch.arange(m - n, m, device=q.device)[:, None], torch.arange(m, device=q.device)[None]
        see = j <= i
        if window:
            see = see & (j > i - window)
        ys, ts = [], []
        for h in range(q.shape[1]):
            s = qq[:, h] @ k[h // g].t() * scale
            mag = (qq[:, h].abs() @ k[h // g].abs().t() * abs(scale)).masked_fill(~see, 0).amax(-1, keepdim=True)
            s = s.masked_fill(~see, -math.inf)
            top = s.amax(-1, keepdim=True)
            w = torch.where(see, torch.exp(s - torch.where(top.isfinite(), top, 0)), 0.0)
            l = w.sum(-1, keepdim=True)
            inv = torch.where(l > 0, 1 / l, 0.0)
            y = w @ v[h // g] * inv
            A = w @ v[h // g].abs() * inv
            delta = (D + 2) * 2.0 ** -24 * mag
            tol = half * y.abs() + (half + 2 * delta + 2.0 ** -18) * A * (1 + 2 * half) + tiny * (l > 0)
            if dt == torch.float16:
                tol = tol + 2.0 ** -25 * (see.double() @ v[h // g].abs()) * inv
            ys.append(y)
            ts.append(tol)
        outs.append(torch.stack(ys, 1))
        tols.append(torch.stack(ts, 1))
    return torch.cat(outs), torch.cat(tols)


def make(dt, H, kv, D, ps, news, lens, seed=0, spread=1.0, spare=3):
    """q, caches, starts, lengths, table: pages in random order; rows that no
    token wrote hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-m // ps) for m in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int().cpu()
    table = torch.full((len(lens), max(max(need), 1)), -7, dtype=torch.int32)
    q = (torch.randn(sum(news), H, D, generator=g, device="cuda") * spread).to(dt)
    kc = torch.randn(pages, kv, ps, D, generator=g, device="cuda").to(dt)
    vc = torch.randn(pages, kv, ps, D, generator=g, device="cuda").to(dt)
    written = torch.zeros(pages, ps, dtype=torch.bool)
    at = 0
    for b, (n, m) in enumerate(zip(need, lens)):
        mine = order[at:at + n]
        table[b, :n] = mine
        at += n
        rows = torch.arange(m)
        written[mine.long()[rows // ps], rows % ps] = True
    dead = ~written.cuda()
    kc[dead[:, None].expand(-1, kv, -1)] = math.nan
    vc[dead[:, None].expand(-1, kv, -1)] = math.nan
    starts = torch.tensor([0] + news).cumsum(0).int().cuda()
    return q, kc, vc, starts, torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda()


def check(y, ref, tol, what=""):
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: {y[i].item()} against "
                             f"{ref[i].item()}, tolerance {tol[i].item()}")


def run(dt, H, kv, D, ps, news, lens, window=0, seed=0, spread=1.0, scale=None):
    import gptq_bit_weight_amd as q4
    announce(f"attend {dt} H={H} kv={kv} D={D} ps={ps} news={news[:8]} lens={lens[:8]} window={window}")
    q, kc, vc, starts, lengths, table = make(dt, H, kv, D, ps, news, lens, seed, spread)
    y = q4.PagedCache(kc, vc).attend(q, starts, lengths, table, window=window, scale=scale)
    check(y, *reference(q, kc, vc, news, lens, table, window, scale))
    return y


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("H,kv,D", [(4, 4, 128), (8, 1, 64), (6, 2, 256), (16, 2, 128), (7, 1, 128), (3, 3, 64), (16, 1, 256)])
@pytest.mark.parametrize("ps", [16, 64])
def test_single_tokens(dt, H, kv, D, ps):
    run(dt, H, kv, D, ps, [1] * 7, [1, 2, 31, 32, 33, 500, 1027], seed=D + ps)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,ps", [(64, 1), (128, 5), (256, 8), (128, 24), (128, 48), (64, 128), (8, 16), (40, 32), (80, 16), (96, 7),
                                  (136, 16), (200, 16)])
def test_page_sizes_and_head_dims(dt, D, ps):
    run(dt, 4, 2, D, ps, [1, 3, 1, 20], [77, 3, 301, 95], seed=D * ps)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_windows(dt, window, D):
    run(dt, 4, 2, D, 16, [1, 1, 40, 7, 130], [300, 5, 333, 7, 450], window=window, seed=window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 3, 17])
def test_windows_inside_the_last_rows(D, window):
    """The first visible key in the last, half written 16 rows of a tile of keys."""
    lens = list(range(1, 140, 3))
    run(torch.float16, 4, 2, D, 16, [1] * len(lens), lens, window=window, seed=1)
    run(torch.bfloat16, 4, 2, D, 64, [min(m, 30) for m in lens], lens, window=window, seed=2)
    run(torch.bfloat16, 4, 2, D, 7, [min(m, 30) for m in lens], lens, window=window, seed=2)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("H,kv,D", [(16, 1, 128), (2, 2, 64), (4, 2, 256)])
def test_chunks_split_over_keys(dt, H, kv, D):
    """Few row tiles over long contexts: their keys are split, joined in order."""
    run(dt, H, kv, D, 64, [70], [12001], seed=3)
    run(dt, H, kv, D, 16, [300, 1, 40], [9000, 4000, 60], seed=4)
    run(dt, H, kv, D, 16, [300, 1, 40], [9000, 4000, 60], window=3000, seed=4)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("H,kv,D", [(4, 4, 64), (8, 2, 128), (12, 4, 128), (4, 1, 256), (5, 1, 128)])
@pytest.mark.parametrize("news,lens", [
    ([64], [64]), ([128], [500]), ([257], [257]), ([1, 300, 17], [900, 300, 80]), ([65, 0, 2], [65, 40, 700]),
    ([600], [2000]), ([33] * 9, [33, 40, 65, 100, 129, 200, 300, 400, 1000])])
def test_chunks(dt, H, kv, D, news, lens):
    run(dt, H, kv, D, 16, news, lens, seed=sum(lens))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_long_context(dt):
    """One request whose keys many workgroups share."""
    run(dt, 8, 1, 128, 64, [1], [40001], seed=5)
    run(dt, 4, 4, 64, 16, [2], [20003], seed=6)
    run(dt, 8, 2, 128, 32, [40, 1], [9001, 17], seed=7)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_sharp_and_flat(dt):
    run(dt, 4, 2, 128, 16, [1, 100], [700, 400], spread=30.0, seed=8)      # one key takes nearly all
    run(dt, 4, 2, 128, 16, [1, 100], [700, 400], spread=0.0, seed=9)       # the mean
    run(dt, 4, 2, 128, 16, [1, 100], [700, 400], scale=-0.3, seed=10)
    run(dt, 4, 2, 128, 16, [1, 100], [700, 400], scale=0.0, seed=11)


def test_many_requests():
    """More requests than a wave has lanes, some without tokens, all lengths."""
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(1, 700, (200,), generator=g).tolist()
    news = [0 if i % 5 == 3 else 1 for i in range(200)]
    run(torch.bfloat16, 8, 2, 128, 16, news, lens)
    news = [min(m, [0, 1, 3, 50][i % 4]) for i, m in enumerate(lens)]
    run(torch.float16, 4, 2, 64, 16, news, lens, window=90)


def test_tokens_that_see_nothing():
    """More new tokens than cached ones: those at negative positions give zeros."""
    for D in (64, 128, 256):
        for news, lens in (([5], [3]), ([1, 2, 40], [0, 0, 9]), ([300], [20]), ([300, 1], [0, 0])):
            y = run(torch.bfloat16, 4, 2, D, 16, news, lens)
            at = 0
            for n, m in zip(news, lens):
                assert (y[at:at + max(n - m, 0)] == 0).all()
                at += n


def test_pages_before_the_window_may_be_gone():
    """Table entries that no visible key needs are not used: they may be any
    number, and their pages any content."""
    import gptq_bit_weight_amd as q4
    for news, lens, window in (([1], [1000], 100), ([200], [1000], 64), ([40, 1], [700, 333], 17)):
        q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, news, lens)
        ref, tol = reference(q, kc, vc, news, lens, table, window)
        for b, (n, m) in enumerate(zip(news, lens)):
            first = max(0, m - n - window + 1) // 16
            kc[table[b, :first].long()] = math.nan
            vc[table[b, :first].long()] = math.nan
            table[b, :first] = -(1 << 31) if b % 2 else 2 ** 31 - 1
        check(q4.PagedCache(kc, vc).attend(q, starts, lengths, table, window=window), ref, tol)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news,lens,window,ps", [
    ([4], [40], 0, 16), ([200], [200], 0, 16), ([200], [333], 70, 16), ([5, 1], [50, 9], 7, 16), ([70], [6000], 0, 64),
    ([130], [131], 0, 7), ([1], [500], 33, 16)])
def test_values_that_are_not_finite_stay_with_those_who_see_them(dt, D, news, lens, window, ps):
    """One value and one key of the cache infinite or NaN: tokens before it (or
    past its window) are as without it, in every row of the same tile of keys;
    of those that see the value, only its column changes, and a NaN key's
    tokens are NaN."""
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(dt, 4, 2, D, ps, news, lens, spread=0.1)
    n, m = news[0], lens[0]
    pos = torch.arange(m - n, m, device="cuda")
    for at in sorted({m - 1, m - max(1, n // 2), max(0, m - n), max(0, m - n - window)}):
        page, row = int(table[0, at // ps]), at % ps
        for bad, where in ((math.inf, vc), (-math.inf, vc), (math.nan, vc), (math.nan, kc)):
            keep = where[page, 1, row, 3].item()
            clean = reference(q, kc, vc, news, lens, table, window)
            where[page, 1, row, 3] = bad
            y = q4.PagedCache(kc, vc).attend(q, starts, lengths, table, window=window)
            where[page, 1, row, 3] = keep
            sees = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
            sees[:n] = (pos >= at) & (pos < at + window if window else True)
            hit = torch.zeros_like(y, dtype=torch.bool)
            hit[:, 2:, 3 if where is vc else slice(None)] = sees.view(-1, *([1] * (1 if where is vc else 2)))
            got = y[hit]
            assert (torch.isnan(got) if math.isnan(bad) else got == bad).all(), (at, bad)
            check(torch.where(hit, 0, y), torch.where(hit, 0, clean[0]), clean[1], f"{bad} at key {at}")


def test_very_low_scores():
    """Scores far below zero, all of them the same number: a softmax goes by
    differences, so the result is that of scores of zero."""
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(torch.bfloat16, 4, 2, 128, 16, [1, 40], [30, 90])
    q[:], kc[:] = 2.0 ** 60, -(2.0 ** 50)
    y = q4.PagedCache(kc, vc).attend(q, starts, lengths, table)
    check(y, *reference(torch.zeros_like(q), kc, vc, [1, 40], [30, 90], table))


def test_strides():
    """q as a view of a fused row, out as a view, a cache of another order,
    a table that is a view of a wider one."""
    import gptq_bit_weight_amd as q4
    news, lens = [1, 90, 3], [200, 90, 50]
    q, kc, vc, starts, lengths, table = make(torch.bfloat16, 8, 2, 128, 16, news, lens)
    ref, tol = reference(q, kc, vc, news, lens, table)
    T = q.shape[0]
    wide = torch.zeros(T, 12, 128, dtype=q.dtype, device="cuda")
    wide[:, 2:10] = q
    store = torch.stack([kc, vc], 2).permute(0, 3, 2, 1, 4).contiguous()     # [pages, rows, k or v, heads, dim]
    k2, v2 = (store[:, :, i].transpose(1, 2) for i in (0, 1))
    t2 = torch.full((3, table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    t2[:, :table.shape[1]] = table
    out = torch.full((T, 10, 130), 7.0, dtype=q.dtype, device="cuda")
    cache = q4.PagedCache(k2, v2)
    y = cache.attend(wide[:, 2:10], starts, lengths, t2[:, :table.shape[1]], out=out[:, 1:9, 1:129])
    check(y, ref, tol)
    assert (out[:, 0] == 7).all() and (out[:, 9] == 7).all() and (out[:, :, 0] == 7).all() and (out[:, :, 129] == 7).all()
    # queries that 16 bytes do not divide are copied first
    odd = torch.zeros(T, 8, 129, dtype=q.dtype, device="cuda")[:, :, 1:]
    odd.copy_(q)
    check(cache.attend(odd, starts, lengths, table), ref, tol)


@pytest.mark.parametrize("news,H", [([1, 1, 1], 8), ([40, 33, 64], 8), ([200, 1, 90], 2)])
def test_requests_that_share_a_row_of_the_table(news, H):
    """One row of pages expanded over the requests, and rows that lie half over each
    other, on both kernels, on the current stream and another."""
    import gptq_bit_weight_amd as q4
    lens = [300] * 3
    q, kc, vc, starts, lengths, table = make(torch.float16, H, 2, 128, 16, news, lens)
    kc.nan_to_num_()
    vc.nan_to_num_()
    cache = q4.PagedCache(kc, vc)
    width = table.shape[1]
    flat = table.flatten()
    for t in (table[:1].expand(3, width), flat.as_strided((3, width), (5, 1))):
        ref = reference(q, kc, vc, news, lens, t.cpu())
        check(cache.attend(q, starts, lengths, t), *ref)
        assert torch.equal(cache.attend(q, starts, lengths, t), cache.attend(q, starts, lengths, t.contiguous()))
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        y = cache.attend(q, starts, lengths, t, stream=s)
        s.synchronize()
        check(y, *ref)
    one = table[:1].as_strided((1, width), (1, 1))          # (a single row's stride is any)
    check(cache.attend(q[:news[0]], starts[:2], lengths[:1], one), *reference(q[:news[0]], kc, vc, news[:1], lens[:1], one.cpu()))


def test_queries_off_sixteen_bytes():
    """A dense q whose first value is not on 16 bytes."""
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, [1, 3], [200, 90])
    odd = torch.zeros(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    odd.copy_(q)
    ref = reference(q, kc, vc, [1, 3], [200, 90], table)
    cache = q4.PagedCache(kc, vc)
    check(cache.attend(odd, starts, lengths, table), *ref)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = cache.attend(odd, starts, lengths, table, stream=s)
    s.synchronize()
    check(y, *ref)


def test_runs_agree_to_the_bit():
    import gptq_bit_weight_amd as q4
    for news, lens in (([1, 1], [30000, 77]), ([300, 1], [5000, 900])):
        q, kc, vc, starts, lengths, table = make(torch.bfloat16, 8, 2, 128, 64, news, lens)
        cache = q4.PagedCache(kc, vc)
        a = cache.attend(q, starts, lengths, table)
        for _ in range(5):
            assert torch.equal(a, cache.attend(q, starts, lengths, table))


def test_cache_beyond_31_bits():
    """Pages whose offsets pass 2^32 bytes and 2^31 values."""
    import gptq_bit_weight_amd as q4
    pages = (1 << 31) // (8 * 64 * 128) + 40
    kc = torch.zeros(pages, 8, 64, 128, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    kc[-32:].normal_()
    vc[-32:].normal_()
    for n, H in ((1, 16), (200, 8)):
        table = torch.arange(pages - 1, pages - 33, -1, dtype=torch.int32, device="cuda")[None].contiguous()
        lens = [2000]
        q = torch.randn(n, H, 128, device="cuda").half()
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        y = q4.PagedCache(kc, vc).attend(q, starts, torch.tensor(lens, dtype=torch.int32, device="cuda"), table)
        check(y, *reference(q, kc, vc, [n], lens, table))


def test_graph_replays():
    """Captured once; lengths, table and data change between replays, with
    eager calls of the same stream beside them."""
    import gptq_bit_weight_amd as q4
    for news, lens, H in (([1, 1, 1], [900, 5000, 64], 16), ([100, 1, 60], [900, 5000, 64], 8)):
        q, kc, vc, starts, lengths, table = make(torch.float16, H, 2, 128, 16, news, lens)
        cache = q4.PagedCache(kc, vc)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = cache.attend(q, starts, lengths, table)
        for i in range(4):
            q.normal_()
            cur = [m - 3 * i for m in lens]
            cur = [max(m, n) for m, n in zip(cur, news)]
            lengths.copy_(torch.tensor(cur, dtype=torch.int32))
            graph.replay()
            eager = cache.attend(q, starts, lengths, table)
            torch.cuda.synchronize()
            assert torch.equal(y, eager), i
            check(y, *reference(q, kc, vc, news, cur, table), what=f"replay {i}")


def test_other_stream():
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, [1, 1], [3000, 77])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = q4.PagedCache(kc, vc).attend(q, starts, lengths, table, stream=s)
    s.synchronize()
    check(y, *reference(q, kc, vc, [1, 1], [3000, 77], table))


def test_bad_tables_stay_inside():
    """Entries, lengths and starts outside their ranges read and write nothing
    outside the tensors (the result has no meaning)."""
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, [1, 40], [300, 200])
    kc.nan_to_num_()
    vc.nan_to_num_()
    cache = q4.PagedCache(kc, vc)
    guard = torch.full((43, 8, 128), 5.0, dtype=q.dtype, device="cuda")
    out = guard[1:42]
    for tb, ln, st in ((torch.full_like(table, 10 ** 9), lengths, starts), (torch.full_like(table, -5), lengths, starts),
                       (table, torch.full_like(lengths, 10 ** 9), starts), (table, torch.full_like(lengths, -3), starts),
                       (table, lengths, torch.tensor([-4, 99, 7], dtype=torch.int32, device="cuda"))):
        cache.attend(q, st, ln, tb, out=out)
        torch.cuda.synchronize()
        assert (guard[0] == 5).all() and (guard[42] == 5).all()


def test_refusals():
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, [1, 1], [30, 20])
    c = q4.PagedCache(kc, vc)
    good = dict(q=q, starts=starts, lengths=lengths, table=table)
    bad = [dict(q=q.bfloat16()), dict(q=q[:, :7]), dict(q=q[..., :64]), dict(q=q[0]), dict(q=q.cpu()), dict(starts=starts.long()),
           dict(starts=starts[:2]), dict(lengths=lengths[:1]), dict(table=table[:1]), dict(table=table[:, :0]),
           dict(lengths=lengths.cpu()), dict(table=table.float()), dict(window=-1), dict(scale=math.nan), dict(scale=math.inf),
           dict(out=q), dict(out=torch.empty_like(q)[:1]), dict(out=torch.empty_like(q).bfloat16()), dict(table=table[0])]
    for i, kw in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            c.attend(**{**good, **kw})
            pytest.fail(f"case {i} was taken")
    k9 = torch.zeros(2, 2, 16, 72 + 4, dtype=torch.float16, device="cuda")
    with pytest.raises(NotImplementedError):
        q4.PagedCache(k9, k9.clone()).attend(torch.zeros(2, 2, 76, dtype=torch.float16, device="cuda"), starts, lengths, table)
    k9 = torch.zeros(2, 2, 16, 264, dtype=torch.float16, device="cuda")
    with pytest.raises(NotImplementedError):
        q4.PagedCache(k9, k9.clone()).attend(torch.zeros(2, 2, 264, dtype=torch.float16, device="cuda"), starts, lengths, table)
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert c.attend(q[:0], e, lengths[:0], table[:0]).shape == (0, 8, 128)
    assert c.attend(q[:0], torch.zeros(3, dtype=torch.int32, device="cuda"), lengths, table).shape == (0, 8, 128)


def test_two_threads_on_one_stream():
    """Two threads with caches of their own on the same stream, chunks whose keys
    are split (two launches a call) beside single tokens: each has what it has alone."""
    import threading

    import gptq_bit_weight_amd as q4
    work = []
    for i, (news, lens, D) in enumerate((([70], [9001], 128), ([300, 1, 40], [5000, 900, 60], 128), ([33], [6000], 256))):
        q, kc, vc, starts, lengths, table = make(torch.bfloat16, 8, 2, D, 16, news, lens, seed=i)
        c = q4.PagedCache(kc, vc)
        y = c.attend(q, starts, lengths, table)
        check(y, *reference(q, kc, vc, news, lens, table))
        work.append((c, q, starts, lengths, table, y, []))
    torch.cuda.synchronize()
    errors = []

    def run(c, q, starts, lengths, table, y, outs):
        try:
            for _ in range(200):
                outs.append(c.attend(q, starts, lengths, table))
        except Exception as e:      # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for w in work:
        assert len(w[6]) == 200
        for i, y in enumerate(w[6]):
            assert torch.equal(y, w[5]), i


def test_captured_stream_that_is_not_the_current_one():
    """A capture begun on a stream that the calls are given and that is not current:
    replays on one stream beside eager calls on the captured one."""
    import gptq_bit_weight_amd as q4
    news, lens = [70, 1], [9001, 300]
    q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, news, lens)
    ref = reference(q, kc, vc, news, lens, table)
    cache = q4.PagedCache(kc, vc)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    cache.attend(q, starts, lengths, table, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph.capture_begin()
    y = cache.attend(q, starts, lengths, table, stream=s)
    with torch.cuda.stream(s):
        graph.capture_end()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        graph.replay()              # (on the current stream)
        outs.append(cache.attend(q, starts, lengths, table, stream=s))
    torch.cuda.synchronize()
    check(y, *ref)
    for o in outs:
        assert torch.equal(o, y)


@pytest.mark.parametrize("window", [200, 201, 304, 2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 10 ** 30])
def test_windows_past_the_cache(window):
    """A window of all the keys there are, or of any larger number, is none, also for
    tokens at negative positions (more new tokens than cached ones)."""
    import gptq_bit_weight_amd as q4
    for D in (64, 128, 256):
        for news, lens in (([300], [200]), ([3], [2]), ([1, 1, 40], [200, 3, 9]), ([300, 1], [0, 190])):
            q, kc, vc, starts, lengths, table = make(torch.bfloat16, 4, 2, D, 16, news, lens)
            y = q4.PagedCache(kc, vc).attend(q, starts, lengths, table, window=window)
            check(y, *reference(q, kc, vc, news, lens, table), what=f"{D} {news} {lens}")


def test_out_that_meets_an_input_is_refused():
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(torch.float16, 8, 2, 128, 16, [1, 1], [30, 20])
    c = q4.PagedCache(kc, vc)
    flat = torch.zeros(2 * 8 * 128 + 64, dtype=torch.float16, device="cuda")
    ints = flat[-8:].view(torch.int32)
    ints[:2].copy_(lengths)
    for kw in (dict(out=kc.view(-1)[:2048].view(2, 8, 128)), dict(out=vc.view(-1)[256:2304].view(2, 8, 128)),
               dict(out=flat[64:].view(2, 8, 128), lengths=ints[:2])):
        with pytest.raises(ValueError, match="overlaps"):
            c.attend(**{**dict(q=q, starts=starts, lengths=lengths, table=table), **kw})
    # parts of one wider row that lie side by side are not in each other's way
    arena = torch.zeros(2, 3, 8, 128, dtype=torch.float16, device="cuda")
    arena[:, 0] = q
    check(c.attend(arena[:, 0], starts, lengths, table, out=arena[:, 1]), *reference(q, kc, vc, [1, 1], [30, 20], table))
    assert (arena[:, 2] == 0).all() and torch.equal(arena[:, 0], q)
    with pytest.raises(ValueError, match="overlaps"):
        c.attend(arena[:, 0], starts, lengths, table, out=arena.view(2, 24, 128)[:, 7:15])


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news,lens", [([1] * 150, [6000] * 150), ([1, 3], [6000, 9000]), ([100], [12001]), ([64, 70], [6000, 5000])])
@pytest.mark.parametrize("where", [0, -1])
def test_many_small_weights_count(dt, D, news, lens, where):
    """One key with the largest weight and a value of 0, thousands with weights of
    2^-25.1 of it and values of 1: what they add up to is the whole result. Tolerance as
    above but for the last term: a weight rounds to a step of 2^-24 from 2^15 (few rows)
    or 2^7 (many) up, so it is off by 2^-32 of the largest at most."""
    import gptq_bit_weight_amd as q4
    announce(f"small weights {dt} D={D} {news[:3]} {lens[:3]} {where}")
    q, kc, vc, starts, lengths, table = make(dt, 4, 2, D, 16, news, lens)
    q.zero_()
    q[..., 0] = 1
    low = torch.tensor(-17.4).to(dt).item()
    kc[:], vc[:] = 0, 1
    kc[..., 0] = low
    for b, (n, m) in enumerate(zip(news, lens)):
        at = 0 if where == 0 else m - n          # the first key, or the first new one
        page = int(table[b, at // 16])
        kc[page, :, at % 16, 0] = 0
        vc[page, :, at % 16] = 0
    y = q4.PagedCache(kc, vc).attend(q, starts, lengths, table, scale=1.0)
    ref, tol = reference(q, kc, vc, news, lens, table, scale=1.0)
    if dt == torch.float16:                      # (tol has 2^-25 for each visible key in place of 2^-32)
        keys = torch.cat([torch.arange(m - n, m) for n, m in zip(news, lens)]).to(ref)[:, None, None] + 1
        tol = tol - (2.0 ** -25 - 2.0 ** -32) * (keys - 1) / (1 + (keys - 1) * math.exp(low))
    assert (ref > 1e-4).all()
    check(y, ref, tol)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news,lens", [([1, 1, 2], [40, 3, 900]), ([1, 5], [6000, 3]), ([70], [9001]), ([200, 90, 1], [200, 40, 5])])
def test_scores_of_minus_infinity_have_no_softmax(dt, D, news, lens):
    """Tokens whose every visible score is -inf are NaN, by the definition; with one
    finite score they have that key's value; those that see no key stay zero."""
    import gptq_bit_weight_amd as q4
    q, kc, vc, starts, lengths, table = make(dt, 4, 2, D, 16, news, lens)
    q.abs_().add_(0.1)
    kc[..., 0] = torch.where(kc[..., 0].isnan(), kc[..., 0], -math.inf)
    cache = q4.PagedCache(kc, vc)
    y = cache.attend(q, starts, lengths, table)
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(news, lens)]).cuda()
    assert y[pos >= 0].isnan().all() and (y[pos < 0] == 0).all()
    page = table[:, 0].long()
    kc[page, :, 0] = 0
    y = cache.attend(q, starts, lengths, table)
    want = torch.cat([vc[p, :, 0].repeat_interleave(2, 0)[None].expand(n, -1, -1) for n, p in zip(news, page.tolist())])
    assert torch.equal(y, torch.where((pos >= 0)[:, None, None], want, 0))
