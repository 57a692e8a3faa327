"""Cases, plain forms and inputs of the operators around the paged cache: the
cache held in 4 bits (the write of new tokens, attention over it), attention
with a sliding window and first tokens that stay visible, and the pages' own
operators (forking and freeing requests, compacting the pool).

``own`` selects what run() calls: the plain form in elementary torch
operations, or this package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LARGEST = 65440.0       # finite values beyond it are held as it


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # a decode step of eight requests: rotate q and k, quantise k and v into the cache; read the rows back
        dict(name="append4 8 tokens", op="append4", dtype="f16", T=8, heads=32, kv=32, dim=128, group=32, turned=True,
             far=4096, page=16),
        # a long prompt's chunk, far into a long context
        dict(name="append4 16384 tokens", op="append4", dtype="bf16", T=16384, heads=64, kv=8, dim=128, group=32,
             turned=True, far=131072, page=64),
        # a token of one request
        dict(name="attend4 1 token over 700", op="attend4", dtype="f16", heads=32, kv=32, dim=128, group=64, page=16,
             B=1, new=1, length=700, window=0, sinks=0, ragged=False),
        # a decode step of 64 requests of different lengths, grouped heads
        dict(name="attend4 64 x 1 over 8192", op="attend4", dtype="bf16", heads=64, kv=8, dim=128, group=32, page=64,
             B=64, new=1, length=8192, window=0, sinks=0, ragged=True),
        # a token at the end of one long context
        dict(name="attend4 1 token over 131000", op="attend4", dtype="bf16", heads=64, kv=8, dim=128, group=128, page=64,
             B=1, new=1, length=131000, window=0, sinks=0, ragged=False),
        # a chunk of a long prompt
        dict(name="attend4 2048 over 8192", op="attend4", dtype="bf16", heads=32, kv=8, dim=128, group=32, page=64,
             B=1, new=2048, length=8192, window=0, sinks=0, ragged=False),
        # a decode step of streaming requests: the window and four sinks, 16-bit cache
        dict(name="sinks 48 x 1 window 4096", op="attend", dtype="bf16", heads=64, kv=8, dim=128, group=0, page=64,
             B=48, new=1, length=16000, window=4096, sinks=4, ragged=True),
        # chunks of several prompts beside single tokens, window and sinks
        dict(name="sinks 6 chunks", op="attend", dtype="f16", heads=32, kv=8, dim=64, group=0, page=16,
             B=6, new=701, length=4096, window=1024, sinks=16, ragged=True),
        # one of four samples of one short prompt, which are then dropped
        dict(name="fork 1 into 3", op="fork", dtype="f16", kv=32, dim=128, page=16, parents=1, copies=3, length=500, spare=9),
        # eight samples of each of eight prompts
        dict(name="fork 8 into 56", op="fork", dtype="bf16", kv=8, dim=128, page=64, parents=8, copies=7, length=8100, spare=100),
        # a small pool in pieces
        dict(name="compact 300 pages", op="compact", dtype="f16", kv=2, dim=64, page=16, pages=300, used=170, requests=12),
        # a large one
        dict(name="compact 4000 pages", op="compact", dtype="bf16", kv=8, dim=128, page=64, pages=4000, used=2500, requests=64),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append4", "attend4", "attend4", "attend4", "attend", "attend", "fork", "compact"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "append4":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        turned = rng.random() < 0.6
        T = _spread(rng, 1, 4096)
        return dict(op=op, dtype=dtype, T=T, heads=kv * rng.choice([1, 2, 4, 7]) if turned else 0, kv=kv, dim=dim,
                    group=32 if turned else rng.choice([g for g in (32, 64, 128, 256) if g <= dim]), turned=turned,
                    far=T + _spread(rng, 16, 1000000), page=rng.choice([16, 32, 64, 128]))
    if op == "fork":
        page = rng.choice([16, 32, 64])
        return dict(op=op, dtype=dtype, kv=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 256]), page=page,
                    parents=_spread(rng, 1, 16), copies=_spread(rng, 1, 8), length=_spread(rng, 1, 6000),
                    spare=_spread(rng, 1, 150))
    if op == "compact":
        pages = _spread(rng, 40, 3000)
        return dict(op=op, dtype=dtype, kv=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]),
                    pages=pages, used=int(pages * rng.uniform(0.2, 0.95)), requests=_spread(rng, 1, 64))
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    B = _spread(rng, 1, 48)
    new = 1 if rng.random() < 0.5 else _spread(rng, 2, 1200)
    most = min(16384, (1 << 18) // B)
    # (scores of the padded batch stay within those of the largest listed case)
    while B * new * heads * most > 1 << 29 and most > 2 * new:
        most //= 2
    while B > 1 and B * new * heads * most > 1 << 29:
        B //= 2
    length = max(new, _spread(rng, 16, most))
    window = rng.choice([0, _spread(rng, 16, length)]) if op == "attend4" else _spread(rng, 16, length)
    return dict(op=op, dtype=dtype, heads=heads, kv=kv, dim=dim,
                group=rng.choice([g for g in (32, 64, 128, 256) if g <= dim]) if op == "attend4" else 0,
                page=rng.choice([16, 32, 64, 128]), B=B, new=new, length=length, window=window,
                sinks=rng.choice([1, 4, 16, 100]) if window and (op == "attend" or rng.random() < 0.5) else 0,
                ragged=B > 1 and rng.random() < 0.7)


# ----------------------------------------------------------------- inputs ---

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def _frequencies(dim):
    """Radians a position of each rotated pair."""
    return 10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64, device=DEV) / (dim // 2))


def _prepare_append(case, g):
    dt = DTYPES[case["dtype"]]
    T, H, kv, D, ps, G = (case[n] for n in ("T", "heads", "kv", "dim", "page", "group"))
    # q, k and v are views of the fused projection's rows
    fused = _normal(g, (T, (H + 2 * kv) * D), dt)
    q = fused[:, :H * D].view(T, H, D)
    k = fused[:, H * D:(H + kv) * D].view(T, kv, D)
    v = fused[:, (H + kv) * D:].view(T, kv, D)
    pos = (torch.arange(T, device=DEV) + int(torch.randint(0, case["far"] - T + 1, (1,), generator=g, device=DEV)))
    pages = -(-T // ps) + 3
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(T, device=DEV) + ps // 2
    slots = order[at // ps] * ps + at % ps
    s = dict(case=case, q=q, k=k, v=v, positions=pos, slots=slots)
    if own:
        import gptq_bit_weight_amd as q4
        s["cache"] = q4.PagedCache4.empty(pages, kv, ps, D, group=G)
        if case["turned"]:
            s["rotary"] = q4.Rotary(D)
    else:
        shape = (pages, kv, ps, D)
        s.update(codes=[torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2)],
                 scales=[torch.zeros(shape[:3] + (D // G, 2), dtype=torch.float16, device=DEV) for _ in range(2)],
                 freq=_frequencies(D))
    return s


def _attend_lengths(case):
    """New tokens and cached keys of each request."""
    B, new, length = case["B"], case["new"], case["length"]
    if not case["ragged"]:
        return [new] * B, [length] * B
    lens = [max(1, length - (length * 7 * i) // (8 * B)) for i in range(B)]
    news = [min(n, max(1, new - (new * i) // B) if i % 3 != 2 else 1) for i, n in enumerate(lens)]
    return news, lens


def _codes(g, shape, G):
    """A quantised cache: packed codes (two a byte, the first in the low half), and
    each group's scale and least value."""
    pages, kv, ps, D = shape
    packed = torch.empty((pages, kv, ps, D // 2), dtype=torch.uint8, device=DEV)
    for at in range(0, pages, 512):
        c = torch.randn((min(512, pages - at), kv, ps, D), generator=g, device=DEV).mul_(2.8).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        packed[at:at + 512] = c[..., 0::2] | c[..., 1::2] << 4
    step = torch.rand((pages, kv, ps, D // G), generator=g, device=DEV) * 0.2 + 0.25
    least = -step * (7.5 + torch.randn(step.shape, generator=g, device=DEV) * 0.5)
    return packed, torch.stack([step, least], -1).half()


def _prepare_attend(case, g):
    dt = DTYPES[case["dtype"]]
    H, kv, D, ps, G = case["heads"], case["kv"], case["dim"], case["page"], case["group"]
    news, lens = _attend_lengths(case)
    T, most = sum(news), max(lens)
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).tolist()
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    q = _normal(g, (T, H, D), dt)
    starts = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    s = dict(case=case, q=q, starts=starts.to(DEV), lengths=torch.tensor(lens, dtype=torch.int32, device=DEV),
             table=table.to(DEV))
    if G:
        s["k"], s["ks"] = _codes(g, (pages, kv, ps, D), G)
        s["v"], s["vs"] = _codes(g, (pages, kv, ps, D), G)
    else:
        s["k"], s["v"] = _normal(g, (pages, kv, ps, D), dt), _normal(g, (pages, kv, ps, D), dt)
    if own:
        import gptq_bit_weight_amd as q4
        s["cache"] = q4.PagedCache4(s["k"], s["v"], s["ks"], s["vs"]) if G else q4.PagedCache(s["k"], s["v"])
    else:
        s.update(most_new=max(news), most=most)
    return s


def _fork_lengths(case):
    return [max(1, case["length"] - (case["length"] * i) // (2 * case["parents"])) for i in range(case["parents"])]


def _prepare_fork(case, g):
    dt = DTYPES[case["dtype"]]
    kv, D, ps, n, m = case["kv"], case["dim"], case["page"], case["parents"], case["copies"]
    lens = _fork_lengths(case)
    need = [-(-x // ps) for x in lens]
    pages, R, width = sum(need) + case["spare"], n * (m + 1), max(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    who = torch.randperm(R, generator=g, device=DEV).to(torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32)
    lengths = torch.zeros(R, dtype=torch.int32)
    at = 0
    for r, x, k in zip(who[:n].tolist(), lens, need):
        table[r, :k] = order[at:at + k]
        lengths[r] = x
        at += k
    counts = torch.zeros(pages, dtype=torch.int32)
    counts[order[:at].long()] = 1
    s = dict(case=case, parents=who[:n].repeat_interleave(m), children=who[n:], k=_normal(g, (pages, kv, ps, D), dt),
             v=_normal(g, (pages, kv, ps, D), dt))
    return _hold(s, table, lengths, counts)


def _prepare_compact(case, g):
    dt = DTYPES[case["dtype"]]
    kv, D, ps, P, U, R = case["kv"], case["dim"], case["page"], case["pages"], case["used"], case["requests"]
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32).cpu()[:U]
    # the first page of every request is the same one (a prompt that they have in common)
    edges = [1 + (U - 1) * i // R for i in range(R + 1)]
    width = 1 + max(edges[i + 1] - edges[i] for i in range(R))
    table = torch.full((R, width), -1, dtype=torch.int32)
    lengths = torch.zeros(R, dtype=torch.int32)
    counts = torch.zeros(P, dtype=torch.int32)
    for i in range(R):
        mine = torch.cat([order[:1], order[edges[i]:edges[i + 1]]])
        table[i, :mine.numel()] = mine
        lengths[i] = mine.numel() * ps - i % ps
        counts[mine.long()] += 1
    s = dict(case=case, k=_normal(g, (P, kv, ps, D), dt), v=_normal(g, (P, kv, ps, D), dt))
    s = _hold(s, table, lengths, counts)
    s.update(table0=s["table"].clone(), counts0=s["counts"].clone())
    return s


def _hold(s, table, lengths, counts):
    """The bookkeeping on the GPU: with the package's operators, in its Pages."""
    if own:
        import gptq_bit_weight_amd as q4
        s["cache"] = q4.PagedCache(s["k"], s["v"])
        s["pages"] = q4.Pages(s["cache"], *table.shape)
        for to, t in ((s["pages"].table, table), (s["pages"].lengths, lengths), (s["pages"].counts, counts)):
            to.copy_(t)
        s.update(table=s["pages"].table, lengths=s["pages"].lengths, counts=s["pages"].counts)
    else:
        s.update(table=table.to(DEV), lengths=lengths.to(DEV), counts=counts.to(DEV))
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"append4": _prepare_append, "fork": _prepare_fork, "compact": _prepare_compact}.get(case["op"], _prepare_attend)(case, g)


# ------------------------------------------------------------ plain forms ---

def _plain_turn(x, s):
    n = x.shape[-1] // 2
    ang = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = x[..., :n].float(), x[..., n:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _plain_quantise(x, G):
    """Codes [.., dim], and scales and least values [.., groups, 2]. In 64 bits:
    a value half way between two codes has to go to the even one."""
    y = x.double().clamp(-LARGEST, LARGEST).unflatten(-1, (-1, G))
    least = y.amin(-1).half()
    step = ((y.amax(-1) - least.double()).float() / 15).half()
    c = torch.round((y - least.double()[..., None]) / step.double()[..., None].clamp_min(2.0 ** -30)).clamp(0, 15)
    c = torch.where(step[..., None] == 0, 0.0, c)
    return c.flatten(-2).to(torch.uint8), torch.stack([step, least], -1)


def _plain_values(codes, scales):
    """What codes [.., dim] stand for, in binary16."""
    c = codes.float().unflatten(-1, (scales.shape[-2], -1))
    return (c * scales[..., :1].float() + scales[..., 1:].float()).flatten(-2).half()


def _plain_append(s):
    case = s["case"]
    ps = case["page"]
    page, off = s["slots"] // ps, s["slots"] % ps
    k = _plain_turn(s["k"], s) if case["turned"] else s["k"]
    out = {"q": _plain_turn(s["q"], s)} if case["turned"] else {}
    for name, x, codes, scales in zip("kv", (k, s["v"]), s["codes"], s["scales"]):
        codes[page, :, off], scales[page, :, off] = _plain_quantise(x, case["group"])
        out[name] = _plain_values(codes[page, :, off], scales[page, :, off])
    return out


def _plain_rows(s, name, page, row):
    """Keys or values [B, most, kv, dim] in 32 bits."""
    x = s[name][page, :, row]
    if not s["case"]["group"]:
        return x.float()
    c = torch.stack([x & 15, x >> 4], -1).flatten(-2)
    return _plain_values(c, s[name + "s"][page, :, row]).float()


def _plain_attend(s):
    case, most_new, most = s["case"], s["most_new"], s["most"]
    kv, D, ps = case["kv"], case["dim"], case["page"]
    g = case["heads"] // kv
    starts, lens = s["starts"].long(), s["lengths"].long()
    n = starts[1:] - starts[:-1]
    B = lens.numel()
    # requests padded to the longest: queries [B, kv, g * new, D], keys [B, kv, most, D]
    i = torch.arange(most_new, device=DEV)
    real = i < n[:, None]
    row = torch.where(real, starts[:-1, None] + i, 0)
    q = s["q"].float()[row].reshape(B, most_new, kv, g, D).permute(0, 2, 3, 1, 4).reshape(B, kv, g * most_new, D)
    j = torch.arange(most, device=DEV)
    page = s["table"].long()[:, j // ps]
    k = _plain_rows(s, "k", page, j % ps).permute(0, 2, 3, 1)          # [B, kv, D, most]
    v = _plain_rows(s, "v", page, j % ps).transpose(1, 2)              # [B, kv, most, D]
    pos = (lens - n)[:, None] + i                                      # [B, new]
    see = (j <= pos[:, :, None]) & (j < lens[:, None, None])
    if case["window"]:
        see = see & ((j > pos[:, :, None] - case["window"]) | (j < case["sinks"]))
    sc = (q @ k.contiguous()).reshape(B, kv, g, most_new, most) * D ** -0.5
    sc = sc.masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.reshape(B, kv, g * most_new, most) @ v.contiguous()
    o = o.reshape(B, kv, g, most_new, D).permute(0, 3, 1, 2, 4).reshape(B, most_new, kv * g, D)
    return o[real].to(s["q"].dtype)


def _held(s, who):
    """Pages of the requests `who`: their table rows, and which entries hold a page."""
    need = -(-s["lengths"].long()[who] // s["case"]["page"])
    rows = s["table"].long()[who]
    return need, rows, torch.arange(rows.shape[1], device=DEV) < need[:, None]


def _plain_fork(s):
    ps, table, lengths, counts = s["case"]["page"], s["table"], s["lengths"], s["counts"]
    R, P = lengths.numel(), counts.numel()
    par, chi = s["parents"].long(), s["children"].long()
    i = torch.arange(par.numel(), device=DEV)
    # a pair counts if its child is empty and no pair before it names the child
    first = torch.full((R,), par.numel(), device=DEV).scatter_reduce_(0, chi, i, "amin")
    fine = (first[chi] == i) & (lengths[chi] == 0)
    need, rows, held = _held(s, par)
    tail = fine & (lengths[par] % ps != 0)
    rank = torch.cumsum(tail, 0) - 1
    free = torch.cat([(counts <= 0).nonzero()[:, 0], torch.zeros(1, dtype=torch.int64, device=DEV)])
    done = fine & (~tail | (rank < free.numel() - 1))
    new = free[rank.clamp(0, free.numel() - 1)]
    tail = tail & done
    last = rows.gather(1, (need - 1).clamp_min(0)[:, None])[:, 0]
    src, dst = last[tail], new[tail]
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    rows = torch.where(tail[:, None] & (torch.arange(rows.shape[1], device=DEV) == need[:, None] - 1), new[:, None], rows)
    held = held & done[:, None]
    counts += torch.bincount(rows[held & (rows >= 0)], minlength=P).int()
    table[chi[done]] = torch.where(held, rows, table.long()[chi])[done].int()
    lengths[chi[done]] = lengths[par][done]
    _plain_free(s, chi)
    return done.int()


def _plain_free(s, who):
    # (of a request named twice the same is freed once)
    who = torch.unique(who)
    _, rows, held = _held(s, who)
    gone = held & (rows >= 0)
    s["counts"] -= torch.bincount(rows[gone], minlength=s["counts"].numel()).int()
    s["table"][who] = torch.where(held, -1, rows).int()
    s["lengths"][who] = 0


def _plain_compact(s):
    used = s["counts"] > 0
    P = used.numel()
    i = torch.arange(P, device=DEV)
    low = i < used.sum()
    src, dst = (used & ~low).nonzero()[:, 0], (~used & low).nonzero()[:, 0]
    to = torch.where(used, i, -1)
    to[src] = dst
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    s["counts"][dst] = s["counts"][src]
    s["counts"][src] = 0
    _, rows, held = _held(s, torch.arange(s["table"].shape[0], device=DEV))
    s["table"].copy_(torch.where(held & (rows >= 0), to[rows.clamp_min(0)], rows))
    return to.int()


def _books(s, more):
    return dict(more, table=s["table"], lengths=s["lengths"], counts=s["counts"], k=s["k"], v=s["v"])


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "append4":
        if not own:
            return _plain_append(s)
        if case["turned"]:
            q = s["cache"].append(s["k"], s["v"], s["slots"], rotary=s["rotary"], positions=s["positions"], q=s["q"])
            out = {"q": q}
        else:
            s["cache"].append(s["k"], s["v"], s["slots"])
            out = {}
        out["k"], out["v"] = s["cache"].read(s["slots"])
        return out
    if op == "fork":
        if not own:
            return _books(s, {"done": _plain_fork(s)})
        done = s["pages"].fork(s["parents"], s["children"])
        s["pages"].free(s["children"])
        return _books(s, {"done": done})
    if op == "compact":
        # the pool in pieces again (its pages that moved are still where they were)
        s["table"].copy_(s["table0"])
        s["counts"].copy_(s["counts0"])
        return _books(s, {"to": s["pages"].compact() if own else _plain_compact(s)})
    if not own:
        return _plain_attend(s)
    return s["cache"].attend(s["q"], s["starts"], s["lengths"], s["table"], window=case["window"], sinks=case["sinks"])


def work(case):
    op = case["op"]
    if op == "append4":
        T, H, kv, D, G = (case[n] for n in ("T", "heads", "kv", "dim", "group"))
        rows = T * kv * 2
        packed = D // 2 + 4 * (D // G)
        # q turned; k and v quantised; the rows read back
        return {"bytes": 4 * T * H * D + rows * (2 * D + packed) + rows * (packed + 2 * D) + 16 * T,
                "flops": 6 * T * (H + kv) * D // 2 + 8 * rows * D}
    if op == "fork":
        page = 2 * 2 * case["kv"] * case["page"] * case["dim"]
        lens, ps, m = _fork_lengths(case), case["page"], case["copies"]
        tails = min(sum(m for x in lens if x % ps), case["spare"])
        entries = sum(m * -(-x // ps) for x in lens)
        return {"bytes": 2 * tails * page + 4 * 4 * entries, "flops": 0}
    if op == "compact":
        page = 2 * 2 * case["kv"] * case["page"] * case["dim"]
        P, U = case["pages"], case["used"]
        return {"bytes": 2 * (U * (P - U) // P) * page + 8 * U + 8 * P, "flops": 0}
    H, kv, D, w, sinks, G = (case[n] for n in ("heads", "kv", "dim", "window", "sinks", "group"))
    news, lens = _attend_lengths(case)
    pairs = keys = 0
    for n, m in zip(news, lens):
        if w:
            # (a token at p sees min(p + 1, window) keys, and the sinks before those)
            pairs += sum(min(p + 1, w + min(sinks, max(0, p + 1 - w))) for p in range(m - n, m))
            keys += min(m, n + w - 1 + min(sinks, max(0, m - n - w + 1)))
        else:
            pairs += (m - n + 1 + m) * n // 2
            keys += m
    row = D // 2 + 4 * (D // G) if G else 2 * D
    return {"bytes": 2 * keys * kv * row + 4 * sum(news) * H * D, "flops": 4 * pairs * H * D}


# ------------------------------------------------------------ definitions ---

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append4": _exact_append, "fork": _exact_fork, "compact": _exact_compact}.get(case["op"], _exact_attend)(s)


def _exact_turned(x, s):
    n = x.shape[-1] // 2
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV), s["positions"].double()[:, None] * s["freq"])[:, None]
    z = torch.complex(x[..., :n].double(), x[..., n:].double()) * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_held(x, G):
    """What the cache stands for after x (of the cache's 16-bit type) was written."""
    shape = x.shape
    y = x.double().reshape(-1, G).clamp(-LARGEST, LARGEST)
    least = y.min(1, keepdim=True).values.half().double()
    step = ((y.max(1, keepdim=True).values - least) / 15).float().half().double()
    code = ((y - least) / torch.where(step > 0, step, 1.0)).round().clamp(0, 15)
    return (least + step * torch.where(step > 0, code, 0.0)).half().double().reshape(shape)


def _exact_append(s):
    case = s["case"]
    out = {}
    k = s["k"]
    if case["turned"]:
        out["q"] = _exact_turned(s["q"], s)
        k = _exact_turned(k, s).to(k.dtype)
    return dict(out, k=_exact_held(k, case["group"]), v=_exact_held(s["v"], case["group"]))


def _exact_cached(s, name, pages, m):
    """[kv, m, dim] of one request."""
    case = s["case"]
    x = s[name][pages]
    if case["group"]:
        sc = s[name + "s"][pages].double()
        both = torch.empty(x.shape[:-1] + (case["dim"],), dtype=torch.float64, device=DEV)
        both[..., 0::2], both[..., 1::2] = (x % 16).double(), (x // 16).double()
        each = sc.repeat_interleave(case["group"], -2)
        x = (each[..., 0] * both + each[..., 1]).half()
    return x.double().transpose(0, 1).reshape(case["kv"], -1, case["dim"])[:, :m]


def _exact_attend(s):
    case = s["case"]
    ps, D, g = case["page"], case["dim"], case["heads"] // case["kv"]
    news, lens = _attend_lengths(case)
    out, at = [], 0
    for b, (n, m) in enumerate(zip(news, lens)):
        pages = s["table"][b, :-(-m // ps)].long()
        k, v = (_exact_cached(s, c, pages, m) for c in "kv")
        q = s["q"][at:at + n].double()
        at += n
        i, j = torch.arange(m - n, m, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
        hide = j > i
        if case["window"]:
            hide = hide | ((j <= i - case["window"]) & (j >= case["sinks"]))
        heads = []
        for h in range(case["heads"]):
            sc = q[:, h] @ k[h // g].t() / math.sqrt(D)
            heads.append(torch.softmax(sc.masked_fill(hide, -math.inf), -1) @ v[h // g])
        out.append(torch.stack(heads, 1))
    return torch.cat(out)


def _exact_fork(s):
    ps, table, lengths = s["case"]["page"], s["table"].tolist(), s["lengths"].tolist()
    counts = s["counts"].tolist()
    k, v = s["k"].double(), s["v"].double()
    free = [p for p, c in enumerate(counts) if c <= 0]
    done, made = [], {}
    for r, c in zip(s["parents"].tolist(), s["children"].tolist()):
        ok = lengths[c] == 0 and c not in made
        if ok and lengths[r] % ps:
            ok = bool(free)
            if ok:
                new, old = free.pop(0), table[r][lengths[r] // ps]
                k[new], v[new] = s["k"][old].double(), s["v"][old].double()
        if ok:
            made[c] = r
        done.append(int(ok))
    # the children are freed again: no count changes, their entries name no page
    for c in s["children"].tolist():
        n = lengths[made[c]] if c in made else lengths[c]
        for e in range(-(-n // ps)):
            table[c][e] = -1
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"done": ints(done), "table": ints(table), "lengths": s["lengths"], "counts": ints(counts), "k": k, "v": v}


def _exact_compact(s):
    ps, table, counts = s["case"]["page"], s["table"].tolist(), s["counts"].tolist()
    U = sum(c > 0 for c in counts)
    holes = iter([p for p in range(U) if counts[p] <= 0])
    to = [(p if p < U else next(holes)) if counts[p] > 0 else -1 for p in range(len(counts))]
    k, v, after = s["k"].double(), s["v"].double(), [0] * len(counts)
    for p, t in enumerate(to):
        if t >= 0:
            after[t] = counts[p]
            if t != p:
                k[t], v[t] = s["k"][p].double(), s["v"][p].double()
    for row, n in zip(table, s["lengths"].tolist()):
        for e in range(-(-n // ps)):
            row[e] = to[row[e]] if row[e] >= 0 else row[e]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"to": ints(to), "table": ints(table), "lengths": s["lengths"], "counts": ints(after), "k": k, "v": v}
