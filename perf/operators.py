"""Cases, plain forms and inputs of the operators around a quantized
projection: the adapters of many requests beside it, rotary positions (with
the write to the paged cache), and attention of new tokens over that cache.

``own`` selects what run() calls: the plain form in elementary torch
operations, or this package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one request's token through the attention output projection
        dict(name="adapters 1 row", op="adapters", dtype="f16", K=4096, parts="4096", G=128, M=1, slots=4,
             rank=16, spread="runs", none=0, act=False),
        # a decode step of 32 requests, an adapter each, over the fused q/k/v projection
        dict(name="adapters 32 requests qkv", op="adapters", dtype="bf16", K=4096, parts="4096,4096,4096",
             G=128, M=32, slots=64, rank=16, spread="rows", none=3, act=False),
        # short prompts and single tokens mixed in one batch, over an act-order layer
        dict(name="adapters mixed 77 rows", op="adapters", dtype="f16", K=4096, parts="11008", G=128, M=77,
             slots=12, rank=32, spread="runs", none=9, act=True),
        # a batch of prompts through the MLP's up projection
        dict(name="adapters prompts 2048 rows", op="adapters", dtype="f16", K=4096, parts="11008", G=128,
             M=2048, slots=8, rank=64, spread="runs", none=100, act=False),
        # one decode step of eight requests: rotate q and k, write k and v to the cache
        dict(name="rotary append 8 tokens", op="append", dtype="f16", T=8, heads=32, kv=32, dim=128, rot=128,
             layout="half", scaling="none", far=4096, page=16),
        # a long prompt's chunk, far into a long context
        dict(name="rotary append 16384 tokens", op="append", dtype="bf16", T=16384, heads=64, kv=8, dim=128,
             rot=128, layout="half", scaling="by_parts", far=131072, page=64),
        # part of the head, interleaved pairs, an odd number of tokens at positions near a million;
        # and the gradient's pass over the same
        dict(name="rotary part of head 1003", op="rotate", dtype="bf16", T=1003, heads=32, kv=0, dim=128,
             rot=64, layout="interleaved", scaling="linear", far=1000000, page=0),
        # a token of one request
        dict(name="attend 1 token over 500", op="attend", dtype="f16", heads=32, kv=32, dim=128, page=16,
             B=1, new=1, length=500, window=0, ragged=False),
        # a decode step of 64 requests of different lengths, grouped heads
        dict(name="attend 64 x 1 over 8192", op="attend", dtype="bf16", heads=64, kv=8, dim=128, page=64,
             B=64, new=1, length=8192, window=0, ragged=True),
        # a token at the end of one long context
        dict(name="attend 1 token over 131000", op="attend", dtype="bf16", heads=64, kv=8, dim=128, page=64,
             B=1, new=1, length=131000, window=0, ragged=False),
        # chunks of several prompts beside single tokens, sliding window
        dict(name="attend 6 chunks window", op="attend", dtype="f16", heads=32, kv=8, dim=64, page=16,
             B=6, new=701, length=4096, window=1024, ragged=True),
        # a chunk of a long prompt
        dict(name="attend 4096 over 8192", op="attend", dtype="bf16", heads=32, kv=8, dim=128, page=64,
             B=1, new=4096, length=8192, window=0, ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "append", "rotate", "attend", "attend", "attend"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "adapters":
        G = rng.choice([32, 64, 128])
        K = G * _spread(rng, max(1, 512 // G), 11008 // G)
        if rng.random() < 0.3:
            n = 8 * _spread(rng, 16, 512)
            parts = [n, 8 * _spread(rng, 8, 256), 8 * _spread(rng, 8, 256)]
        else:
            parts = [8 * _spread(rng, 16, 1376)]
        M = _spread(rng, 1, 1500)
        slots = _spread(rng, 1, 48)
        return dict(op=op, dtype=dtype, K=K, parts=",".join(map(str, parts)), G=G, M=M, slots=slots,
                    rank=rng.choice([4, 8, 16, 24, 32, 64]), spread=rng.choice(["runs", "rows"]),
                    none=_spread(rng, 1, M) // 3, act=rng.random() < 0.25)
    if op in ("append", "rotate"):
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        T = _spread(rng, 1, 4096)
        return dict(op=op, dtype=dtype, T=T, heads=kv * rng.choice([1, 2, 4, 7]), kv=kv if op == "append" else 0,
                    dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "by_parts"]),
                    far=T + _spread(rng, 16, 1000000), page=rng.choice([16, 32, 64, 128]) if op == "append" else 0)
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
    return dict(op=op, dtype=dtype, heads=heads, kv=kv, dim=dim, page=rng.choice([16, 32, 64, 128]), B=B,
                new=new, length=length, window=rng.choice([0, 0, 0, _spread(rng, 16, length)]),
                ragged=B > 1 and rng.random() < 0.7)


# ----------------------------------------------------------------- inputs ---

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def _frequencies(case):
    """Radians a position of each rotated pair, and the factor on the result."""
    n, base, f = case["rot"] // 2, 10000.0, 8.0
    kind = case["scaling"]
    if kind == "base":
        base *= f ** (case["rot"] / (case["rot"] - 2.0))
    freq = base ** (-torch.arange(n, dtype=torch.float64) / n)
    if kind == "linear":
        freq = freq / f
    if kind == "by_parts":
        # pairs that turn often within the original length keep their
        # frequency, slow ones are stretched, a ramp between
        turns = 4096.0 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        freq = freq * keep + freq / f * (1 - keep)
        return freq, 0.1 * math.log(f) + 1.0
    return freq, 1.0


def _scaling(case):
    """The same scaling in this package's terms."""
    return {"none": None, "linear": dict(kind="linear", factor=8.0), "base": dict(kind="base", factor=8.0),
            "by_parts": dict(kind="by_parts", factor=8.0, original_length=4096, low=1.0, high=32.0)}[case["scaling"]]


def _prepare_adapters(case, g):
    dt = DTYPES[case["dtype"]]
    K, G, M, S, r = case["K"], case["G"], case["M"], case["slots"], case["rank"]
    ns = [int(n) for n in case["parts"].split(",")]
    N, ng = sum(ns), K // G
    words = lambda shape: torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)  # noqa: E731
    qweight = [words((K // 8, n)) for n in ns]
    qzeros = [words((ng, n // 8)) for n in ns]
    scales = [(torch.rand((ng, n), generator=g, device=DEV) * 0.015 + 0.005).half() for n in ns]
    g_idx = None
    if case["act"]:
        order = torch.randperm(K, generator=g, device=DEV)
        g_idx = torch.empty(K, dtype=torch.int32, device=DEV)
        g_idx[order] = (torch.arange(K, device=DEV) // G).to(torch.int32)
    x = _normal(g, (M, K), dt)
    bias = _normal(g, (N,), dt, 0.1)
    A = _normal(g, (S, len(ns), r, K), dt, K ** -0.5)
    B = _normal(g, (S, N, r), dt, 0.1)
    c = torch.rand((S,), generator=g, device=DEV) * 2 + 0.5
    if case["spread"] == "rows":
        index = torch.randperm(max(S, M), generator=g, device=DEV)[:M] % S
    else:   # runs of rows, one request's prompt each
        index = torch.sort(torch.randint(0, S, (M,), generator=g, device=DEV)).values
    index = index.to(torch.int32)
    index[torch.randperm(M, generator=g, device=DEV)[:case["none"]]] = -1
    s = dict(case=case, x=x, bias=bias, index=index)
    if own:
        import gptq_bit_weight_amd as q4
        s["W"] = q4.Q4Matrix.concat(list(zip(qweight, qzeros, scales)), g_idx, groupsize=G)
        s["bank"] = q4.Q4Adapters(s["W"], slots=S, rank=r, dtype=dt)
        for i, ci in enumerate(c.tolist()):
            s["bank"].load(i, A[i], B[i], ci)
        return s
    part = torch.cat([torch.full((n,), i, device=DEV) for i, n in enumerate(ns)])
    group = g_idx.long() if g_idx is not None else torch.arange(K, device=DEV) // G
    return dict(s, qweight=torch.cat(qweight, 1), qzeros=torch.cat(qzeros, 1), scales=torch.cat(scales, 1),
                group=group, A=A, B=B, c=c, part=part)


def _prepare_append(case, g):
    dt = DTYPES[case["dtype"]]
    T, H, kv, D, ps = case["T"], case["heads"], case["kv"], case["dim"], case["page"]
    # q, k and v are views of the fused projection's rows
    fused = _normal(g, (T, (H + 2 * kv) * D), dt)
    q = fused[:, :H * D].view(T, H, D)
    pos = (torch.arange(T, device=DEV) + int(torch.randint(0, case["far"] - T + 1, (1,), generator=g, device=DEV)))
    freq, mag = _frequencies(case)
    s = dict(case=case, q=q, positions=pos)
    if kv:
        k = fused[:, H * D:(H + kv) * D].view(T, kv, D)
        v = fused[:, (H + kv) * D:].view(T, kv, D)
        pages = -(-T // ps) + 3
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + ps // 2
        slots = order[at // ps] * ps + at % ps
        kc = _normal(g, (pages, kv, ps, D), dt)
        vc = _normal(g, (pages, kv, ps, D), dt)
        s.update(k=k, v=v, slots=slots, kc=kc, vc=vc)
    if own:
        import gptq_bit_weight_amd as q4
        s["rotary"] = q4.Rotary(D, case["rot"], layout=case["layout"], scaling=_scaling(case))
        if kv:
            s["cache"] = q4.PagedCache(kc, vc)
    else:
        s.update(freq=freq.to(DEV), mag=mag)
    return s


def _attend_lengths(case):
    """New tokens and cached keys of each request."""
    B, new, length = case["B"], case["new"], case["length"]
    if not case["ragged"]:
        return [new] * B, [length] * B
    lens = [max(1, length - (length * 7 * i) // (8 * B)) for i in range(B)]
    news = [min(n, max(1, new - (new * i) // B) if i % 3 != 2 else 1) for i, n in enumerate(lens)]
    return news, lens


def _prepare_attend(case, g):
    dt = DTYPES[case["dtype"]]
    H, kv, D, ps = case["heads"], case["kv"], case["dim"], case["page"]
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
    kc = _normal(g, (pages, kv, ps, D), dt)
    vc = _normal(g, (pages, kv, ps, D), dt)
    starts = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    s = dict(case=case, q=q, starts=starts.to(DEV), lengths=torch.tensor(lens, dtype=torch.int32, device=DEV),
             table=table.to(DEV), kc=kc, vc=vc)
    if own:
        import gptq_bit_weight_amd as q4
        s["cache"] = q4.PagedCache(kc, vc)
    else:
        s.update(most_new=max(news), most=most)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "adapters":
        return _prepare_adapters(case, g)
    if case["op"] == "attend":
        return _prepare_attend(case, g)
    return _prepare_append(case, g)


# ------------------------------------------------------------ plain forms ---

def _dequant(s):
    shifts = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    qw, qz = s["qweight"], s["qzeros"]
    q = ((qw[:, None, :] >> shifts[None, :, None]) & 15).reshape(-1, qw.shape[1])
    z = ((qz[:, :, None] >> shifts) & 15).reshape(qz.shape[0], -1)
    return s["scales"].float()[s["group"]] * (q - z[s["group"]]).float()


def _plain_adapters(s):
    x, A, B, idx = s["x"].float(), s["A"].float(), s["B"].float(), s["index"].long()
    S, P, r, K = A.shape
    t = (x @ A.reshape(-1, K).t()).reshape(-1, S, P * r)
    mine = (idx[:, None] == torch.arange(S, device=DEV)).float() * s["c"]
    t = (t * mine[:, :, None]).reshape(-1, S * P * r)
    in_part = (s["part"] == torch.arange(P, device=DEV)[:, None]).float()          # [P, N]
    b = (B.transpose(1, 2)[:, None] * in_part[None, :, None, :]).reshape(S * P * r, -1)
    return (x @ _dequant(s) + t @ b + s["bias"].float()).to(s["x"].dtype)


def _plain_rotate(x, s, sign=1.0):
    case = s["case"]
    rot, n = case["rot"], case["rot"] // 2
    ang = s["positions"].double()[:, None] * s["freq"]
    cos, sin = (ang.cos() * s["mag"]).float()[:, None], (ang.sin() * (s["mag"] * sign)).float()[:, None]
    f = x.float()
    if case["layout"] == "half":
        a, b = f[..., :n], f[..., n:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, f[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    if not s["case"]["kv"]:
        return {"y": _plain_rotate(s["q"], s), "back": _plain_rotate(s["q"], s, -1.0)}
    ps = s["case"]["page"]
    page, off = s["slots"] // ps, s["slots"] % ps
    s["kc"][page, :, off] = _plain_rotate(s["k"], s)
    s["vc"][page, :, off] = s["v"]
    return {"q": _plain_rotate(s["q"], s), "k": s["kc"], "v": s["vc"]}


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
    k = s["kc"][page, :, j % ps].float().permute(0, 2, 3, 1)          # [B, kv, D, most]
    v = s["vc"][page, :, j % ps].float().transpose(1, 2)              # [B, kv, most, D]
    pos = (lens - n)[:, None] + i                                     # [B, new]
    see = (j <= pos[:, :, None]) & (j < lens[:, None, None])
    if case["window"]:
        see = see & (j > pos[:, :, None] - case["window"])
    sc = (q @ k.contiguous()).reshape(B, kv, g, most_new, most) * D ** -0.5
    sc = sc.masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.reshape(B, kv, g * most_new, most) @ v.contiguous()
    o = o.reshape(B, kv, g, most_new, D).permute(0, 3, 1, 2, 4).reshape(B, most_new, kv * g, D)
    return o[real].to(s["q"].dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"adapters": _plain_adapters, "attend": _plain_attend}.get(op, _plain_append)(s)
    if op == "adapters":
        return s["W"].matmul_adapters(s["x"], s["bank"], s["index"], s["bias"])
    if op == "attend":
        return s["cache"].attend(s["q"], s["starts"], s["lengths"], s["table"], window=s["case"]["window"])
    if op == "rotate":
        return {"y": s["rotary"].rotate(s["q"], s["positions"]),
                "back": s["rotary"].rotate(s["q"], s["positions"], transpose=True)}
    q = s["cache"].append(s["k"], s["v"], s["slots"], rotary=s["rotary"], positions=s["positions"], q=s["q"])
    return {"q": q, "k": s["kc"], "v": s["vc"]}


def work(case):
    if case["op"] == "adapters":
        K, M, r = case["K"], case["M"], case["rank"]
        ns = [int(n) for n in case["parts"].split(",")]
        N, P, ng = sum(ns), len(ns), K // case["G"]
        used = min(case["slots"], M)
        return {"bytes": K * N // 2 + ng * N * 2.5 + 2 * (M * K + M * N + N) + 2 * used * r * (P * K + N),
                "flops": 2 * M * K * N + 2 * M * r * (P * K + N)}
    if case["op"] == "attend":
        H, kv, D, w = case["heads"], case["kv"], case["dim"], case["window"]
        news, lens = _attend_lengths(case)
        pairs = keys = 0
        for n, m in zip(news, lens):
            first, last = m - n, m - 1       # positions of the request's queries
            full = (first + 1 + last + 1) * n // 2
            if w:
                over = lambda p: max(0, p + 1 - w)  # noqa: E731  keys before the window
                cut = (over(first) + over(last)) * (min(n, over(last)) if over(first) == 0 else n) // 2
                full -= cut
            pairs += full
            keys += min(m, n + w - 1) if w else m
        return {"bytes": 2 * (2 * keys * kv * D + 2 * sum(news) * H * D), "flops": 4 * pairs * H * D}
    T, H, kv, D = case["T"], case["heads"], case["kv"], case["dim"]
    if not kv:   # the rotation and its gradient's pass, over the same input
        return {"bytes": 2 * 3 * T * H * D + 8 * T, "flops": 12 * T * H * case["rot"] // 2}
    return {"bytes": 2 * 2 * T * (H + 2 * kv) * D + 16 * T, "flops": 6 * T * (H + kv) * case["rot"] // 2}


# ------------------------------------------------------------ definitions ---

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"adapters": _exact_adapters, "attend": _exact_attend}.get(case["op"], _exact_append)(s)


def _exact_adapters(s):
    case = s["case"]
    K, N = case["K"], s["scales"].shape[1]
    k, n = torch.arange(K, device=DEV)[:, None], torch.arange(N, device=DEV)[None, :]
    code = (s["qweight"].long()[k // 8, n] // 16 ** (k % 8)) % 16
    zero = (s["qzeros"].long()[s["group"][:, None], n // 8] // 16 ** (n % 8)) % 16
    w = (code - zero).double().mul_(s["scales"].double()[s["group"]])
    x = s["x"].double()
    y = x @ w + s["bias"].double()
    edges = [0]
    for m in case["parts"].split(","):
        edges.append(edges[-1] + int(m))
    for a in range(case["slots"]):
        rows = (s["index"] == a).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        for p in range(len(edges) - 1):
            t = x[rows] @ s["A"][a, p].double().t() * s["c"][a].double()
            y[rows, edges[p]:edges[p + 1]] += t @ s["B"][a, edges[p]:edges[p + 1]].double().t()
    return y


def _exact_rotated(x, s, back=False):
    case = s["case"]
    n = case["rot"] // 2
    turn = torch.polar(torch.full((1,), s["mag"], dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * s["freq"])[:, None]
    if back:
        turn = turn.conj()
    d = x.double().clone()
    first = slice(0, n) if case["layout"] == "half" else slice(0, 2 * n, 2)
    second = slice(n, 2 * n) if case["layout"] == "half" else slice(1, 2 * n, 2)
    z = torch.complex(d[..., first].contiguous(), d[..., second].contiguous()) * turn
    d[..., first], d[..., second] = z.real, z.imag
    return d


def _exact_append(s):
    if not s["case"]["kv"]:
        return {"y": _exact_rotated(s["q"], s), "back": _exact_rotated(s["q"], s, True)}
    ps = s["case"]["page"]
    k, v = s["kc"].double(), s["vc"].double()
    k[s["slots"] // ps, :, s["slots"] % ps] = _exact_rotated(s["k"], s)
    v[s["slots"] // ps, :, s["slots"] % ps] = s["v"].double()
    return {"q": _exact_rotated(s["q"], s), "k": k, "v": v}


def _exact_attend(s):
    case = s["case"]
    ps, D, g = case["page"], case["dim"], case["heads"] // case["kv"]
    news, lens = _attend_lengths(case)
    out, at = [], 0
    for b, (n, m) in enumerate(zip(news, lens)):
        pages = s["table"][b, :-(-m // ps)].long()
        k, v = (c[pages].double().transpose(0, 1).reshape(case["kv"], -1, D)[:, :m] for c in (s["kc"], s["vc"]))
        q = s["q"][at:at + n].double()
        at += n
        i, j = torch.arange(m - n, m, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
        hide = (j > i) | (j <= i - case["window"]) if case["window"] else j > i
        heads = []
        for h in range(case["heads"]):
            sc = q[:, h] @ k[h // g].t() / math.sqrt(D)
            heads.append(torch.softmax(sc.masked_fill(hide, -math.inf), -1) @ v[h // g])
        out.append(torch.stack(heads, 1))
    return torch.cat(out)
