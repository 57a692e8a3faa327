"""A cache held in 4 bits, from its definition in 64 bits, and attention with
sinks over values."""
import math

import torch

LARGEST = 65440.0


def quantise(x, G):
    """Codes [.., dim], steps and least values [.., dim / G] (float64) of 16-bit x."""
    y = x.double()
    fine = y.isfinite().unflatten(-1, (-1, G)).all(-1)
    y = torch.nan_to_num(y, 0.0, 0.0, 0.0).clamp(-LARGEST, LARGEST).unflatten(-1, (-1, G))
    least = y.amin(-1).half().double()
    step = ((y.amax(-1) - least).float() / 15).half().double()
    code = torch.round((y - least[..., None]) / torch.where(step > 0, step, 1.0)[..., None]).clamp(0, 15)
    code = torch.where((step > 0)[..., None] & fine[..., None], code, 0.0)
    nan = torch.tensor(math.nan, dtype=torch.float64, device=x.device)
    return code.flatten(-2), torch.where(fine, step, nan), torch.where(fine, least, nan)


def to_half(x):
    """float64 rounded once to binary16, in float64 (a cast rounds to float32 first)."""
    y = x.half().double()
    # (the cast is off by one place at most: its neighbours in binary16 are looked at)
    ulp = torch.where(y.abs() < 2.0 ** -14, 2.0 ** -24, torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -14))) - 10))
    best = y
    for s in (-1.0, 1.0):
        z = y + s * ulp
        closer = (x - z).abs() < (x - best).abs()
        best = torch.where(closer, z, best)
    return torch.where(y.isfinite(), best, y)


def values(code, step, least):
    """What codes stand for: RNE(s c + m), in float64."""
    c = code.unflatten(-1, (step.shape[-1], -1))
    return to_half(c * step[..., None] + least[..., None]).flatten(-2)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def turned(x, positions, rot, layout, base=10000.0):
    """Keys turned in 64 bits, rounded through float32 to their type."""
    n = rot // 2
    freq = base ** (-torch.arange(n, dtype=torch.float64, device=x.device) / n)
    ang = (positions.double()[:, None] * freq)[:, None]
    d = x.double().clone()
    a, b = (slice(0, n), slice(n, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    p, q = d[..., a].clone(), d[..., b].clone()
    d[..., a], d[..., b] = p * ang.cos() - q * ang.sin(), q * ang.cos() + p * ang.sin()
    return d.float().to(x.dtype)


def attention(q, k, v, news, lens, window=0, sinks=0, scale=None, weights=None):
    """(result, tolerance) in float64: k and v are lists of [kv, length, dim] (float64), one a
    request. The tolerance is derived as in test_gpu_attend.py: weights are rounded to
    `weights` (the type of the second product), the result to q's."""
    dt, D = q.dtype, q.shape[2]
    weights = weights or dt
    scale = D ** -0.5 if scale is None else scale
    half, whalf = torch.finfo(dt).eps / 2, torch.finfo(weights).eps / 2
    tiny = torch.finfo(dt).smallest_normal * half
    outs, tols, at = [], [], 0
    for kb, vb, n, m in zip(k, v, news, lens):
        if n == 0:
            continue
        qq = q[at:at + n].double()
        at += n
        if m == 0:
            outs.append(torch.zeros_like(qq))
            tols.append(torch.zeros_like(qq))
            continue
        g = q.shape[1] // kb.shape[0]
        i, j = torch.arange(m - n, m, device=q.device)[:, None], torch.arange(m, device=q.device)[None]
        see = j <= i
        if window:
            see = see & ((j > i - window) | (j < sinks))
        ys, ts = [], []
        for h in range(q.shape[1]):
            kk, vv = kb[h // g], vb[h // g]
            # (what a row does not see does not reach it, whatever it is)
            seen = see.any(0)
            kk, vv = torch.where(seen[:, None], kk, 0.0), torch.where(seen[:, None], vv, 0.0)
            s = qq[:, h] @ kk.t() * scale
            mag = (qq[:, h].abs() @ kk.abs().t() * abs(scale)).masked_fill(~see, 0).amax(-1, keepdim=True)
            s = s.masked_fill(~see, -math.inf)
            top = s.amax(-1, keepdim=True)
            w = torch.where(see, torch.exp(s - torch.where(top.isfinite(), top, 0)), 0.0)
            l = w.sum(-1, keepdim=True)
            inv = torch.where(l > 0, 1 / l, 0.0)
            y = w @ vv * inv
            A = w @ vv.abs() * inv
            delta = (D + 2) * 2.0 ** -24 * mag
            tol = half * y.abs() + (whalf + 2 * delta + 2.0 ** -18) * A * (1 + 2 * half) + tiny * (l > 0)
            if weights == torch.float16:
                tol = tol + 2.0 ** -25 * (see.double() @ vv.abs()) * inv
            ys.append(y)
            ts.append(tol)
        outs.append(torch.stack(ys, 1))
        tols.append(torch.stack(ts, 1))
    return torch.cat(outs), torch.cat(tols)


def rows_of(pool, table, lens):
    """[kv, length, dim] of each request from values [pages, kv, page size, dim]."""
    ps = pool.shape[2]
    out = []
    for b, m in enumerate(lens):
        pages = table[b, :-(-m // ps)].long().to(pool.device)
        out.append(pool[pages].transpose(0, 1).reshape(pool.shape[1], -1, pool.shape[3])[:, :m].double())
    return out
