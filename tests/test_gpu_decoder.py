"""The operators together, as examples/decoder_attention.py runs them: prompts
in chunks, single tokens beside them and captured decode steps over one paged
cache, against the same block in 64 bits.

Tolerance: the reference carries a bound on the error beside each value. A bound
grows by half a step of the type where the block rounds (the projections'
outputs, the turned q and k, the softmax's weights, the attention's output, the
sum with x) and by 2^-18 of the sum of magnitudes where fp32 adds up; it passes
through a product by the other factor's magnitude, through the rotation by |cos|
and |sin|, and through the softmax as exp(2 d) - 1, d the largest bound of a visible
score (its own error and the sum's), with 2^-25 for subnormal weights.
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


def dense(layers):
    """[K, N] of packed layers side by side, exactly."""
    out = []
    for qw, qz, sc in layers:
        sh = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
        q = ((qw[:, None, :] >> sh[None, :, None]) & 15).reshape(-1, qw.shape[1])
        z = ((qz[:, :, None] >> sh) & 15).reshape(qz.shape[0], -1)
        g = q.shape[0] // z.shape[0]
        out.append((q - z.repeat_interleave(g, 0)).double() * sc.double().repeat_interleave(g, 0))
    return torch.cat(out, 1)


def projected(x, w, A, B, c, parts):
    """x W + c B A x, and the same of magnitudes."""
    y, m = x @ w, x.abs() @ w.abs()
    if A is not None:
        at = 0
        for p, n in enumerate(parts):
            a, b = A[p].double(), B[at:at + n].double()
            y[:, at:at + n] += c * (x @ a.t()) @ b.t()
            m[:, at:at + n] += c * (x.abs() @ a.abs().t()) @ b.abs().t()
            at += n
    return y, m


def reference(block, x, adapter):
    """(output, tolerance) of one request's tokens, in 64 bits."""
    H, kv, D = block.heads, block.kv_heads, block.dim
    eps = torch.finfo(block.dtype).eps
    half, small = eps / 2, 2.0 ** -18            # (fp32 sums: some 2^-24 times their length's root, at most this)
    ad = block.adapters[adapter] if adapter >= 0 else (None,) * 4
    x = x.double()
    y, m = projected(x, dense(block.qkv_layers), ad[0], ad[1], 2.0, [H * D, kv * D, kv * D])
    err = half * y.abs() + small * m             # of the projection's outputs
    T = x.shape[0]
    pos = torch.arange(T, device="cuda", dtype=torch.float64)
    ang = pos[:, None] * 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def turn(t, e):
        a, b, ea, eb = t[..., :D // 2], t[..., D // 2:], e[..., :D // 2], e[..., D // 2:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
        er = ea * c.abs() + eb * s.abs()
        return r, torch.cat([er, ea * s.abs() + eb * c.abs()], -1) + (half + small) * r.abs() + half * torch.cat([er, er], -1)

    q, eq = turn(y[:, :H * D].view(T, H, D), err[:, :H * D].view(T, H, D))
    k, ek = turn(y[:, H * D:(H + kv) * D].view(T, kv, D), err[:, H * D:(H + kv) * D].view(T, kv, D))
    v, ev = y[:, (H + kv) * D:].view(T, kv, D), err[:, (H + kv) * D:].view(T, kv, D)
    see = pos[None] <= pos[:, None]
    os_, es = [], []
    for h in range(H):
        kk, vv, ekk, evv = k[:, h * kv // H], v[:, h * kv // H], ek[:, h * kv // H], ev[:, h * kv // H]
        sc = q[:, h] @ kk.t() * D ** -0.5
        ds = (eq[:, h] @ kk.abs().t() + q[:, h].abs() @ ekk.t() + eq[:, h] @ ekk.t()) * D ** -0.5 + small
        w = torch.softmax(sc.masked_fill(~see, -math.inf), -1)
        d = ds.masked_fill(~see, 0).amax(-1, keepdim=True)
        dw = w * (torch.exp(2 * d) - 1 + half + small) + 2.0 ** -25 * see.double()
        o = w @ vv
        eo = dw @ vv.abs() + (w + dw) @ evv
        es.append(eo + half * (o.abs() + eo))
        os_.append(o)
    o, eo = torch.stack(os_, 1).reshape(T, -1), torch.stack(es, 1).reshape(T, -1)
    w = dense([block.o_layer])
    z, m = projected(o, w, ad[2], ad[3], 2.0, [w.shape[1]])
    _, ez = projected(eo, w.abs(), None if ad[2] is None else ad[2].abs(), None if ad[2] is None else ad[3].abs(), 2.0, [w.shape[1]])
    ez = ez + small * m
    ez = ez + half * (z.abs() + ez)
    out = x + z
    return out, ez + half * (out.abs() + ez)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,page_size", [(4, 4, 16), (8, 2, 7)])
def test_block(dt, heads, kv, page_size):
    from examples.decoder_attention import AttentionBlock, serve
    announce(f"decoder block {dt} {heads}/{kv} pages of {page_size}")
    block = AttentionBlock(512, heads, kv, 64, group=64, pages=256, page_size=page_size, adapters=3, rank=12, dtype=dt, seed=heads)
    g = torch.Generator(device="cuda").manual_seed(7)
    prompts = [torch.randn(n, 512, generator=g, device="cuda").to(dt) for n in (150, 1, 33, 64)]
    adapters = [2, 0, -1, 1]
    outs, history, _ = serve(block, prompts, adapters, chunk=64, steps=5)
    for p, a, o, r in zip(prompts, adapters, outs, range(4)):
        # the decode steps' inputs are their own outputs before them
        x = torch.cat([p, o[-1:], history[:-1, r]])
        ref, tol = reference(block, x, a)
        y = torch.cat([o, history[:, r]]).double()
        bad = ~((y - ref).abs() <= tol)
        assert not bad.any(), (r, int(bad.sum()), bad.nonzero()[0].tolist(), ((y - ref).abs() / tol).max().item())
