"""Rotary positions and the write to the paged cache on the GPU, against the
definition in 64 bits.

Tolerance, derived: the result is rounded once to its type (half a step: eps / 2
of |y|, and half of the smallest subnormal step), from fp32 values whose cosine and
sine are within 2^-23 (the polynomials' omitted terms and the roundings of the
angle, the argument and the evaluation, each under 2^-24 of at most 1) and
whose two products and sum round once each: together below 2^-21 (|a| + |b|) times the
factor on the result.
"""
import math

import pytest

from tests.gpu_util import announce, torch_mod

torch = torch_mod()
pytestmark = pytest.mark.gpu

SCALINGS = {
    "none": None, "linear": dict(kind="linear", factor=8.0), "base": dict(kind="base", factor=8.0),
    "by_parts": dict(kind="by_parts", factor=8.0, original_length=4096, low=1.0, high=32.0),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


def frequencies(rot, kind, f=8.0):
    n, b = rot // 2, 10000.0
    if kind == "base":
        b *= f ** (rot / (rot - 2))
    w = b ** (-torch.arange(n, dtype=torch.float64) / n)
    if kind == "linear":
        w = w / f
    if kind == "by_parts":
        keep = ((4096 * w / (2 * math.pi) - 1) / 31).clamp(0, 1)
        return w * keep + w / f * (1 - keep), 0.1 * math.log(f) + 1
    return w, 1.0


def rotated(x, positions, rot, layout, kind, transpose=False):
    """The definition in 64 bits on the CPU, and |a| + |b| of each value's pair (0: a copy)."""
    w, mag = frequencies(rot, kind)
    x, n = x.cpu().double(), rot // 2
    ang = positions.cpu().double()[:, None] * w
    c, s = (ang.cos() * mag)[:, None], (ang.sin() * (-mag if transpose else mag))[:, None]
    ia = torch.arange(n) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (n if layout == "half" else 1)
    y, m = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m[..., ia] = m[..., ib] = (a.abs() + b.abs()) * mag
    return y, m


def check(y, ref, m, what):
    y = y.cpu()
    half = torch.finfo(y.dtype).eps / 2
    tiny = torch.finfo(y.dtype).smallest_normal * half
    tol = half * ref.abs() + tiny + m * 2.0 ** -21 * (1 + half)
    tol = torch.where(m == 0, torch.zeros_like(tol), tol)       # copies are exact
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: worst {(err - tol).max().item()} over, at {(err - tol).argmax().item()}"


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,dim,rot,kind", [
    (1, 1, 2, 2, "none"), (3, 2, 6, 4, "linear"), (5, 3, 64, 64, "none"), (7, 4, 64, 16, "base"), (9, 2, 128, 96, "linear"),
    (33, 7, 128, 128, "by_parts"), (17, 3, 80, 80, "none"), (5, 2, 80, 20, "none"), (2, 5, 256, 64, "by_parts"),
    (3, 1, 512, 512, "none"), (601, 9, 128, 64, "none")])
def test_rotate(dt, layout, T, H, dim, rot, kind):
    import gptq_bit_weight_amd as q4
    announce(f"rotate {dt} {layout} T={T} H={H} dim={dim} rot={rot} {kind}")
    g = torch.Generator().manual_seed(T * 1000 + dim)
    x = torch.randn(T, H, dim, generator=g).to(dt).cuda()
    pos = torch.randint(-5, 1 << 20, (T,), generator=g).cuda()
    pos[0] = 0
    r = q4.Rotary(dim, rot, layout=layout, scaling=SCALINGS[kind])
    for tr in (False, True):
        ref, m = rotated(x, pos, rot, layout, kind, tr)
        check(r.rotate(x, pos, transpose=tr), ref, m, f"transpose={tr}")
    ref, m = rotated(x, pos, rot, layout, kind)
    check(r.rotate(x, pos.int()), ref, m, "int32 positions")
    check(r.rotate(x, pos, out=x), ref, m, "in place")


def test_far_positions():
    """Angles at the end of 31 bits and beyond: modulo a turn, in rational
    arithmetic by the 64-bit table."""
    import gptq_bit_weight_amd as q4
    r = q4.Rotary(64)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 40 + 7], device="cuda")
    x = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    w, _ = frequencies(64, "none")
    import ctypes
    turns = (ctypes.c_uint64 * 256)()
    q4.load_library().q4_rotary_plan(64, 64, 0, 10000.0, 1.0, 0, 0.0, 0.0, turns, ctypes.byref(ctypes.c_float()))
    ang = torch.tensor([[((p * turns[i]) % 2 ** 64) / 2 ** 64 * 2 * math.pi for i in range(32)] for p in pos.tolist()],
                       dtype=torch.float64)
    xd = x.cpu().double()
    a, b = xd[..., :32], xd[..., 32:]
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    ref = torch.cat([a * c - b * s, b * c + a * s], -1)
    m = torch.cat([a.abs() + b.abs()] * 2, -1)
    check(r.rotate(x, pos), ref, m, "far")


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H,kv,dim,rot,layout,ps,kind,shift", [
    (1, 4, 4, 128, 128, "half", 16, "none", 0), (8, 32, 32, 128, 128, "half", 16, "by_parts", 0),
    (37, 14, 2, 64, 32, "interleaved", 8, "linear", 0), (700, 8, 1, 64, 64, "half", 64, "none", 0),
    (21, 6, 3, 72, 72, "half", 5, "none", 0), (13, 4, 2, 128, 64, "half", 16, "none", 3),
    (1500, 28, 4, 128, 128, "interleaved", 32, "base", 0)])
def test_append(dt, T, H, kv, dim, rot, layout, ps, kind, shift):
    """Views of one fused row (at an offset that 16 bytes do not divide where
    `shift`), pages in random order, tokens that are not written."""
    import gptq_bit_weight_amd as q4
    announce(f"append {dt} T={T} H={H} kv={kv} dim={dim} rot={rot} {layout} ps={ps} {kind} shift={shift}")
    g = torch.Generator().manual_seed(T + dim)
    fused = torch.randn(T, (H + 2 * kv) * dim + shift, generator=g).to(dt).cuda()[:, shift:]
    q = fused[:, :H * dim].unflatten(1, (H, dim))
    k = fused[:, H * dim:(H + kv) * dim].unflatten(1, (kv, dim))
    v = fused[:, (H + kv) * dim:].unflatten(1, (kv, dim))
    pages = -(-T // ps) + 2
    kc, vc = torch.randn(2, pages, kv, ps, dim, generator=g).to(dt).cuda()
    slots = torch.randperm(pages * ps, generator=g)[:T].cuda()
    if T > 2:
        slots[1], slots[2] = -1, pages * ps      # neither is written
    pos = torch.randint(0, 1 << 20, (T,), generator=g).cuda()
    r = q4.Rotary(dim, rot, layout=layout, scaling=SCALINGS[kind])
    k0, v0 = kc.cpu(), vc.cpu()
    cache = q4.PagedCache(kc, vc)
    qo = cache.append(k, v, slots, rotary=r, positions=pos, q=q)
    check(qo, *rotated(q, pos, rot, layout, kind), "q")
    ref, m = rotated(k, pos, rot, layout, kind)
    sl = slots.cpu()
    live = (sl >= 0) & (sl < pages * ps)
    page, row = sl[live] // ps, sl[live] % ps
    check(kc[page.cuda(), :, row.cuda()], ref[live], m[live], "k")
    v0[page, :, row] = v.cpu()[live]
    assert torch.equal(vc.cpu(), v0)
    kn = kc.cpu()
    kn[page, :, row] = k0[page, :, row]
    assert torch.equal(kn, k0)                   # no other row is touched
    # without a rotary: a copy; 32-bit slots; q turned in place
    cache.append(k, v, slots.int())
    k0[page, :, row] = k.cpu()[live]
    assert torch.equal(kc.cpu(), k0)
    want = rotated(q, pos, rot, layout, kind)
    assert cache.append(k, v, slots, rotary=r, positions=pos, q=q, q_out=q) is q
    check(q, *want, "q in place")


def test_append_strided_cache():
    """A cache held [pages, rows, k or v, heads, dim], seen through views."""
    import gptq_bit_weight_amd as q4
    store = torch.zeros(5, 16, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = (store[:, :, i].transpose(1, 2) for i in (0, 1))
    k, v = torch.randn(2, 20, 3, 64, device="cuda").bfloat16()
    slots = torch.randperm(80, device="cuda")[:20]
    q4.PagedCache(kc, vc).append(k, v, slots)
    flat = store.view(80, 2, 3, 64)
    assert torch.equal(flat[slots, 0], k) and torch.equal(flat[slots, 1], v)
    rest = torch.ones(80, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert (flat[rest] == 0).all()


def test_append_beyond_31_bits():
    """A row of a cache tensor whose offset passes 2^32 bytes and 2^31 values."""
    import gptq_bit_weight_amd as q4
    pages = (1 << 31) // (8 * 64 * 128) + 3
    kc = torch.empty(pages, 8, 64, 128, dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    k, v = torch.randn(2, 3, 8, 128, device="cuda").half()
    slots = torch.tensor([pages * 64 - 1, (pages - 2) * 64, 5], device="cuda")
    q4.PagedCache(kc, vc).append(k, v, slots)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // 64, :, s % 64], k[i]) and torch.equal(vc[s // 64, :, s % 64], v[i])


def test_gradient():
    """autograd against differences of the definition: the rotation is linear,
    so <g, R d> = <R^T g, d> for any direction d."""
    import gptq_bit_weight_amd as q4
    r = q4.Rotary(64, 32, scaling=SCALINGS["by_parts"])
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 3, 64, generator=g).bfloat16().cuda().requires_grad_(True)
    pos = torch.randint(0, 9999, (5,), generator=g).cuda()
    up = torch.randn(5, 3, 64, generator=g).bfloat16().cuda()
    y = r.rotate(x, pos)
    y.backward(up)
    ref, m = rotated(up, pos, 32, "half", "by_parts", True)
    check(x.grad, ref, m, "grad")
    d = torch.randn(5, 3, 64, generator=g).double()
    plus, _ = rotated(x.detach().cpu().double() + d, pos, 32, "half", "by_parts")
    minus, _ = rotated(x.detach().cpu().double() - d, pos, 32, "half", "by_parts")
    diff = ((plus - minus) / 2 * up.cpu().double()).sum()
    # each of the gradient's values is off by at most its half step (and the fp32 part)
    tol = ((ref.abs() * 2.0 ** -8 + m * 2.0 ** -20) * d.abs()).sum()
    assert abs((x.grad.cpu().double() * d).sum() - diff) <= tol


def test_gradient_on_another_stream():
    """The backward pass of a call on a stream that is not the current one waits
    for the gradient it takes, and what takes its result waits for it; and the
    gradient of the gradient."""
    import gptq_bit_weight_amd as q4
    r = q4.Rotary(64, 32, scaling=SCALINGS["by_parts"])
    g = torch.Generator().manual_seed(4)
    pos = torch.arange(700, 705, device="cuda")
    x = torch.randn(5, 3, 64, generator=g).bfloat16().cuda().requires_grad_()
    up = torch.randn(5, 3, 64, generator=g).bfloat16().cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = r.rotate(x, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    slow = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        slow = slow @ slow * 1e-3       # what the gradient comes from takes a while
    up2 = up + (slow[0, 0] * 0).nan_to_num().bfloat16()
    y.backward(up2)
    check(x.grad, *rotated(up, pos, 32, "half", "by_parts", True), "grad")
    x2 = x.detach().clone().requires_grad_()
    w = up.clone().requires_grad_()
    gx, = torch.autograd.grad(r.rotate(x2, pos), x2, w, create_graph=True)
    gw, = torch.autograd.grad(gx, w, x.detach())
    check(gw, *rotated(x.detach(), pos, 32, "half", "by_parts"), "second")


def test_graph_and_streams():
    """Captured, replayed with other data; and a call on a stream that is not
    the current one."""
    import gptq_bit_weight_amd as q4
    r = q4.Rotary(128)
    kc, vc = torch.zeros(2, 4, 2, 16, 128, dtype=torch.float16, device="cuda")
    cache = q4.PagedCache(kc, vc)
    k, v = torch.randn(2, 6, 2, 128, device="cuda").half()
    q = torch.randn(6, 4, 128, device="cuda").half()
    slots = torch.arange(6, device="cuda") * 9
    pos = torch.arange(6, device="cuda")
    cache.append(k, v, slots, rotary=r, positions=pos, q=q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo = cache.append(k, v, slots, rotary=r, positions=pos, q=q)
    for i in range(3):
        pos.add_(100 * i)
        k.normal_()
        q.normal_()
        kc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(qo, *rotated(q, pos, 128, "half", "none"), f"replay {i}")
        check(kc[slots // 16, :, slots % 16], *rotated(k, pos, 128, "half", "none"), f"replay {i} k")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = r.rotate(q, pos, stream=s)
    s.synchronize()
    check(y, *rotated(q, pos, 128, "half", "none"), "stream")


def test_refusals():
    import gptq_bit_weight_amd as q4
    r = q4.Rotary(64)
    x = torch.randn(3, 2, 64, device="cuda").half()
    p = torch.arange(3, device="cuda")
    bad = [
        lambda: r.rotate(x.float(), p), lambda: r.rotate(x, p[:2]), lambda: r.rotate(x, p.float()),
        lambda: r.rotate(x[..., :32], p), lambda: r.rotate(x[0], p), lambda: r.rotate(x.cpu(), p),
        lambda: r.rotate(x, p.cpu()), lambda: r.rotate(x.transpose(1, 2), p),
        lambda: r.rotate(x, p, out=x.bfloat16()), lambda: r.rotate(x, p, out=x[:1].expand(3, 2, 64)),
        lambda: r.rotate(x[:, :1], p, out=x[:, 1:].flip(0)[:2]),
    ]
    flat = torch.zeros(3 * 2 * 64 + 64, dtype=torch.float16, device="cuda")
    bad.append(lambda: r.rotate(flat[:384].view(3, 2, 64), p, out=flat[64:448].view(3, 2, 64)))
    kc, vc = torch.zeros(2, 2, 2, 4, 64, dtype=torch.float16, device="cuda")
    c = q4.PagedCache(kc, vc)
    bad += [
        lambda: q4.PagedCache(kc, vc[:1]), lambda: q4.PagedCache(kc, vc.bfloat16()),
        lambda: q4.PagedCache(kc[:1].expand(2, 2, 4, 64), vc),
        lambda: c.append(x, x, p, rotary=r), lambda: c.append(x, x, p, q=x), lambda: c.append(x[:, :1], x, p),
        lambda: c.append(x, x[:2], p), lambda: c.append(x, x, p[:2]), lambda: c.append(x, x, p, q_out=x),
        lambda: c.append(x, x, p, rotary=q4.Rotary(32), positions=p), lambda: c.append(x, x.bfloat16(), p),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"case {i} was taken")
    r.close()
    with pytest.raises(ValueError, match="closed"):
        r.rotate(x, p)


def test_nothing_to_do():
    import gptq_bit_weight_amd as q4
    r = q4.Rotary(64)
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    assert r.rotate(torch.empty(0, 2, 64, dtype=torch.float16, device="cuda"), e).shape == (0, 2, 64)
    p = torch.arange(2, device="cuda")
    assert r.rotate(torch.empty(2, 0, 64, dtype=torch.float16, device="cuda"), p).shape == (2, 0, 64)


def test_outputs_that_meet_inputs_are_refused():
    """q_out against q, k, v, the cache and the indexes; parts of one row side by side pass."""
    import gptq_bit_weight_amd as q4
    T, H, kv, D, ps = 5, 4, 2, 64, 16
    fused = torch.randn(T, H + 2 * kv + H, D, device="cuda").half()
    q, k, v, rest = fused.split([H, kv, kv, H], 1)
    kc, vc = torch.zeros(2, 3, kv, ps, D, dtype=torch.float16, device="cuda")
    c, r = q4.PagedCache(kc, vc), q4.Rotary(D)
    slots, pos = torch.arange(T, device="cuda"), torch.arange(T, device="cuda") + 3
    args = dict(rotary=r, positions=pos)
    own = torch.zeros(8 * T * H * D, dtype=torch.float16, device="cuda")
    index = own[:4 * T].view(torch.int64)
    index.copy_(slots)
    bad = [
        dict(q=q, q_out=fused[:, H - 1:2 * H - 1]), dict(q=q.clone(), q_out=fused[:, H:2 * H]), dict(q=q.clone(), q_out=fused[:, 2:2 + H]),
        dict(q=q.clone(), q_out=kc.view(-1)[:T * H * D].view(T, H, D)), dict(q=q.clone(), q_out=vc.view(-1)[64:64 + T * H * D].view(T, H, D)),
        dict(q=q, q_out=own[8:8 + T * H * D].view(T, H, D), slots=index), dict(q=q, q_out=own[8:8 + T * H * D].view(T, H, D), positions=index),
    ]
    for i, kw in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps"):
            c.append(**{**dict(k=k, v=v, slots=slots, **args), **kw})
            pytest.fail(f"case {i} was taken")
    with pytest.raises(ValueError, match="overlaps"):
        r.rotate(q.contiguous(), index, out=own[8:8 + T * H * D].view(T, H, D))
    assert (kc == 0).all() and (vc == 0).all()
    keep = fused.clone()
    out = c.append(k, v, slots, q=q.clone(), q_out=rest, **args)
    assert out is rest
    check(rest, *rotated(keep[:, :H], pos, D, "half", "none"), "beside")
    assert torch.equal(fused[:, :H + 2 * kv], keep[:, :H + 2 * kv])
    c.append(k, v, slots, q=q, q_out=q, **args)
    check(q, *rotated(keep[:, :H], pos, D, "half", "none"), "in place")
    assert torch.equal(fused[:, H:H + 2 * kv], keep[:, H:H + 2 * kv])


def test_tangents():
    """Forward derivatives: a tangent is turned as x is, on another stream too."""
    import gptq_bit_weight_amd as q4
    from torch.autograd import forward_ad
    r = q4.Rotary(64, 32, scaling=SCALINGS["by_parts"])
    g = torch.Generator().manual_seed(5)
    x, v = torch.randn(2, 5, 3, 64, generator=g).bfloat16().cuda()
    pos = torch.arange(700, 705, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for tr in (False, True):
        for stream in (None, s):
            with forward_ad.dual_level():
                y, dy = forward_ad.unpack_dual(r.rotate(forward_ad.make_dual(x, v), pos, transpose=tr, stream=stream))
            torch.cuda.synchronize()
            check(y, *rotated(x, pos, 32, "half", "by_parts", tr), "value")
            check(dy, *rotated(v, pos, 32, "half", "by_parts", tr), "tangent")
    with forward_ad.dual_level(), pytest.raises(ValueError, match="tangent"):
        r.rotate(x, pos, out=forward_ad.make_dual(x, v))
