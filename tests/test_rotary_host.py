"""Host side of the rotary positions and the paged cache: the table against
the definition in exact-enough arithmetic, and what is refused before any GPU
call."""
import ctypes
import math
from fractions import Fraction

import pytest

import gptq_bit_weight_amd as q4

KINDS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}


def _plan(dim, rot, kind="none", base=10000.0, factor=1.0, original=0, low=0.0, high=0.0):
    lib = q4.load_library()
    turns, mag = (ctypes.c_uint64 * 256)(), ctypes.c_float(0)
    st = lib.q4_rotary_plan(dim, rot, KINDS.get(kind, kind), base, factor, original, low, high, turns, ctypes.byref(mag))
    return st, list(turns)[:max(rot, 0) // 2], mag.value


@pytest.mark.parametrize("rot", [2, 4, 64, 96, 128, 512])
@pytest.mark.parametrize("kind", ["none", "linear", "base", "by_parts"])
def test_table(rot, kind):
    if kind == "base" and rot == 2:
        pytest.skip("refused")
    f = 8.0
    st, turns, mag = _plan(512, rot, kind, factor=f if kind != "none" else 1.0, original=4096, low=1.0, high=32.0)
    assert st == 0
    n = rot // 2
    for i, t in enumerate(turns):
        b = 10000.0 * (f ** (rot / (rot - 2)) if kind == "base" else 1.0)
        w = b ** (-i / n)
        if kind == "linear":
            w /= f
        if kind == "by_parts":
            keep = min(1.0, max(0.0, (4096 * w / (2 * math.pi) - 1.0) / 31.0))
            w = w * keep + w / f * (1 - keep)
        got = float(Fraction(t, 2 ** 64)) * 2 * math.pi
        assert abs(got - w) <= 1e-13 * w + 2.0 ** -64 * 7, (i, got, w)   # (double's own rounding in w)
    assert mag == pytest.approx(0.1 * math.log(f) + 1 if kind == "by_parts" else 1.0, rel=1e-7)


def test_first_pair_is_one_radian():
    _, turns, _ = _plan(128, 128)
    # 2^64 / (2 pi) to the unit
    assert abs(turns[0] - 2935890503282001226) <= 1


@pytest.mark.parametrize("dim,rot,kw,status", [
    (128, 127, {}, 1), (128, 130, {}, 1), (128, 0, {}, 1), (1, 2, {}, 1), (514, 64, {}, 2),
    (128, 128, dict(base=1.0), 1), (128, 128, dict(base=math.inf), 1), (128, 128, dict(kind=9), 1),
    (128, 128, dict(kind="linear", factor=0.5), 1), (128, 128, dict(kind="linear", factor=math.nan), 1),
    (128, 2, dict(kind="base", factor=2.0), 1),
    (128, 64, dict(kind="by_parts", factor=2.0, original=0, low=1.0, high=2.0), 1),
    (128, 64, dict(kind="by_parts", factor=2.0, original=9, low=2.0, high=2.0), 1),
])
def test_plan_refuses(dim, rot, kw, status):
    assert _plan(dim, rot, **kw)[0] == status
    assert q4.load_library().q4_last_error()


@pytest.mark.parametrize("kw,exc", [
    (dict(rot=7), ValueError), (dict(layout="other"), ValueError), (dict(scaling=dict(kind="x")), ValueError),
    (dict(scaling=dict(kind="linear")), ValueError), (dict(scaling=dict(kind="none", factor=2.0)), ValueError),
    (dict(scaling=dict(kind="linear", factor=0.1)), ValueError),
])
def test_rotary_refuses(kw, exc):
    with pytest.raises(exc):
        q4.Rotary(64, **kw)


def test_rotary_head_too_long():
    with pytest.raises(NotImplementedError):
        q4.Rotary(1024)


def test_cache_refuses():
    import torch
    good = torch.zeros(2, 2, 4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        q4.PagedCache(good, good.clone())
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        q4.PagedCache(good.float(), good.float())
    with pytest.raises(ValueError, match="pages"):
        q4.PagedCache(good[0], good[0])
    with pytest.raises(ValueError, match="contiguous"):
        q4.PagedCache(good.transpose(2, 3), good)
    with pytest.raises(TypeError):
        q4.PagedCache(None, good)


def _cache(**kw):
    from gptq_bit_weight_amd.attention import _Cache
    c = _Cache(4096, 8192, (ctypes.c_int64 * 3)(64, 32, 8), (ctypes.c_int64 * 3)(64, 32, 8), 4, 2, 4, 8, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("cache,args", [
    (dict(k=None), {}), (dict(pages=0), {}), (dict(dim=0), {}), (dict(page_size=-1), {}),
    ({}, dict(k=None)), ({}, dict(slots=None)), ({}, dict(slot_bits=16)), ({}, dict(tokens=-1)), ({}, dict(q=4096)),
])
def test_append_refuses_before_any_gpu_call(cache, args):
    a = dict(k=4096, v=4096, slots=4096, slot_bits=64, tokens=3, q=None)
    a.update(args)
    st = q4.load_library().q4_cache_append(ctypes.byref(_cache(**cache)), a["k"], 16, 8, a["v"], 16, 8, a["slots"],
                                           a["slot_bits"], a["tokens"], None, None, 32, a["q"], 16, 8, a["q"], 16, 8,
                                           2, None)
    assert st == 1


def test_append_of_no_tokens():
    assert q4.load_library().q4_cache_append(ctypes.byref(_cache()), None, 0, 0, None, 0, 0, None, 64, 0, None, None,
                                             32, None, 0, 0, None, 0, 0, 0, None) == 0


def test_cache_rows_fit_31_bits():
    c = _cache(pages=1 << 20, page_size=1 << 12)
    assert q4.load_library().q4_cache_append(ctypes.byref(c), 4096, 0, 0, 4096, 0, 0, 4096, 64, 1, None, None, 32,
                                             None, 0, 0, None, 0, 0, 0, None) == 2


class _Plain:
    """A rotation of heads of 4 values on the CPU, in the place of the library's."""
    dim = 4

    def _rotate(self, x, positions, transpose, out, stream):
        import torch
        assert not x.requires_grad and x.data_ptr()
        c, s = positions.to(x.dtype).cos()[:, None, None], positions.to(x.dtype).sin()[:, None, None] * (-1 if transpose else 1)
        a, b = x[..., :2], x[..., 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)


def test_derivatives_backward_and_forward():
    """What rotate() records: gradients and tangents, of each other too, against
    differences, and through the functional transforms."""
    import torch
    from torch.autograd import forward_ad

    plain, pos = _Plain(), torch.tensor([5, 0, -3])
    g = torch.Generator().manual_seed(2)
    x, v = torch.randn(2, 3, 2, 4, generator=g, dtype=torch.float64)

    def rotate(t, transpose=False):
        return q4.Rotary.rotate(plain, t, pos, transpose=transpose)

    want = rotate(v)
    with forward_ad.dual_level():
        for tangent in (v, v.transpose(0, 2).contiguous().transpose(0, 2)):
            y, dy = forward_ad.unpack_dual(rotate(forward_ad.make_dual(x, tangent)))
            assert torch.equal(y, rotate(x)) and torch.equal(dy, want)
            with torch.no_grad():
                assert torch.equal(forward_ad.unpack_dual(rotate(forward_ad.make_dual(x, tangent))).tangent, want)
        assert forward_ad.unpack_dual(rotate(x)).tangent is None
    assert torch.equal(torch.func.jvp(rotate, (x,), (v,))[1], want)
    assert torch.allclose(torch.func.grad(lambda t: (rotate(t) * v).sum())(x), rotate(v, True))
    # (R^T R = 1: the gradient of |R x|^2 / 2 is x, its tangent v)
    assert torch.allclose(torch.func.jvp(torch.func.grad(lambda t: (rotate(t) ** 2).sum() / 2), (x,), (v,))[1], v)
    leaf = x.clone().requires_grad_()
    assert torch.autograd.gradcheck(rotate, (leaf,), check_forward_ad=True)
    assert torch.autograd.gradgradcheck(lambda t: rotate(t) ** 2, (leaf,))


def test_outputs_with_a_tangent_are_refused():
    import torch
    from torch.autograd import forward_ad
    from gptq_bit_weight_amd.attention import _writable
    x = torch.zeros(3, 2, 4, dtype=torch.float16)
    with forward_ad.dual_level():
        _writable(x, "out")
        with pytest.raises(ValueError, match="tangent"):
            _writable(forward_ad.make_dual(x, x), "out")
