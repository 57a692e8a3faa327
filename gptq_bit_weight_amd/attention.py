"""Rotary positions, a paged cache of keys and values, and attention of new
tokens over it: what a decoder layer needs between its quantized
projections.

    rope = q4.Rotary(dim, scaling=dict(kind="linear", factor=8.0))
    cache = q4.PagedCache(k_pages, v_pages)          # [pages, kv heads, page size, dim]
    q = cache.append(k, v, slots, rotary=rope, positions=positions, q=q)
    o = cache.attend(q, starts, lengths, table)

Like the rest of the binding this only checks tensors and passes pointers and
a HIP stream to the C ABI (``include/q4.h``).
"""
from __future__ import annotations

import ctypes
import threading

import torch
from torch.autograd import forward_ad

from . import _check, _raise, load_library

__all__ = ["Rotary", "PagedCache"]

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}
_SCALING_KEYS = {"none": set(), "linear": {"factor"}, "base": {"factor"},
                 "by_parts": {"factor", "original_length", "low", "high"}}
_HALVES = (torch.float16, torch.bfloat16)


# (A call's Python costs as much as a small kernel, so what is looked up for
# each is kept cheap: the current stream's handle without a Stream object is
# 0.1 us against 1.8.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_dense = torch.contiguous_format
_Tensor, _int32_t, _int64_t = torch.Tensor, torch.int32, torch.int64
_wrote = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version   # tells autograd of a tuple of tensors written in place


def _recorded(t):
    """Whether a derivative goes by t: backward, or forward (it has a tangent)."""
    return (t.requires_grad and torch.is_grad_enabled()) or (
        forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None)


def _writable(t, name):
    """An output given by the caller, or the cache: no derivative goes through a write."""
    if _recorded(t):
        raise ValueError(f"{name} requires a gradient, or has a tangent, and cannot be written in place "
                         "(under torch.no_grad() a gradient's may)")


class _Cache(ctypes.Structure):
    """q4_cache of include/q4.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("dim", ctypes.c_int), ("bf16", ctypes.c_int)]


def _heads(t, name, device, dtype=None, tokens=None, heads=None, dim=None):
    """Check a [tokens, heads, dim] tensor whose head values are dense; returns
    its shape and strides."""
    if isinstance(t, _Tensor):
        d = t.dtype
        if d in _HALVES and (dtype is None or d is dtype) and t.device == device:
            s = t.shape
            if len(s) == 3 and (tokens is None or s[0] == tokens) and (heads is None or s[1] == heads) and (dim is None or s[2] == dim):
                st = t.stride()
                if st[2] == 1 or s[2] <= 1:
                    return s, st
                raise ValueError(f"{name}: the values of a head must be contiguous")
            want = [("tokens" if tokens is None else tokens), ("heads" if heads is None else heads), ("dim" if dim is None else dim)]
            raise ValueError(f"{name} must be {want}, got {list(s)}")
        if d not in _HALVES or (dtype is not None and d != dtype):
            raise ValueError(f"{name} must be {dtype or 'float16 or bfloat16'}, got {d}")
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise TypeError(f"{name} must be a torch.Tensor")


def _index(t, name, device, n):
    """Check an index vector of n int32 or int64; returns its width in bits."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.dtype
    if d is not _int64_t and d is not _int32_t:
        raise ValueError(f"{name} must be int32 or int64, got {d}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape [{n}], got {list(t.shape)}")
    return 64 if d is _int64_t else 32


def _int32(t, name, device, dims):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _int32_t or t.dim() != dims or t.device != device:
        raise ValueError(f"{name} must be int32 with {dims} dimensions on {device}, got {t.dtype} {list(t.shape)} on {t.device}")


def _distinct(t, name):
    """An output's elements must be distinct places in memory."""
    span = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda p: p[1]):
        if size > 1:
            if stride < span:
                raise ValueError(f"{name} overlaps itself")
            span = stride * (size - 1) + span


def _table_rows(table, stream=None):
    """A page table and its row stride, at least its width. Rows that share memory
    (one row expanded over the requests) are copied: the C call takes them apart only.
    One row has no stride of its own."""
    B, width = table.shape
    ts = table.stride(0)
    if B == 1:
        return table, width
    if ts < width:
        if stream is not None:
            table.record_stream(stream)
        return _on(stream, torch.clone, table, memory_format=_dense), width
    return table, ts


def _out_like(x, out, name, stream):
    """The output for x: `out` checked, or a new dense tensor made on the
    stream that the call runs on."""
    if out is None:
        if stream is None:
            return torch.empty_like(x, memory_format=_dense)
        with torch.cuda.stream(stream):
            return torch.empty_like(x, memory_format=_dense)
    _heads(out, name, x.device, x.dtype, *x.shape)
    _writable(out, name)
    _distinct(out, name)            # (the C call refuses one that meets an input)
    return out


def _call(fn, what, device, stream, args, used=()):
    """Call a C function on `stream` (the device's current one by default)."""
    if stream is None:
        sp = _raw_stream(device.index)
    else:
        if stream.device != device:
            raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on {device}")
        sp = stream.cuda_stream
        for t in used:          # their memory stays until the stream is done with it
            t.record_stream(stream)
    if _device() == device.index:
        st = fn(*args, sp)
    else:
        with torch.cuda.device(device):
            st = fn(*args, sp)
    if st:
        _check(st, what)


class _Rotate(torch.autograd.Function):
    """The rotation is linear: a tangent is turned as x is, a gradient the other way."""

    @staticmethod
    def forward(x, rotary, positions, transpose, stream):
        return rotary._rotate(x.detach(), positions, transpose, None, stream)

    @staticmethod
    def setup_context(ctx, inputs, output):
        _, ctx.rotary, positions, ctx.transpose, ctx.stream = inputs
        ctx.save_for_backward(positions)
        ctx.save_for_forward(positions)

    @staticmethod
    def _turn(ctx, t, transpose):
        positions, = ctx.saved_tensors
        if t.stride(2) != 1:
            t = t.contiguous()
        # (on the forward pass's stream, between what makes the gradient and what
        # takes it, which are on the one that was current then)
        s = ctx.stream
        if s is not None:
            now = torch.cuda.current_stream(t.device)
            s.wait_stream(now)
        out = _Rotate.apply(t, ctx.rotary, positions, transpose, s)
        if s is not None:
            now.wait_stream(s)
            out.record_stream(now)
        return out

    @staticmethod
    def backward(ctx, grad):
        return _Rotate._turn(ctx, grad, not ctx.transpose), None, None, None, None

    @staticmethod
    def jvp(ctx, tangent, *rest):
        return _Rotate._turn(ctx, tangent, ctx.transpose)


class Rotary:
    """Rotary positions for heads of `dim` values (at most 512) whose first
    `rot` (default all) are rotated: pairs (i, i + rot/2) (layout "half") or
    (2i, 2i + 1) ("interleaved"), pair i by base^(-2i / rot) radians a position.

    scaling: None, or a dict with "kind" and
      "linear": factor -- every frequency divided by it;
      "base": factor -- base times factor^(rot / (rot - 2));
      "by_parts": factor, original_length, low, high -- pairs that turn at least
        `high` times in original_length positions keep their frequency, those
        under `low` turns are divided by factor, a ramp between; the result is
        multiplied by 0.1 ln(factor) + 1.

    Positions are int32 or int64 of any sign; angles are exact modulo a turn.
    The table lives on `device` (default: the current one).
    """

    def __init__(self, dim: int, rot: int | None = None, *, layout: str = "half", base: float = 10000.0,
                 scaling: dict | None = None, device=None):
        self._h = None
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
        s = dict(scaling or {"kind": "none"})
        kind = s.pop("kind", None)
        if kind not in SCALINGS:
            raise ValueError(f"scaling kind must be one of {sorted(SCALINGS)}, got {kind!r}")
        if set(s) != _SCALING_KEYS[kind]:
            raise ValueError(f"scaling {kind!r} takes {sorted(_SCALING_KEYS[kind])}, got {sorted(s)}")
        self.dim, self.rot = int(dim), int(dim if rot is None else rot)
        self.layout = layout
        lib = load_library()
        args = (self.dim, self.rot, SCALINGS[kind], base, s.get("factor", 1.0), s.get("original_length", 0),
                s.get("low", 0.0), s.get("high", 0.0))
        # (the arguments' own checks need no device)
        turns, mag = (ctypes.c_uint64 * 256)(), ctypes.c_float(1.0)
        _check(lib.q4_rotary_plan(*args, turns, ctypes.byref(mag)), "Rotary")
        self.magnitude = float(mag.value)
        dev = torch.device("cuda" if device is None else device)
        self.device = torch.device(dev.type, torch.cuda.current_device()) if dev.index is None else dev
        with torch.cuda.device(self.device):
            h = lib.q4_rotary_make(self.dim, self.rot, LAYOUTS[layout], *args[2:])
        if not h:
            _raise(lib.q4_last_status(), "q4_rotary_make")
        self._h = ctypes.c_void_p(h)

    def _handle(self):
        if self._h is None:
            raise ValueError("Rotary is closed")
        return self._h

    def _rotate(self, x, positions, transpose, out, stream):
        dev = self.device
        (T, H, _), xs = _heads(x, "x", dev, None, None, None, self.dim)
        bits = _index(positions, "positions", dev, T)
        written = out is not None
        out = _out_like(x, out, "out", stream)
        os_ = out.stride()
        _call(load_library().q4_rotary_apply, "q4_rotary_apply", dev, stream,
              (self._handle(), x.data_ptr(), xs[0], xs[1], out.data_ptr(), os_[0], os_[1], positions.data_ptr(), bits,
               T, H, 1 if transpose else 0, 1 if x.dtype == torch.bfloat16 else 0), (x, positions, out))
        if written:
            _wrote((out,))
        return out

    def rotate(self, x, positions, *, transpose: bool = False, out=None, stream=None):
        """x [tokens, heads, dim] (float16 or bfloat16, any token and head
        strides) turned by positions [tokens]; with `transpose` the other way
        with the same factor: the gradient's pass. fp32, rounded once. out may
        be x itself. Without `out` the call is differentiable in x (backward and
        forward); one that requires a gradient is refused while gradients are recorded."""
        if out is None and isinstance(x, torch.Tensor) and _recorded(x):
            return _Rotate.apply(x, self, positions, transpose, stream)
        return self._rotate(x, positions, transpose, out, stream)

    def close(self):
        if getattr(self, "_h", None) is not None:
            torch.cuda.synchronize(self.device)
            load_library().q4_rotary_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedCache:
    """Keys and values in pages: two tensors [pages, kv heads, page size, dim]
    (float16 or bfloat16, any strides of the first three dimensions, dense
    values), which stay the caller's and are written in place."""

    def __init__(self, k, v):
        for t, nm in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{nm} must be a torch.Tensor")
            if t.dtype not in _HALVES:
                raise ValueError(f"{nm} must be float16 or bfloat16, got {t.dtype}")
            if t.dim() != 4 or 0 in t.shape:
                raise ValueError(f"{nm} must be [pages, kv heads, page size, dim], got {list(t.shape)}")
            if t.stride(3) != 1 and t.shape[3] > 1:
                raise ValueError(f"{nm}: the values of a row must be contiguous")
            if t.device.type != "cuda":
                raise ValueError(f"{nm} must be on the GPU, got {t.device}")
            _distinct(t, nm)
        if v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must have the same shape, dtype and device")
        self.k, self.v, self.device, self.dtype = k, v, k.device, k.dtype
        self.pages, self.kv_heads, self.page_size, self.dim = (int(n) for n in k.shape)
        if self.pages * self.page_size > 2 ** 31 - 1:
            raise NotImplementedError("more than 2^31 - 1 rows in the cache")
        self._c = _Cache(k.data_ptr(), v.data_ptr(), (ctypes.c_int64 * 3)(*k.stride()[:3]),
                         (ctypes.c_int64 * 3)(*v.stride()[:3]), self.pages, self.kv_heads, self.page_size,
                         self.dim, 1 if k.dtype == torch.bfloat16 else 0)
        self._ref = ctypes.byref(self._c)
        self._need = {}

    def append(self, k, v, slots, *, rotary=None, positions=None, q=None, q_out=None, stream=None):
        """Write the keys (turned by `rotary` at `positions`, copied without
        it) and values [tokens, kv heads, dim] of new tokens to rows slots
        [tokens]: slot s is row s % page_size of page s // page_size; a slot
        outside the cache (-1 for padding) is not written, the others must differ
        (of two tokens with one slot a mixture may be left). With q [tokens,
        heads, dim], returns it turned too (in q_out, which may be q). No
        gradient goes through it (Rotary.rotate has one)."""
        dev, dt, D, kv = self.device, self.dtype, self.dim, self.kv_heads
        (T, _, _), ks = _heads(k, "k", dev, dt, None, kv, D)
        _, vs = _heads(v, "v", dev, dt, T, kv, D)
        sb = _index(slots, "slots", dev, T)
        pb, pp, rh, qa = 32, None, None, (None, 0, 0, None, 0, 0, 0)
        used, written = (k, v, slots), (self.k, self.v)
        if self.k.requires_grad or self.v.requires_grad or forward_ad._current_level >= 0:
            _writable(self.k, "the cache's k")
            _writable(self.v, "the cache's v")
        if rotary is not None:
            if rotary.dim != D:
                raise ValueError(f"rotary turns heads of {rotary.dim} values, the cache has {D}")
            if rotary.device != dev:
                raise ValueError(f"rotary is on {rotary.device}, the cache on {dev}")
            if positions is None:
                raise ValueError("positions are needed with rotary")
            pb, pp, rh = _index(positions, "positions", dev, T), positions.data_ptr(), rotary._handle()
            used += (positions,)
        if q is not None:
            if rotary is None:
                raise ValueError("q is given without rotary")
            (_, H, _), qs = _heads(q, "q", dev, dt, T, None, D)
            if q_out is not None:
                written += (q_out,)
            q_out = _out_like(q, q_out, "q_out", stream)
            if H:
                os_ = q_out.stride()
                qa = (q.data_ptr(), qs[0], qs[1], q_out.data_ptr(), os_[0], os_[1], H)
            used += (q, q_out)
        elif q_out is not None:
            raise ValueError("q_out is given without q")
        _call(load_library().q4_cache_append, "q4_cache_append", dev, stream,
              (self._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slots.data_ptr(), sb, T, rh, pp, pb)
              + qa, used if stream is None else used + (self.k, self.v))
        _wrote(written)
        return q_out

    def attend(self, q, starts, lengths, table, *, window: int = 0, scale=None, out=None, stream=None):
        """Attention of new tokens over the cache: q [tokens, heads, dim] holds
        the new tokens of every request one after the other, request b's are
        rows starts[b] .. starts[b + 1] - 1 (starts int32 [requests + 1]) and
        the last of its lengths[b] cached tokens (lengths int32 [requests]);
        key j is row j % page_size of page table[b, j // page_size] (table int32
        [requests, width]). A token sees the keys up to its own, with `window`
        only the last `window` of them; one that sees none gives zeros. heads is
        a multiple of the cached heads, scale defaults to dim ** -0.5. Lengths
        stay on the device; nothing waits for it. No gradient goes through it.
        Several threads may call at once, on one stream too."""
        dev, dt = self.device, self.dtype
        (T, H, D), qs = _heads(q, "q", dev, dt, None, None, self.dim)
        if H % self.kv_heads or not H:
            raise ValueError(f"q has {H} heads, the cache {self.kv_heads}")
        _int32(starts, "starts", dev, 1)
        _int32(lengths, "lengths", dev, 1)
        _int32(table, "table", dev, 2)
        B, width = table.shape
        if lengths.shape[0] != B or starts.shape[0] != B + 1:
            raise ValueError(f"table [{B}, {width}] takes lengths [{B}] and starts [{B + 1}], got {list(lengths.shape)} "
                             f"and {list(starts.shape)}")
        if (B and width == 0) or (T and not B):
            raise ValueError("table has no pages" if B else f"{T} tokens of no request")
        if not (starts.is_contiguous() and lengths.is_contiguous()) or (width > 1 and table.stride(1) != 1):
            raise ValueError("starts, lengths and the rows of table must be contiguous")
        window = min(int(window), 2 ** 31 - 1)       # (more keys than any cache has)
        if window < 0:
            raise ValueError(f"window must not be negative, got {window}")
        if q.data_ptr() % 16 or qs[0] % 8 or qs[1] % 8:
            if stream is not None:
                q.record_stream(stream)
            q = _on(stream, torch.clone, q, memory_format=_dense)
            qs = q.stride()
        written = out is not None
        if not written:
            out = _out_like(q, None, "out", stream)
        else:
            _heads(out, "out", dev, dt, T, H, D)
            _writable(out, "out")
            _distinct(out, "out")
        ts = table.stride(0)
        if ts < width:
            table, ts = _table_rows(table, stream)
        os_ = out.stride()
        need = self._need.get(H) or self._workspace_bytes(H)
        # (under capture the call's own: a graph may replay beside other work of the
        # stream it was captured on)
        ws = _Workspace() if _capturing(dev, stream) else _workspace(dev, stream)
        with ws.lock:
            if ws.bytes < need:
                ws.hold(_on(stream, _new_workspace, need, dev))
            _call(load_library().q4_attend, "q4_attend", dev, stream,
                  (self._ref, q.data_ptr(), qs[0], qs[1], H, T, starts.data_ptr(), lengths.data_ptr(), table.data_ptr(),
                   width, ts, B, window, D ** -0.5 if scale is None else scale, out.data_ptr(), os_[0], os_[1],
                   ws.at, ws.bytes),
                  () if stream is None else (q, out, starts, lengths, table, self.k, self.v))
        if written:
            _wrote((out,))
        return out

    def _workspace_bytes(self, heads):
        with torch.cuda.device(self.device):
            need = load_library().q4_attend_workspace(self._ref, heads)
        if not need:
            _raise(load_library().q4_last_status(), "q4_attend_workspace")
        self._need[heads] = need
        return need


class _Workspace:
    """A stream's workspace of q4_attend, shared by every cache. A call is up to two
    launches that hand partial results over in it, and several threads may use one
    stream (the default one is every thread's): the lock keeps a call's launches side by
    side, and the memory until they are made."""
    __slots__ = ("lock", "at", "bytes", "memory")

    def __init__(self):
        self.lock, self.at, self.bytes, self.memory = threading.Lock(), None, 0, None

    def hold(self, memory):
        self.at, self.bytes, self.memory = memory.data_ptr(), memory.numel(), memory


_workspaces: dict = {}      # (device, stream) -> its _Workspace


def _workspace(device, stream):
    key = (device.index, _raw_stream(device.index) if stream is None else stream.cuda_stream)
    # (setdefault: two threads that come first get one and the same)
    return _workspaces.get(key) or _workspaces.setdefault(key, _Workspace())


_WORKSPACE_ZEROS = 1 << 16  # bytes of it that q4_attend wants zero before the first call


def _new_workspace(n, device):
    # (a graph makes one at each replay: filling it all took longer than a small call)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:_WORKSPACE_ZEROS].zero_()
    return ws


def _capturing(device, stream):
    """Whether the stream that a call runs on is being captured."""
    if stream is None:
        if _device() == device.index:
            return torch.cuda.is_current_stream_capturing()
        stream = torch.cuda.current_stream(device)
    return _on(stream, torch.cuda.is_current_stream_capturing)


def _on(stream, f, *args, **kw):
    if stream is None:
        return f(*args, **kw)
    with torch.cuda.stream(stream):
        return f(*args, **kw)
