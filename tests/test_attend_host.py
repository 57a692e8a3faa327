"""What attention over the paged cache and the adapters refuse before any GPU
call."""
import ctypes
import math

import pytest

import gptq_bit_weight_amd as q4


def _attend(lib, cache=None, **kw):
    from gptq_bit_weight_amd.attention import _Cache
    c = _Cache(4096, 8192, (ctypes.c_int64 * 3)(2048, 1024, 64), (ctypes.c_int64 * 3)(2048, 1024, 64), 4, 2, 16, 64, 0)
    for k, v in (cache or {}).items():
        if k in ("k_stride", "v_stride"):
            v = (ctypes.c_int64 * 3)(*v)
        setattr(c, k, v)
    a = dict(q=4096, q_token=512, q_head=64, heads=8, tokens=3, starts=4096, lengths=4096, table=4096, width=2, stride=2,
             requests=2, window=0, scale=0.125, out=65536, o_token=512, o_head=64, ws=4096, ws_bytes=1 << 40)
    a.update(kw)
    return lib.q4_attend(ctypes.byref(c), a["q"], a["q_token"], a["q_head"], a["heads"], a["tokens"], a["starts"],
                         a["lengths"], a["table"], a["width"], a["stride"], a["requests"], a["window"], a["scale"],
                         a["out"], a["o_token"], a["o_head"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("cache,kw,status", [
    (dict(k=None), {}, 1), (dict(dim=60), {}, 2), (dict(dim=264), {}, 2), (dict(pages=0), {}, 1),
    (dict(k_stride=(2048, 1024, 60)), {}, 2), (dict(v_stride=(2044, 1024, 64)), {}, 2), (dict(k=4104), {}, 2),
    (dict(k_stride=(2048, 1024, 1 << 26)), {}, 2), (dict(k_stride=(-2048, 1024, 64)), {}, 2),
    ({}, dict(heads=0), 1), ({}, dict(heads=7), 1), ({}, dict(tokens=-1), 1), ({}, dict(requests=-1), 1),
    ({}, dict(window=-1), 1), ({}, dict(scale=math.nan), 1), ({}, dict(scale=math.inf), 1), ({}, dict(q=None), 1),
    ({}, dict(starts=None), 1), ({}, dict(lengths=None), 1), ({}, dict(table=None), 1), ({}, dict(out=None), 1),
    ({}, dict(width=0), 1), ({}, dict(stride=1), 1), ({}, dict(q=4098), 2), ({}, dict(q_token=508), 2),
    ({}, dict(tokens=1 << 30), 2),
])
def test_attend_refuses(cache, kw, status):
    lib = q4.load_library()
    assert _attend(lib, cache, **kw) == status
    assert lib.q4_last_error()


def test_attend_of_nothing():
    lib = q4.load_library()
    assert _attend(lib, tokens=0) == 0
    assert _attend(lib, requests=0) == 0


@pytest.mark.parametrize("slots,rank,status", [(0, 8, 1), (3, 0, 1), (-1, 8, 1), (4097, 8, 2), (3, 1025, 2), (4096, 1024, 0)])
def test_adapters_sizes(slots, rank, status):
    assert q4.load_library().q4_check_adapters(slots, rank) == status


def test_adapters_null():
    lib = q4.load_library()
    assert lib.q4_adapters_make(None, 3, 8, 0) is None
    assert lib.q4_last_status() == 1
    assert lib.q4_adapters_load(None, 0, 4096, 4096, 8, 1.0, None) == 1
    assert lib.q4_adapters_load(None, 0, None, 4096, 8, 1.0, None) == 1
    assert lib.q4_adapters_clear(None, 0, None) == 1
    assert lib.q4_matmul_adapters(None, None, 4096, None, 4096, 8192, 1, 0, None) == 1
    lib.q4_adapters_free(None)


def test_table_rows_that_share_memory():
    """The row stride handed to the C call is one that the tensor has: rows that
    share memory are copied, a single row's stride does not count."""
    import torch
    from gptq_bit_weight_amd.attention import _table_rows
    base = torch.arange(60, dtype=torch.int32)
    cases = [base[:7].expand(5, 7), base[:7][None].expand(5, 7), base.as_strided((4, 6), (3, 1)), base[:3, None].expand(3, 1),
             base[:1].expand(4, 1), base.view(10, 6), base.view(10, 6)[::2, :4], base.view(10, 6)[:1, :4], base.as_strided((1, 5), (0, 1)),
             base.as_strided((1, 5), (2, 1))]
    for t in cases:
        got, stride = _table_rows(t)
        B, width = t.shape
        assert stride >= width and torch.equal(got, t)
        # what the kernel reads: entry (b, i) at b * stride + i, inside the tensor's storage
        at = got.storage_offset() + torch.arange(B)[:, None] * stride + torch.arange(width)
        whole = torch.empty(0, dtype=torch.int32).set_(got.untyped_storage())
        assert int(at.max()) < whole.numel()
        assert torch.equal(whole[at], t)
    t = base.view(10, 6)
    assert _table_rows(t)[0] is t                # (rows apart are taken as they are)


def test_calls_of_two_threads_on_one_stream_follow_each_other(monkeypatch):
    """The C call makes two launches that share the stream's workspace: another
    thread's may not come between them, nor free the workspace before them."""
    import threading
    import time

    import torch
    from gptq_bit_weight_amd import attention

    inside, most, sizes, errors = [], [], [], []

    class Library:
        @staticmethod
        def q4_attend(*a):
            inside.append(1)
            most.append(len(inside))
            at, n = a[-3], a[-2]
            time.sleep(0.002)
            sizes.append((at, n) if any(w.memory is not None and w.at == at and w.memory.numel() >= n
                                        for w in attention._workspaces.values()) else None)
            inside.pop()
            return 0

    monkeypatch.setattr(attention, "load_library", lambda: Library)
    monkeypatch.setattr(attention, "_raw_stream", lambda i: 7)
    monkeypatch.setattr(attention, "_device", lambda: None)
    monkeypatch.setattr(attention, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    def cache(need):
        c = object.__new__(attention.PagedCache)
        c.device, c.dtype, c.dim, c.kv_heads, c._need, c._ref = torch.device("cpu"), torch.float16, 64, 2, {4: need}, None
        c.k = c.v = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
        return c

    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    starts, lengths = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)

    def work(c):
        try:
            for _ in range(20):
                c.attend(q, starts, lengths, table)
        except Exception as e:      # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(cache(1 << 16 + i),)) for i in (1, 0, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert len(most) == 60 and max(most) == 1
    assert None not in sizes


@pytest.mark.parametrize("captured", ["given", "current", "neither"])
def test_a_captured_stream_that_is_not_the_current_one(monkeypatch, captured):
    """It is the stream the call runs on that counts: a graph gets a workspace of
    its own, an eager call the stream's."""
    import contextlib

    import torch
    from gptq_bit_weight_amd import attention

    seen, now = [], ["current"]

    class Library:
        @staticmethod
        def q4_attend(*a):
            seen.append(a[-3])
            return 0

    class Stream:
        device, cuda_stream = torch.device("cpu"), 9

    @contextlib.contextmanager
    def stream(s):
        was, now[0] = now[0], "given" if isinstance(s, Stream) else s
        yield
        now[0] = was

    monkeypatch.setattr(attention, "load_library", lambda: Library)
    monkeypatch.setattr(attention, "_raw_stream", lambda i: 7)
    monkeypatch.setattr(attention, "_device", lambda: None)
    monkeypatch.setattr(attention, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0] == captured)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    c = object.__new__(attention.PagedCache)
    c.device, c.dtype, c.dim, c.kv_heads, c._need, c._ref = torch.device("cpu"), torch.float16, 64, 2, {4: 1 << 16}, None
    c.k = c.v = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    starts, lengths = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    c.attend(q, starts, lengths, table, stream=Stream())
    c.attend(q, starts, lengths, table)
    held = [attention._workspaces.get((None, h)) for h in (9, 7)]
    for workspace, at, which in zip(held, seen, ("given", "current")):
        assert (workspace is None) == (captured == which)
        assert workspace is None or workspace.at == at


@pytest.mark.parametrize("window", [0, 7, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 10 ** 30])
def test_no_window_is_cut_to_32_bits(monkeypatch, window):
    """What the C call gets, an int, is the window or at least every row of the cache."""
    import torch
    from gptq_bit_weight_amd import attention

    seen = []

    class Library:
        @staticmethod
        def q4_attend(*a):
            seen.append(a[12])
            return 0

    monkeypatch.setattr(attention, "load_library", lambda: Library)
    monkeypatch.setattr(attention, "_raw_stream", lambda i: 7)
    monkeypatch.setattr(attention, "_device", lambda: None)
    monkeypatch.setattr(attention, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    c = object.__new__(attention.PagedCache)
    c.device, c.dtype, c.dim, c.kv_heads, c._need, c._ref = torch.device("cpu"), torch.float16, 64, 2, {4: 1 << 16}, None
    c.k = c.v = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    c.attend(torch.zeros(3, 4, 64, dtype=torch.float16), torch.tensor([0, 3], dtype=torch.int32),
             torch.tensor([20], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32), window=window)
    got = ctypes.c_int(seen[0]).value
    assert got == seen[0] and (got == window or got >= 2 * 16)


# out is 3 tokens of 8 heads of 64 at 65536: 1024 bytes a token. (Each call is refused
# later on too, for its workspace or the missing device: nothing is launched.)
@pytest.mark.parametrize("cache,kw,meets", [
    ({}, {}, False), ({}, dict(q=65536), True), ({}, dict(q=65536 + 2048), True), ({}, dict(q=65536 + 1024, o_token=1024, q_token=1024), False),
    ({}, dict(q=65536 + 1024, o_token=1024, q_token=1032), True), (dict(k=65536), {}, True), (dict(v=65536 - 1024), {}, True),
    (dict(k=65536 - 16384), {}, False), (dict(v=65536 + 3072), {}, False), ({}, dict(starts=65536 - 8), True),
    ({}, dict(starts=65536 - 12), False), ({}, dict(lengths=65536 + 3068), True), ({}, dict(table=65536 - 12, stride=3), True),
    ({}, dict(table=65536 - 20, stride=3), False),
])
def test_attend_out_that_meets_an_input(cache, kw, meets):
    lib = q4.load_library()
    assert _attend(lib, cache, ws=None, **kw) != 0
    assert (b"overlaps" in lib.q4_last_error()) == meets


def _stand_in(monkeypatch):
    """The binding over a library that does nothing, on CPU tensors."""
    import torch
    from gptq_bit_weight_amd import attention

    class Library:
        q4_attend = q4_cache_append = q4_rotary_apply = staticmethod(lambda *a: 0)

    monkeypatch.setattr(attention, "load_library", lambda: Library)
    monkeypatch.setattr(attention, "_raw_stream", lambda i: 7)
    monkeypatch.setattr(attention, "_device", lambda: None)
    monkeypatch.setattr(attention, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    c = object.__new__(attention.PagedCache)
    c.device, c.dtype, c.dim, c.kv_heads, c._need, c._ref = torch.device("cpu"), torch.float16, 64, 2, {4: 1 << 16}, None
    c.k, c.v = torch.zeros(2, 2, 2, 16, 64, dtype=torch.float16).clone().unbind(0)
    r = object.__new__(attention.Rotary)
    r.device, r.dim, r._h = torch.device("cpu"), 64, 1
    monkeypatch.setattr(attention.Rotary, "close", lambda self: None)
    return c, r


def test_writes_in_place_are_told_to_autograd(monkeypatch):
    """Outputs that the caller gives, and the cache: a tensor saved for a backward
    pass is found changed, one that requires a gradient is refused."""
    import torch
    c, r = _stand_in(monkeypatch)
    T = 3
    make = lambda h: torch.randn(T, h, 64).half()  # noqa: E731
    pos = torch.arange(T)
    starts, lengths = torch.tensor([0, T], dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    calls = {
        "rotate": lambda t: r.rotate(t, pos, out=t),
        "append": lambda t: c.append(make(2), make(2), pos, rotary=r, positions=pos, q=t, q_out=t),
        "attend": lambda t: c.attend(make(4), starts, lengths, table, out=t),
    }
    for name, call in calls.items():
        w = torch.ones(T, 4, 64, dtype=torch.float16, requires_grad=True)
        t = make(4)
        y = (w * t).sum()                        # saves t
        at = t._version
        call(t)
        assert t._version > at, name
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        for leaf in (make(4).requires_grad_(), make(4).requires_grad_() * 1):
            with pytest.raises(ValueError, match="requires a gradient"):
                call(leaf)
            with torch.no_grad():
                at = leaf._version
                call(leaf)
                assert leaf._version > at, name
        with torch.inference_mode():
            call(make(4))
    at = c.k._version, c.v._version
    c.append(make(2), make(2), pos)
    assert c.k._version > at[0] and c.v._version > at[1]
    c.v.requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        c.append(make(2), make(2), pos)
    with torch.no_grad():
        c.append(make(2), make(2), pos)
    # what the calls make themselves is not written in place
    assert r.rotate(make(4), pos)._version == 0 and c.attend(make(4), starts, lengths, table)._version == 0


def test_the_host_only_part_needs_no_torch():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.modules['torch'] = None; from gptq_bit_weight_amd import *; check_shape(128, 64, 64); "
            "import gptq_bit_weight_amd as q4; q4.Q4Adapters")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-500:]
    from gptq_bit_weight_amd import PagedCache, Rotary
    assert PagedCache is q4.PagedCache and Rotary is q4.Rotary
