"""Which pages of a cache hold which request's tokens, on the device: pages are
allotted, shared, given back and moved by kernels, so that a serving step is
launched (or captured) as a whole without the host knowing a length.

    pages = q4.Pages(cache, requests=64, width=128)
    slots = pages.extend(starts, tokens)             # room for new tokens
    q = cache.append(k, v, slots, rotary=rope, positions=positions, q=q)
    o = cache.attend(q, starts, pages.lengths, pages.table)
    pages.fork(parents, children); pages.free(done); pages.trim(window, sinks); pages.compact()
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import load_library
from .attention import _Paged, _call, _index, _int32, _on, _wrote

__all__ = ["Pages"]


class _Pages(ctypes.Structure):
    """q4_pages of include/q4.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "lengths", "counts", "work")] + [
        (n, ctypes.c_int) for n in ("requests", "width", "pages", "page_size")]


class Pages:
    """The books of a PagedCache or PagedCache4 for up to `requests` requests of at
    most `width` pages: `table` int32 [requests, width], `lengths` int32 [requests]
    (tokens in the cache, as attend() takes them) and `counts` int32 [pages], how many
    entries of requests name a page (0: it is free). The tensors may be read, and
    written by who keeps them in step. All calls are asynchronous, may be captured, and
    belong on one stream at a time.

    fork() and compact() copy pages of `cache` alone. Layers that share one table are
    therefore heads of one pool: k [pages, layers * kv heads, page size, dim], of which
    layer l appends to and attends over a cache of the slice k[:, l * kv:(l + 1) * kv],
    and Pages gets the cache over all of it."""

    def __init__(self, cache, requests: int, width: int):
        if not isinstance(cache, _Paged):
            raise TypeError(f"cache must be a PagedCache or PagedCache4, got {type(cache).__name__}")
        requests, width = int(requests), int(width)
        if requests < 1 or width < 1:
            raise ValueError(f"{requests} requests of {width} pages")
        if requests * width > 1 << 30 or width * cache.page_size > 1 << 30:
            raise NotImplementedError(f"{requests} requests of {width} pages of {cache.page_size} rows")
        dev = self.device = cache.device
        self.cache, self.requests, self.width = cache, requests, width
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.counts = torch.zeros(cache.pages, dtype=torch.int32, device=dev)
        need = load_library().q4_pages_workspace(requests, cache.pages)
        self._work = torch.empty(need // 4, dtype=torch.int32, device=dev)
        self._tensors = (self.table, self.lengths, self.counts, self._work)
        self._c = _Pages(*(t.data_ptr() for t in self._tensors), requests, width, cache.pages, cache.page_size)
        self._ref = ctypes.byref(self._c)
        # (a call is up to two launches that share the scratch)
        self._lock = threading.Lock()

    def _run(self, what, stream, args, used=(), writes=()):
        with self._lock:
            _call(getattr(load_library(), what), what, self.device, stream, (self._ref,) + args,
                  () if stream is None else self._tensors + tuple(used) + tuple(writes))
        _wrote(self._tensors[:3] + tuple(writes))

    def _list(self, t, name, n=None):
        if n is None:
            n = t.shape[0] if isinstance(t, torch.Tensor) and t.dim() == 1 else -1
        return t.data_ptr(), _index(t, name, self.device, n), n

    def extend(self, starts, tokens: int, *, stream=None):
        """Room for `tokens` new tokens, request r's starts[r] .. starts[r + 1] - 1 of
        them (int32 [requests + 1], from 0): lengths grow, the lowest free pages are
        taken, and the slots for append() are returned, int32 [tokens]. A request whose
        row of the table is too short gets nothing, and neither does one that
        the free pages do not suffice for, nor any after it that needs some: its length
        stays and its slots are -1."""
        _int32(starts, "starts", self.device, 1)
        tokens = int(tokens)
        if starts.shape[0] != self.requests + 1 or not starts.is_contiguous() or not 0 <= tokens <= 1 << 30:
            raise ValueError(f"starts must be contiguous with shape [{self.requests + 1}], got {list(starts.shape)} for {tokens} tokens")
        slots = _on(stream, self.lengths.new_empty, tokens)
        self._run("q4_pages_extend", stream, (starts.data_ptr(), tokens, slots.data_ptr()), (starts,))
        return slots

    def fork(self, parents, children, *, stream=None):
        """Request children[i] (one without tokens) becomes a copy of request parents[i]
        (int32 or int64 [n]): they share its pages, but a last one that is not full,
        which is copied. Returns int32 [n], 1 where that was done: not for an index
        outside the requests, a child that has tokens or that an earlier pair names, or
        where no free page was left. All pairs see the requests as they were before."""
        pp, pb, n = self._list(parents, "parents")
        cp, cb, _ = self._list(children, "children", n)
        written = self.cache._writes()
        done = _on(stream, self.lengths.new_empty, (2, n))
        self._run("q4_pages_fork", stream, (self.cache._pool(), pp, pb, cp, cb, n, done.data_ptr()),
                  (parents, children), written)
        return done.select(0, 0)

    def free(self, requests, *, stream=None):
        """Gives back the pages of requests (int32 or int64 [n]; one named twice is freed
        once, one outside not at all): their lengths are 0, their entries -1."""
        p, bits, n = self._list(requests, "requests")
        self._run("q4_pages_free", stream, (p, bits, n), (requests,))

    def trim(self, window: int, sinks: int = 0, *, stream=None):
        """Gives back the pages that no later token sees anything of with this window and
        these sinks; their entries are -1. Comes after attend() for the tokens that
        extend() made room for."""
        window, sinks = min(int(window), 2 ** 31 - 1), min(int(sinks), 2 ** 31 - 1)
        if window < 1 or sinks < 0:
            raise ValueError(f"window {window}, {sinks} sinks")
        self._run("q4_pages_trim", stream, (window, sinks))

    def compact(self, *, stream=None):
        """Moves pages so that those in use come first. Returns int32 [pages]: where each page
        went, -1 for one that was free."""
        written = self.cache._writes()
        to = _on(stream, self.counts.new_empty, self.cache.pages)
        self._run("q4_pages_compact", stream, (self.cache._pool(), to.data_ptr()), (), written)
        return to
