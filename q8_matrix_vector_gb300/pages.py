"""Pages of a cache: Python binding of ``include/kvpage.h``.

``Pages`` keeps which request holds which pages of a ``Cache`` or ``Cache4`` on the device: pages are given out as
requests grow, shared when one is forked, copied when a shared one would be written, given back, and brought together.
Nothing waits for the host, so a decode step with it can be a CUDA graph.  This module only checks arguments and passes
device pointers and the current stream to ``libq8mv.so``.
"""
from __future__ import annotations

import ctypes

import torch

from .kv import _current, _elsewhere, _fail, _ints, _library, _Plan, _stream


class State(ctypes.Structure):
    """kvpage_state_t"""
    _fields_ = [("refs", ctypes.c_void_p), ("table", ctypes.c_void_p), ("held", ctypes.c_void_p)]


def _bind(lib: ctypes.CDLL) -> None:
    i32, i64, p, ref = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.POINTER
    for name, args in (
            ("kvpage_plan", [ref(p), i64, i32, i32, i32, ctypes.c_int]),
            ("kvpage_extend", [p, ref(State), p, p, i32, p, p, p, p, p]),
            ("kvpage_fork", [p, ref(State), p, p]),
            ("kvpage_free", [p, ref(State), p, p]),
            ("kvpage_compact", [p, ref(State), p, p, p, p]),
            ("kvpage_destroy", [p])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int


_bind(_library())


class Pages(_Plan):
    """Who holds which of ``pages`` pages of ``page_size`` tokens, for ``requests`` requests of up to ``columns`` pages.

    The state is three int32 tensors: ``refs`` [pages] (holders of a page, 0: free), ``table`` [requests, columns] (a
    request's pages in order, -1 behind: the table that attention takes) and ``held`` [requests].  Copies of them are
    snapshots that can be copied back.  Calls on one object must be ordered (one stream, or otherwise).
    """

    _destroy = "kvpage_destroy"

    def __init__(self, pages: int, page_size: int, requests: int, columns: int, device: int = -1):
        self.pages, self.page_size, self.requests, self.columns = pages, page_size, requests, columns
        self._make("kvpage_plan", pages, page_size, requests, columns, int(device))
        self._refs = torch.zeros(pages, dtype=torch.int32, device=self._where)
        self._table = torch.full((requests, columns), -1, dtype=torch.int32, device=self._where)
        self._held = torch.zeros(requests, dtype=torch.int32, device=self._where)
        self._state = State(self._refs.data_ptr(), self._table.data_ptr(), self._held.data_ptr())
        self._ref = ctypes.byref(self._state)
        lib = _library()
        self._extend, self._fork, self._free, self._compact = (getattr(lib, "kvpage_" + n) for n in
                                                               ("extend", "fork", "free", "compact"))

    # the library has their addresses: they are written to, not replaced
    refs, table, held = (property(lambda self, n=n: getattr(self, n)) for n in ("_refs", "_table", "_held"))

    def _run(self, fn, what, *args):
        device = self.device
        if _current() == device:
            status = fn(self._h, self._ref, *args, _stream(device))
        else:
            status = _elsewhere(fn, device, self._h, self._ref, *args)
        if status:
            _fail(status, what)

    def extend(self, lengths, tokens, width: int):
        """Pages for tokens[b] more tokens past the first lengths[b] ([requests] int32 each) of each request: fresh ones,
        the lowest free, past those that it holds, and in place of shared ones that these tokens are written to.

        Returns (slots [requests, width] int64, src, dst, ok [requests] int32): the slots of the first ``width`` new
        tokens, -1 behind the last; a page that was shared and is about to be written, and its copy, -1 for none (call
        ``copy_pages(src, dst)`` of every cache next); and 0 for a request that got nothing and stays as it was, as
        there are not enough free pages for all up to it, or not enough columns."""
        device, n = self.device, self.requests
        if width < 0:
            raise ValueError(f"width must not be negative, got {width}")
        at_lengths = _ints(lengths, torch.int32, n, device, "lengths")
        at_tokens = _ints(tokens, torch.int32, n, device, "tokens")
        slots = torch.empty((n, width), dtype=torch.int64, device=self._where)
        held = self._held
        src, dst, ok = torch.empty_like(held), torch.empty_like(held), torch.empty_like(held)
        self._run(self._extend, "kvpage_extend", at_lengths, at_tokens, width, slots.data_ptr(), src.data_ptr(),
                  dst.data_ptr(), ok.data_ptr())
        return slots, src, dst, ok

    def fork(self, parents) -> None:
        """Each request b becomes what parents[b] ([requests] int32) was, all at once, sharing its pages; it gives back
        what it held.  parents[b] = b changes nothing; a parent that is no request, as -1, leaves b without pages."""
        self._run(self._fork, "kvpage_fork", _ints(parents, torch.int32, self.requests, self.device, "parents"))

    def free(self, lengths) -> None:
        """Each request keeps the pages of its first lengths[b] tokens ([requests] int32; 0: none) and gives the others
        back: those of drafts that were not accepted, or of a request that has ended."""
        self._run(self._free, "kvpage_free", _ints(lengths, torch.int32, self.requests, self.device, "lengths"))

    def compact(self):
        """Moves the held pages to the lowest numbers.  Returns (src, dst [pages // 2], count [1], int32): pages
        src[i] are dst[i] now for i < count, -1 behind (call ``copy_pages(src, dst, count)`` of every cache next)."""
        most = self.pages // 2
        src = torch.empty(most, dtype=torch.int32, device=self._where)
        dst, count = torch.empty_like(src), torch.empty(1, dtype=torch.int32, device=self._where)
        self._run(self._compact, "kvpage_compact", src.data_ptr(), dst.data_ptr(), count.data_ptr())
        return src, dst, count
