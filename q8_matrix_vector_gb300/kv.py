"""A Q8_0 key/value cache and the decode operators on it: Python binding of ``include/q8kv.h``.

``Cache`` writes, reads and moves rows, ``TreeAttention`` attends draft trees (a single token is a tree of
one) over it, ``TreeVerify`` decides which drafted tokens are kept.  As in the rest of the package this
module only checks arguments and passes device pointers and the current stream to ``libq8mv.so``.

The checks are written for their own cost: a decode step makes these calls once per layer, and most of
them last a few microseconds on the GPU.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class CacheDesc(ctypes.Structure):
    """q8kv_cache_t"""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("stride_page", ctypes.c_int64), ("stride_head", ctypes.c_int64), ("stride_token", ctypes.c_int64)]


class AttendArgs(ctypes.Structure):
    """q8kv_attend_args_t"""
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("type", ctypes.c_int32),
                ("requests", ctypes.c_int32), ("rows", ctypes.c_int64), ("q_row", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("out_row", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("starts", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_row", ctypes.c_int64), ("table_cols", ctypes.c_int32), ("mask_words", ctypes.c_int32),
                ("mask", ctypes.c_void_p), ("mask_row", ctypes.c_int64), ("scale", ctypes.c_float)]


class VerifyArgs(ctypes.Structure):
    """q8kv_verify_args_t"""
    _fields_ = [("logits", ctypes.c_void_p), ("draft_probs", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("parents", ctypes.c_void_p), ("uniforms", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("path", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("next_token", ctypes.c_void_p), ("logits_row", ctypes.c_int64), ("draft_row", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("requests", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


# One pack instead of an attribute store per field, into bytes of the call's own: the library reads them without the
# interpreter's lock, while another thread may make a call of the same object.
_ATTEND = struct.Struct("=3Qii5q3QqiiQqf4x")
_VERIFY = struct.Struct("=10Q3qiiii")
assert _ATTEND.size == ctypes.sizeof(AttendArgs) and _VERIFY.size == ctypes.sizeof(VerifyArgs)


def _bind(lib: ctypes.CDLL) -> None:
    """Declare the q8kv entry points of the loaded library: undeclared, ctypes would cut pointers to 32 bits."""
    i32, i64, p, ref = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.POINTER
    for name, args in (
            ("q8kv_cache_write", [ref(CacheDesc), i64, p, p, i32, i64, i64, i64, i64, p, p]),
            ("q8kv_cache_read", [ref(CacheDesc), i64, p, p, p, i32, p]),
            ("q8kv_cache_move", [ref(CacheDesc), i64, i64, p, p, p]),
            ("kvpage_copy_q8", [ref(CacheDesc), i64, p, p, p, p]),
            ("q8kv_attend_plan", [ref(p), i32, i32, i32, i32, i64, ctypes.c_int]),
            ("q8kv_attend", [p, ref(CacheDesc), p, p]),
            ("q8kv_attend_check", [p, ref(i32)]),
            ("q8kv_attend_set_wait", [p, ctypes.c_uint64]),
            ("q8kv_attend_destroy", [p]),
            ("q8kv_verify_plan", [ref(p), i32, i64, i32, ctypes.c_int]),
            ("q8kv_verify", [p, p, p]),
            ("q8kv_verify_destroy", [p])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int


def _library():
    from . import _lib

    return _lib


_bind(_library())


def _fail(status: int, what: str):
    from . import Q8mvError

    raise Q8mvError(status, what)


# the raw handle of a device's current stream, and the current device: without the objects and the
# initialisation checks of torch.cuda's own functions, several times their cost
_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice


def _elsewhere(fn, device, *args):
    """fn(*args, current stream) with another device than the current one."""
    with torch.cuda.device(device):
        return fn(*args, _stream(device))


def _ints(t, dtype, numel, device, name):
    """A contiguous device tensor of `numel` numbers of one type (-1: any number): its address."""
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous() and (numel < 0 or t.numel() == numel):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def _rows(t, tail, device, name):
    """A floating [n, *tail] device tensor whose last axis is contiguous: (n, type code, strides)."""
    code = _TYPES.get(t.dtype)
    shape, stride = t.shape, t.stride()
    if code is not None and t.get_device() == device and shape[1:] == tail and (stride[-1] == 1 or tail[-1] == 1):
        return shape[0], code, stride
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if tuple(shape[1:]) != tail:
        raise ValueError(f"{name} must have shape (n, {', '.join(map(str, tail))}), got {tuple(shape)}")
    raise ValueError(f"{name}'s last axis must be contiguous")


def _strides(parts, shape):
    """The strides in rows of a cache's four arrays, (name, tensor, type, row's elements) each, of [pages, heads,
    page_size, ...]: each row contiguous, all with the same strides, no two rows in the same place."""
    device, strides = parts[0][1].get_device(), None
    if device < 0:
        raise ValueError(f"{parts[0][0]} must be a CUDA tensor")
    for name, t, dtype, width in parts:
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != (*shape, width):
            raise ValueError(f"{name} must have shape {(*shape, width)}, got {tuple(t.shape)}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
        if t.data_ptr() % 16:
            raise ValueError(f"{name} must be 16-byte aligned")
        stride = t.stride()
        if (width > 1 and stride[3] != 1) or any(s % width for n, s in zip(t.shape, stride[:3]) if n > 1):
            raise ValueError(f"{name}'s rows must be contiguous and whole rows apart")
        if any(s < width for n, s in zip(t.shape, stride[:3]) if n > 1):
            raise ValueError(f"{name} is expanded: its rows overlap")
        # the stride of an axis of one element says nothing
        mine = tuple(s // width if n > 1 else 1 for n, s in zip(t.shape, stride[:3]))
        if strides is not None and mine != strides:
            raise ValueError(f"{name} must have the strides of {parts[0][0]}, counted in rows")
        strides = mine
    # rows that meet would be written twice
    order = sorted((s, n) for s, n in zip(strides, shape) if n > 1)
    reach = 1
    for s, n in order:
        if s < reach:
            raise ValueError("the cache's rows overlap")
        reach = s * (n - 1) + reach
    return strides


class Cache:
    """A paged Q8_0 key/value cache: int8 codes and one f32 scale per 32 of a row.

    ``Cache(pages, page_size, heads, head_dim)`` allocates one (``layout`` "head" keeps a page's tokens of one
    head together, "token" a token's heads); ``Cache.of`` takes existing tensors.  Token slot s is place
    s % page_size of page s // page_size.
    """

    _prefix = "q8kv_cache"  # of its entry points
    _copier, _fused = "kvpage_copy_q8", "kvrope_write_q8"

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, device="cuda", layout: str = "head"):
        if layout not in ("head", "token"):
            raise ValueError(f"layout must be 'head' or 'token', got {layout!r}")
        if head_dim % 16 != 0 or not 16 <= head_dim <= 256:
            raise ValueError(f"head_dim must be a multiple of 16 up to 256, got {head_dim}")
        shape = (pages, heads, page_size) if layout == "head" else (pages, page_size, heads)
        parts = []
        for _ in range(2):
            for width, dtype in ((head_dim, torch.int8), ((head_dim + 31) // 32, torch.float32)):
                t = torch.zeros(*shape, width, dtype=dtype, device=device)
                parts.append(t if layout == "head" else t.transpose(1, 2))
        self._take(*parts)

    @classmethod
    def of(cls, k_codes, k_scales, v_codes, v_scales) -> "Cache":
        """A cache over existing tensors: codes [pages, heads, page_size, head_dim] int8 and scales
        [pages, heads, page_size, ceil(head_dim / 32)] f32, each row contiguous, all four with the same strides
        counted in rows (permuted views of other orders are fine)."""
        self = cls.__new__(cls)
        self._take(k_codes, k_scales, v_codes, v_scales)
        return self

    def _take(self, k_codes, k_scales, v_codes, v_scales):
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes must have 4 axes, got {k_codes.dim()}")
        pages, heads, page_size, dim = k_codes.shape
        blocks = (dim + 31) // 32
        strides = _strides((("k_codes", k_codes, torch.int8, dim), ("k_scales", k_scales, torch.float32, blocks),
                            ("v_codes", v_codes, torch.int8, dim), ("v_scales", v_scales, torch.float32, blocks)),
                           (pages, heads, page_size))
        self._keep(k_codes, k_scales, v_codes, v_scales, dim)
        self._desc = CacheDesc(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), pages,
                               page_size, heads, dim, 0, *strides)
        self._ref = ctypes.byref(self._desc)

    def _keep(self, k_codes, k_scales, v_codes, v_scales, dim):
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.pages, self.heads, self.page_size = k_codes.shape[:3]
        self.head_dim = dim
        self.device, self._where = k_codes.get_device(), k_codes.device
        self._tail = (self.heads, dim)
        lib, prefix = _library(), self._prefix
        self._write, self._read, self._move = (getattr(lib, f"{prefix}_{n}") for n in ("write", "read", "move"))
        self._copy = getattr(lib, self._copier)

    def write(self, k, v, slots) -> None:
        """Quantise keys and values [n, heads, head_dim] (f32, f16 or bf16) into slots [n] (int64, each once;
        slots outside the cache, as -1, are skipped)."""
        device, tail = self.device, self._tail
        n, code, ks = _rows(k, tail, device, "k")
        n_v, code_v, vs = _rows(v, tail, device, "v")
        if code_v != code or n_v != n:
            raise ValueError("k and v must have the same type and number of tokens")
        at = _ints(slots, torch.int64, n, device, "slots")
        if _current() == device:
            status = self._write(self._ref, n, k.data_ptr(), v.data_ptr(), code, ks[0], ks[1], vs[0], vs[1], at, _stream(device))
        else:
            status = _elsewhere(self._write, device, self._ref, n, k.data_ptr(), v.data_ptr(), code, ks[0], ks[1], vs[0],
                                vs[1], at)
        if status:
            _fail(status, self._prefix + "_write")

    def read(self, slots, dtype=torch.float32, out=None):
        """(k, v) [n, heads, head_dim] of slots [n] (int64) in ``dtype``; zeros for slots outside the cache."""
        device = self.device
        at = _ints(slots, torch.int64, -1, device, "slots")
        n = slots.numel()
        if out is None:
            code = _TYPES.get(dtype)
            if code is None:
                raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
            k = torch.empty((n, *self._tail), dtype=dtype, device=self._where)
            v = torch.empty_like(k)
        else:
            k, v = out
            n_k, code, _ = _rows(k, self._tail, device, "out[0]")
            n_v, code_v, _ = _rows(v, self._tail, device, "out[1]")
            if code != code_v or n_k != n or n_v != n or not k.is_contiguous() or not v.is_contiguous():
                raise ValueError(f"out must be two contiguous tensors of one type with {n} tokens")
        if _current() == device:
            status = self._read(self._ref, n, at, k.data_ptr(), v.data_ptr(), code, _stream(device))
        else:
            status = _elsewhere(self._read, device, self._ref, n, at, k.data_ptr(), v.data_ptr(), code)
        if status:
            _fail(status, self._prefix + "_read")
        return k, v

    def move(self, src, dst) -> None:
        """Slots dst[b, i] become copies of src[b, i] ([batch, path] int64), i in order within a request; pairs
        with a slot outside the cache are skipped, and slots of different requests must not meet."""
        device = self.device
        a = _ints(src, torch.int64, -1, device, "src")
        shape = src.shape
        if shape != dst.shape or not 1 <= len(shape) <= 2:
            raise ValueError(f"src and dst must be [batch, path], got {tuple(src.shape)} and {tuple(dst.shape)}")
        batch, path = shape if len(shape) == 2 else (1, shape[0])
        b = _ints(dst, torch.int64, -1, device, "dst")
        if _current() == device:
            status = self._move(self._ref, batch, path, a, b, _stream(device))
        else:
            status = _elsewhere(self._move, device, self._ref, batch, path, a, b)
        if status:
            _fail(status, self._prefix + "_move")

    def copy_pages(self, src, dst, count=None) -> None:
        """Pages dst[i] become copies of pages src[i] ([n] int32), all heads, for the first ``count`` pairs ([1] int32
        on the device; None: all); pairs with a page outside the cache, as -1, are skipped.  A page may be the source of
        several; no destination may be another pair's source or destination."""
        device = self.device
        a = _ints(src, torch.int32, -1, device, "src")
        n = src.numel()
        b = _ints(dst, torch.int32, n, device, "dst")
        at = _ints(count, torch.int32, 1, device, "count") if count is not None else 0
        if _current() == device:
            status = self._copy(self._ref, n, a, b, at, _stream(device))
        else:
            status = _elsewhere(self._copy, device, self._ref, n, a, b, at)
        if status:
            _fail(status, self._copier)


class _Plan:
    """A library plan: its handle, and its end."""

    _destroy = None

    def close(self) -> None:
        handle = getattr(self, "_h", None)
        if handle:
            self._h = None
            status = getattr(_library(), self._destroy)(handle)
            if status != 0:
                _fail(status, self._destroy)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _make(self, what, *args):
        handle = ctypes.c_void_p()
        status = getattr(_library(), what)(ctypes.byref(handle), *args)
        if status != 0:
            _fail(status, what)
        self._h = handle.value
        device = args[-1]
        self.device = device if device >= 0 else torch.cuda.current_device()
        self._where = torch.device("cuda", self.device)


class TreeAttention(_Plan):
    """Attention of draft trees over a ``Cache``; owns the workspace of calls with up to ``max_requests`` requests
    and ``max_rows`` query rows.  Use one per concurrent stream: calls of one object must be ordered on the device,
    whichever threads make them."""

    _destroy = "q8kv_attend_destroy"
    _name = "q8kv_attend"
    _cache = Cache

    def __init__(self, heads: int, kv_heads: int, head_dim: int, max_requests: int, max_rows: int, device: int = -1):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self._tail, self._packed = (heads, head_dim), (heads * head_dim, head_dim)
        self._scale = 1.0 / math.sqrt(head_dim) if head_dim > 0 else 0.0
        self._make(self._name + "_plan", heads, kv_heads, head_dim, max_requests, max_rows, int(device))
        self._fn = getattr(_library(), self._name)

    def __call__(self, q, cache: Cache, table, lengths, *, starts=None, mask=None, scale=None, out=None, lse=False):
        """out [rows, heads, head_dim] (the type of q); with ``lse`` also the log of each row's sum [rows, heads] f32.

        q [rows, heads, head_dim] f32, f16 or bf16: all requests' nodes one after another, ``starts`` [requests + 1]
        int32 their first rows (None: as many for each request).  lengths [requests] int32: cached tokens before the
        nodes; node j's own key and value are at position lengths + j.  table [requests, columns] int32: the
        requests' pages (the kernel is chosen by how far the table reaches, as the lengths are not known to the host:
        columns far past the longest request cost time, and may change last bits).  mask [rows, words] int32: bit j % 32 of word j // 32 lets a node see node j of its request
        (None: nodes up to itself).  ``scale`` defaults to 1 / sqrt(head_dim).
        """
        device = self.device
        rows, code, qs = _rows(q, self._tail, device, "q")
        at_len = _ints(lengths, torch.int32, -1, device, "lengths")
        requests = lengths.numel()
        shape = table.shape
        if len(shape) != 2 or shape[0] != requests:
            raise ValueError(f"table must be [{requests}, columns], got {tuple(shape)}")
        cols = shape[1]
        at_table = _ints(table, torch.int32, -1, device, "table")
        at_starts = _ints(starts, torch.int32, requests + 1, device, "starts") if starts is not None else 0
        if starts is None and (rows % requests if requests else rows):
            raise ValueError(f"{rows} rows do not divide over {requests} requests: pass starts")
        at_mask = words = 0
        if mask is not None:
            if mask.dim() != 2 or len(mask) != rows:
                raise ValueError(f"mask must be [{rows}, words], got {tuple(mask.shape)}")
            at_mask = _ints(mask, torch.int32, -1, device, "mask")
            words = mask.shape[1]
            if words == 0 or rows == 0:
                # a mask without words lets no node see another: it is not the missing mask
                at_mask, words = at_mask or at_len, 0
        if out is None:
            out = torch.empty((rows, *self._tail), dtype=q.dtype, device=self._where)
            os = self._packed
        else:
            rows_out, code_out, os = _rows(out, self._tail, device, "out")
            if code_out != code or rows_out != rows:
                raise ValueError(f"out must have the type and rows of q, got {out.dtype} {tuple(out.shape)}")
        if cache._prefix != self._cache._prefix:
            raise TypeError(f"cache must be a {self._cache.__name__}, got {type(cache).__name__}")
        if cache.device != device:
            raise ValueError(f"the cache is on cuda:{cache.device}, the plan on cuda:{device}")
        sums = torch.empty((rows, self.heads), dtype=torch.float32, device=self._where) if lse else None
        args = _ATTEND.pack(q.data_ptr(), out.data_ptr(), sums.data_ptr() if lse else 0, code, requests, rows, qs[0], qs[1],
                            os[0], os[1], at_starts, at_len, at_table, cols, cols, words, at_mask, words,
                            self._scale if scale is None else scale)
        if _current() == device:
            status = self._fn(self._h, cache._ref, args, _stream(device))
        else:
            status = _elsewhere(self._fn, device, self._h, cache._ref, args)
        if status:
            _fail(status, self._name)
        return (out, sums) if lse else out

    def check(self) -> int:
        """Synchronise and return (and clear) whether a bounded wait of the plan's kernels ran out (1, else 0)."""
        word = ctypes.c_int32()
        status = getattr(_library(), self._name + "_check")(self._h, ctypes.byref(word))
        if status:
            _fail(status, self._name + "_check")
        return word.value

    def set_wait(self, wait_ns: int = 0) -> None:
        """For tests of the bounded waits: their bound (0: the default)."""
        status = getattr(_library(), self._name + "_set_wait")(self._h, int(wait_ns))
        if status:
            _fail(status, self._name + "_set_wait")


class TreeVerify(_Plan):
    """Verification of drafted tokens for up to ``max_requests`` requests and ``max_rows`` nodes; use one per
    concurrent stream (calls of one object must be ordered on the device, whichever threads make them)."""

    _destroy = "q8kv_verify_destroy"

    def __init__(self, max_requests: int, max_rows: int, vocab: int, device: int = -1):
        self.vocab, self.max_requests = vocab, max_requests
        self._make("q8kv_verify_plan", max_requests, max_rows, vocab, int(device))
        self._fn = _library().q8kv_verify
        self._tail = (vocab,)

    def __call__(self, logits, tokens, parents, uniforms, *, temperature=None, draft_probs=None, starts=None,
                 requests=None):
        """(path [rows], count [requests], next_token [requests]), int32.

        logits [rows, vocab] f32, f16 or bf16: the target's after each node.  tokens, parents [rows] int32: node 0
        of a request is its newest token, the others drafted after their parent (a number within the request, below
        their own).  uniforms [rows] f32 in [0, 1): node 0's draws the next token, the others' test their node.
        temperature [requests] f32 (0: greedy).  draft_probs [rows, vocab] f32: row i is what node i's children were
        drawn from (None: they were not drawn).  starts [requests + 1] int32: requests' first nodes (None: as many
        for each of ``requests``, which is taken from temperature if not given; a plan for one request has one).
        path holds each request's accepted nodes in order from 0, then -1; count how many drafts.
        """
        device = self.device
        rows, code, ls = _rows(logits, self._tail, device, "logits")
        if requests is None:
            if starts is not None:
                requests = starts.numel() - 1
            elif temperature is not None:
                requests = temperature.numel()
            elif self.max_requests == 1:
                requests = 1
            else:
                raise ValueError(f"how many requests the {rows} rows are: pass starts, temperature or requests")
        at_tokens = _ints(tokens, torch.int32, rows, device, "tokens")
        at_parents = _ints(parents, torch.int32, rows, device, "parents")
        at_uniforms = _ints(uniforms, torch.float32, rows, device, "uniforms")
        at_temperature = _ints(temperature, torch.float32, requests, device, "temperature") if temperature is not None else 0
        at_starts = _ints(starts, torch.int32, requests + 1, device, "starts") if starts is not None else 0
        if starts is None and (rows % requests if requests else rows):
            raise ValueError(f"{rows} rows do not divide over {requests} requests: pass starts")
        at_draft, draft_row = 0, 0
        if draft_probs is not None:
            rows_draft, code_draft, ds = _rows(draft_probs, self._tail, device, "draft_probs")
            if code_draft != 0 or rows_draft != rows:
                raise ValueError(f"draft_probs must be float32 with {rows} rows, got {draft_probs.dtype} {tuple(draft_probs.shape)}")
            at_draft, draft_row = draft_probs.data_ptr(), ds[0]
        path, count, token = torch.empty(rows + 2 * requests, dtype=torch.int32, device=self._where).split(
            (rows, requests, requests))
        args = _VERIFY.pack(logits.data_ptr(), at_draft, at_tokens, at_parents, at_uniforms, at_temperature, at_starts,
                            path.data_ptr(), count.data_ptr(), token.data_ptr(), ls[0], draft_row, rows, requests, self.vocab,
                            code, 0)
        if _current() == device:
            status = self._fn(self._h, args, _stream(device))
        else:
            status = _elsewhere(self._fn, device, self._h, args)
        if status:
            _fail(status, "q8kv_verify")
        return path, count, token
