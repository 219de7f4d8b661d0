"""A Q4_0 key/value cache and attention over it: Python binding of ``include/q4kv.h``.

``Cache4`` and ``TreeAttention4`` are used as ``Cache`` and ``TreeAttention``, with half the memory and half the
traffic: 4-bit codes and one f16 scale per 32 of a row.  This module only checks arguments and passes device pointers
and the current stream to ``libq8mv.so``.
"""
from __future__ import annotations

import ctypes

import torch

from .kv import Cache, CacheDesc, TreeAttention, _library, _strides


def blocks4(head_dim: int) -> int:
    """Blocks of 32 that a row of a head has room for: 2, 3, 4, 6 or 8."""
    return next(b for b in (2, 3, 4, 6, 8) if 32 * b >= head_dim)


def _bind(lib: ctypes.CDLL) -> None:
    i32, i64, p, ref = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.POINTER
    for name, args in (
            # q4kv_cache_t has the fields of q8kv_cache_t
            ("q4kv_cache_write", [ref(CacheDesc), i64, p, p, i32, i64, i64, i64, i64, p, p]),
            ("q4kv_cache_read", [ref(CacheDesc), i64, p, p, p, i32, p]),
            ("q4kv_cache_move", [ref(CacheDesc), i64, i64, p, p, p]),
            ("kvpage_copy_q4", [ref(CacheDesc), i64, p, p, p, p]),
            ("q4kv_attend_plan", [ref(p), i32, i32, i32, i32, i64, ctypes.c_int]),
            ("q4kv_attend", [p, ref(CacheDesc), p, p]),
            ("q4kv_attend_check", [p, ref(i32)]),
            ("q4kv_attend_set_wait", [p, ctypes.c_uint64]),
            ("q4kv_attend_destroy", [p])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int


_bind(_library())


class Cache4(Cache):
    """A paged Q4_0 key/value cache: 4-bit codes c, two a byte, and one f16 scale d per 32 of a row, for (c - 8) d.

    Used as ``Cache``: ``write``, ``read``, ``move`` and ``copy_pages`` are the same calls.  ``Cache4.of`` takes existing
    tensors.  A row has 16 bytes for each of ``blocks4(head_dim)`` blocks, in which units of 4 bytes (keys) or 2 (values)
    of all blocks are side by side (``include/q4kv.h`` has the order).
    """

    _prefix = "q4kv_cache"
    _copier, _fused = "kvpage_copy_q4", "kvrope_write_q4"

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, device="cuda", layout: str = "head"):
        if layout not in ("head", "token"):
            raise ValueError(f"layout must be 'head' or 'token', got {layout!r}")
        if head_dim % 16 != 0 or not 16 <= head_dim <= 256:
            raise ValueError(f"head_dim must be a multiple of 16 up to 256, got {head_dim}")
        shape = (pages, heads, page_size) if layout == "head" else (pages, page_size, heads)
        blocks, parts = blocks4(head_dim), []
        for _ in range(2):
            for width, dtype in ((16 * blocks, torch.uint8), (self.scale_columns(head_dim), torch.float16)):
                t = torch.zeros(*shape, width, dtype=dtype, device=device)
                parts.append(t if layout == "head" else t.transpose(1, 2))
        self._take4(*parts, head_dim)

    @staticmethod
    def scale_columns(head_dim: int) -> int:
        """Scales that a row has room for: a row's are 4, 8 or 16 bytes."""
        return {2: 2, 3: 4, 4: 4, 6: 8, 8: 8}[blocks4(head_dim)]

    @classmethod
    def of(cls, k_codes, k_scales, v_codes, v_scales, head_dim: int) -> "Cache4":
        """A cache over existing tensors: codes [pages, heads, page_size, 16 * blocks4(head_dim)] uint8 and scales
        [pages, heads, page_size, scale_columns(head_dim)] f16, each row contiguous, all four with the same strides
        counted in rows (permuted views of other orders are fine)."""
        self = cls.__new__(cls)
        self._take4(k_codes, k_scales, v_codes, v_scales, head_dim)
        return self

    def _take4(self, k_codes, k_scales, v_codes, v_scales, head_dim):
        if head_dim % 16 != 0 or not 16 <= head_dim <= 256:
            raise ValueError(f"head_dim must be a multiple of 16 up to 256, got {head_dim}")
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes must have 4 axes, got {k_codes.dim()}")
        pages, heads, page_size, _ = k_codes.shape
        width, columns = 16 * blocks4(head_dim), self.scale_columns(head_dim)
        strides = _strides((("k_codes", k_codes, torch.uint8, width), ("k_scales", k_scales, torch.float16, columns),
                            ("v_codes", v_codes, torch.uint8, width), ("v_scales", v_scales, torch.float16, columns)),
                           (pages, heads, page_size))
        self._keep(k_codes, k_scales, v_codes, v_scales, head_dim)
        self._desc = CacheDesc(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), pages,
                               page_size, heads, head_dim, 0, *strides)
        self._ref = ctypes.byref(self._desc)


class TreeAttention4(TreeAttention):
    """Attention of draft trees over a ``Cache4``: the calls, arguments and results of ``TreeAttention``."""

    _destroy = "q4kv_attend_destroy"
    _name = "q4kv_attend"
    _cache = Cache4
