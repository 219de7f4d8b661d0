"""Rotary positions: Python binding of ``include/kvrope.h``.

``Rotary`` turns queries and keys by their positions (half or interleaved pairs, the whole head or part of it, for
contexts of any length), and in one call with the write of keys and values to a ``Cache`` or ``Cache4``.  This module
works out the frequencies, checks arguments and passes device pointers and the current stream to ``libq8mv.so``.
"""
from __future__ import annotations

import ctypes
import math
import struct
from fractions import Fraction

import torch

from .kv import Cache, CacheDesc, _current, _elsewhere, _fail, _ints, _library, _Plan, _rows, _stream

_PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


class WriteArgs(ctypes.Structure):
    """kvrope_write_args_t"""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64), ("k_row", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_row", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("out_row", ctypes.c_int64), ("out_head", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("n", ctypes.c_int64), ("heads_q", ctypes.c_int32), ("type", ctypes.c_int32)]


_WRITE = struct.Struct("=4Q8q2Qqii")
assert _WRITE.size == ctypes.sizeof(WriteArgs)


def _bind(lib: ctypes.CDLL) -> None:
    i32, i64, p, ref = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.POINTER
    for name, args in (
            ("kvrope_plan", [ref(p), i32, i32, i32, p, ctypes.c_float, ctypes.c_int]),
            ("kvrope_apply", [p, i64, i32, i32, p, i64, i64, p, p, i64, i64, i32, p]),
            ("kvrope_write_q8", [p, ref(CacheDesc), p, p]),
            ("kvrope_write_q4", [p, ref(CacheDesc), p, p]),
            ("kvrope_destroy", [p])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int


_bind(_library())


def frequencies(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None):
    """(radians a position of each pair, factor of cos and sin) of base^(-2 i / rotary_dim), i < rotary_dim / 2.

    ``scaling`` stretches them for contexts ``factor`` times those of the training:
      * dict(kind="linear", factor): all divided by factor;
      * dict(kind="ntk", factor): base times factor^(d / (d - 2)), so that the slowest pair is divided by factor and the
        fastest stays;
      * dict(kind="yarn", factor, original, fast=32, slow=1, attention=None): pairs that turn more than ``fast`` times in
        ``original`` positions stay, those that turn less than ``slow`` times are divided by factor, linear in the pair's
        number between; cos and sin times ``attention``, 0.1 ln(factor) + 1 if not given (1 for factors up to 1);
      * dict(kind="bands", factor, original, low=1, high=4): pairs that turn more than ``high`` times in ``original``
        positions stay, those below ``low`` are divided by factor, linear in the number of turns between.
    """
    if scaling is None:
        scaling = dict(kind=None)
    scaling = dict(scaling)
    kind = scaling.pop("kind", None)
    known = {None: (), "linear": ("factor",), "ntk": ("factor",),
             "yarn": ("factor", "original", "fast", "slow", "attention"),
             "bands": ("factor", "original", "low", "high")}
    if kind not in known:
        raise ValueError(f"scaling's kind must be one of {sorted(k for k in known if k)}, got {kind!r}")
    if set(scaling) - set(known[kind]):
        raise ValueError(f"scaling of kind {kind!r} takes {known[kind]}, got {sorted(scaling)}")
    missing = [n for n in known[kind][:2] if n not in scaling]
    if missing:
        raise ValueError(f"scaling of kind {kind!r} needs {missing}")
    if not base > 0:
        raise ValueError(f"base must be positive, got {base}")
    factor = float(scaling.get("factor", 1.0))
    if not (math.isfinite(factor) and factor > 0):
        raise ValueError(f"scaling's factor must be positive, got {factor}")
    d = rotary_dim
    if kind == "ntk" and d > 2:
        base = base * factor ** (d / (d - 2))
    freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if kind == "linear":
        return [f / factor for f in freq], 1.0
    if kind == "yarn":
        original = scaling["original"]
        fast, slow = scaling.get("fast", 32.0), scaling.get("slow", 1.0)
        # the pair that turns so many times in the original context
        low, high = (d * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (fast, slow))
        low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(d // 2)]
        attention = scaling.get("attention")
        if attention is None:
            attention = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        return [f * (1 - r) + f / factor * r for f, r in zip(freq, ramp)], attention
    if kind == "bands":
        low, high = scaling.get("low", 1.0), scaling.get("high", 4.0)
        if not high > low:
            raise ValueError(f"scaling's high must be above its low, got {high} and {low}")
        keep = [min(max((scaling["original"] * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in freq]
        return [f * k + f / factor * (1 - k) for f, k in zip(freq, keep)], 1.0
    return freq, 1.0


class Rotary(_Plan):
    """Rotary positions of the first ``rotary_dim`` (None: all) elements of heads of ``head_dim``: pairs (2 i, 2 i + 1)
    if ``interleaved``, else (i, i + rotary_dim / 2).  ``scaling`` as ``frequencies``, or give ``turning`` (radians a
    position of each pair) and ``factor`` (of cos and sin) yourself.  Frequencies are rounded to 2^-64 of a turn; their
    multiples are exact at any position.  One object may be called by several threads and on several streams at once."""

    _destroy = "kvrope_destroy"

    def __init__(self, head_dim: int, rotary_dim: int | None = None, *, base: float = 10000.0, interleaved: bool = False,
                 scaling: dict | None = None, turning=None, factor: float | None = None, device: int = -1):
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if rotary_dim % 2 or not 2 <= rotary_dim <= min(head_dim, 512):
            raise ValueError(f"rotary_dim must be even, 2 to {min(head_dim, 512)}, got {rotary_dim}")
        if turning is None:
            turning, own = frequencies(rotary_dim, base, scaling)
        elif scaling is not None:
            raise ValueError("pass scaling or turning, not both")
        else:
            turning, own = [float(f) for f in turning], 1.0
        if len(turning) != rotary_dim // 2 or not all(math.isfinite(f) for f in turning):
            raise ValueError(f"turning must be {rotary_dim // 2} finite numbers")
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, rotary_dim, bool(interleaved)
        self.turning, self.factor = turning, own if factor is None else float(factor)
        units = [round(Fraction(f) / (2 * _PI) * 2 ** 64) % 2 ** 64 for f in turning]
        self._make("kvrope_plan", head_dim, rotary_dim, int(self.interleaved), (ctypes.c_uint64 * len(units))(*units),
                   self.factor, int(device))
        lib = _library()
        self._apply, self._fused = lib.kvrope_apply, {n: getattr(lib, n) for n in ("kvrope_write_q8", "kvrope_write_q4")}

    def _out(self, x, out, name):
        """(out, its strides): x's shape and type."""
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=self._where)
            return out, out.stride()
        rows, _, stride = _rows(out, tuple(x.shape[1:]), self.device, name)
        if out.dtype != x.dtype or rows != x.shape[0]:
            raise ValueError(f"{name} must have the type and shape of what it takes, got {out.dtype} {tuple(out.shape)}")
        if any(s == 0 for s, n in zip(stride, out.shape) if n > 1):
            raise ValueError(f"{name} is expanded: its rows overlap")
        return out, stride

    def __call__(self, x, positions, *, out=None, inverse: bool = False):
        """x [n, heads, head_dim] (f32, f16 or bf16) turned by positions [n] (int64), or with ``inverse`` by the transpose,
        which is the gradient of the forward turn (and its way back, times the square of ``factor`` where that is not 1).  ``out`` may be x itself; memory that overlaps otherwise is refused."""
        device = self.device
        if x.dim() != 3:
            raise ValueError(f"x must be [n, heads, {self.head_dim}], got {tuple(x.shape)}")
        n, code, xs = _rows(x, (x.shape[1], self.head_dim), device, "x")
        at = _ints(positions, torch.int64, n, device, "positions")
        out, os = self._out(x, out, "out")
        args = (self._h, n, x.shape[1], code, x.data_ptr(), xs[0], xs[1], at, out.data_ptr(), os[0], os[1], int(inverse))
        status = self._apply(*args, _stream(device)) if _current() == device else _elsewhere(self._apply, device, *args)
        if status:
            _fail(status, "kvrope_apply")
        return out

    def write(self, cache, q, k, v, positions, slots, *, out=None):
        """One call for a layer's step: q [n, heads, head_dim] turned (into ``out``, which may be q but must not meet it otherwise, nor k or v), k
        [n, kv heads, head_dim] turned and, without a rounding between, quantised with v into ``cache`` (``Cache`` or
        ``Cache4``) at slots [n] (int64, each once; outside the cache, as -1: skipped).  Returns the turned q (None for
        q None)."""
        device = self.device
        if not isinstance(cache, Cache):
            raise TypeError(f"cache must be a Cache or Cache4, got {type(cache).__name__}")
        if cache.device != device:
            raise ValueError(f"the cache is on cuda:{cache.device}, the plan on cuda:{device}")
        n, code, ks = _rows(k, cache._tail, device, "k")
        n_v, code_v, vs = _rows(v, cache._tail, device, "v")
        if code_v != code or n_v != n:
            raise ValueError("k and v must have the same type and number of tokens")
        at = _ints(positions, torch.int64, n, device, "positions")
        at_slots = _ints(slots, torch.int64, n, device, "slots")
        if q is None:
            heads, qs, os, q_at, out_at = 0, (0, 0), (0, 0), 0, 0
        else:
            if q.dim() != 3:
                raise ValueError(f"q must be [{n}, heads, {self.head_dim}], got {tuple(q.shape)}")
            n_q, code_q, qs = _rows(q, (q.shape[1], self.head_dim), device, "q")
            if code_q != code or n_q != n:
                raise ValueError("q must have the type and number of tokens of k")
            out, os = self._out(q, out, "out")
            heads, q_at, out_at = q.shape[1], q.data_ptr(), out.data_ptr()
        # (in bytes of the call's own: another thread may make a call while the library reads them)
        args = _WRITE.pack(q_at, k.data_ptr(), v.data_ptr(), out_at, qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1], at,
                           at_slots, n, heads, code)
        fn = self._fused[cache._fused]
        if _current() == device:
            status = fn(self._h, cache._ref, args, _stream(device))
        else:
            status = _elsewhere(fn, device, self._h, cache._ref, args)
        if status:
            _fail(status, cache._fused)
        return None if q is None else out
