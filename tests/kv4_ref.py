"""Plain references of the Q4_0 cache, rotary positions and pages, and builders of their test inputs."""
from __future__ import annotations

import numpy as np

from kv_ref import EPS


def blocks4(dim):
    return next(b for b in (2, 3, 4, 6, 8) if 32 * b >= dim)


def columns4(dim):
    return {2: 2, 3: 4, 4: 4, 6: 8, 8: 8}[blocks4(dim)]


def quantise(x):
    """(codes uint8 [..., 32 * blocks], scales f16 [..., blocks]) of the last axis of x f32, as the header defines them."""
    x = np.asarray(x, np.float32)
    nb = blocks4(x.shape[-1])
    y = np.zeros(x.shape[:-1] + (32 * nb,), np.float32)
    y[..., :x.shape[-1]] = x
    y = y.reshape(x.shape[:-1] + (nb, 32))
    with np.errstate(all="ignore"):
        number = np.where(np.isnan(y), np.float32(0), y)
        high, low = number.max(-1), (-number).max(-1)
        top = np.where(low > high, -low, high)
        d = (top * np.float32(-0.125)).astype(np.float16)
        f = d.astype(np.float32)
        inv = np.where(f != 0, np.float32(1) / f, np.float32(0))[..., None]
        z = np.rint(number * inv) + np.float32(8)
        off = np.isnan(y) | (inv == 0)
        codes = np.where(off, 8, np.clip(np.where(np.isnan(z), 8, z), 0, 15)).astype(np.uint8)
    return codes.reshape(x.shape[:-1] + (32 * nb,)), d


def pack(codes, unit):
    """The bytes of rows of codes: pairs, then units of all blocks side by side."""
    b = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    nb = b.shape[-1] // 16
    b = b.reshape(b.shape[:-1] + (nb, 16 // unit, unit))
    return np.ascontiguousarray(np.swapaxes(b, -3, -2).reshape(b.shape[:-3] + (16 * nb,)))


def values(codes, scales, dim):
    """(c - 8) d in 64 bits."""
    with np.errstate(all="ignore"):
        return ((codes.astype(np.float64) - 8) * np.repeat(scales.astype(np.float64), 32, -1))[..., :dim]


class Host:
    """A Q4_0 cache on the host, and its copy on the GPU."""

    def __init__(self, rng, pages, page_size, heads, dim, layout="head", spread=0.5):
        self.page_size, self.dim, self.layout, self.heads = page_size, dim, layout, heads
        gain = np.exp(spread * rng.standard_normal(dim)).astype(np.float32)
        shape = (pages, heads, page_size, dim)
        self.kc, self.ks = quantise(rng.standard_normal(shape, np.float32) * gain)
        self.vc, self.vs = quantise(rng.standard_normal(shape, np.float32) * gain)

    def device(self, q8mv):
        import torch

        parts = []
        for codes, scales, unit in ((self.kc, self.ks, 4), (self.vc, self.vs, 2)):
            wide = np.zeros(scales.shape[:-1] + (columns4(self.dim),), np.float16)
            wide[..., :scales.shape[-1]] = scales
            for a in (pack(codes, unit), wide):
                t = torch.from_numpy(np.ascontiguousarray(a if self.layout == "head" else a.transpose(0, 2, 1, 3))).cuda()
                parts.append(t if self.layout == "head" else t.transpose(1, 2))
        return q8mv.Cache4.of(*parts, self.dim)

    def rows(self, slots):
        """Keys and values [n, heads, dim] of slots, in 64 bits."""
        page, place = slots // self.page_size, slots % self.page_size
        return (values(self.kc[page, :, place], self.ks[page, :, place], self.dim),
                values(self.vc[page, :, place], self.vs[page, :, place], self.dim))

    def steps(self, slots):
        """The scales' magnitudes of the elements of keys and values, [n, heads, dim]."""
        page, place = slots // self.page_size, slots % self.page_size
        return [np.abs(np.repeat(s[page, :, place].astype(np.float64), 32, -1)[..., :self.dim]) for s in (self.ks, self.vs)]


def attend(host, q, table, lengths, starts, sees, scale, dtype):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits, as kv_ref.attend.

    Tolerances, from the kernel's arithmetic (u = 2^-23, the largest error of one truncated or rounded f32 operation).
    Sums run over codes of 0 .. 15 with 8 taken off, so what they round is c + 8 <= |c - 8| + 16 steps:
      * a score: q in two f16 parts (u) or exact, at most 8 truncated sums of a block and 8 of the row, its factor and
        the argument of exp2: 20 u of A = scale * sum |q| (|k| + 16 d); exp2 itself 4 u, its argument's own rounding 2 u
        of |score - max| <= 2 A.  Together e = 24 u A + 8 u.
      * out: the weights' error twice (numerator and sum) and their f16 parts (u, or 2^-11 for bf16 outputs) of
        sum p |v|; 16 truncated sums of 32 keys and a rounded one per 32 keys of sum p (|v| + 16 d); then half an ulp
        of the output's type.
    """
    u = 2.0 ** -23
    heads = q.shape[1]
    group = heads // host.heads
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    lse, tol_lse = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    reach = table.shape[1] * host.page_size
    for b in range(len(lengths)):
        t0, t1 = starts[b], starts[b + 1]
        prefix = max(int(lengths[b]), 0)
        n = min(prefix + t1 - t0, reach)
        if t1 == t0 or n == 0:
            continue
        pos = np.arange(n)
        page = table[b, pos // host.page_size]
        there = (page >= 0) & (page < host.kc.shape[0])
        slots = np.where(there, page, 0).astype(np.int64) * host.page_size + pos % host.page_size
        keys, vals = host.rows(slots)
        kd, vd = host.steps(slots)
        for i in range(t1 - t0):
            seen = there & np.array([p < prefix or sees(b, i, int(p) - prefix) for p in pos])
            if not seen.any():
                continue
            for a in range(heads):
                h = a // group
                x = q[t0 + i, a].astype(np.float64)
                k, v = keys[seen, h], vals[seen, h]
                s = scale * (k @ x)
                most = abs(scale) * ((np.abs(k) + 16 * kd[seen, h]) @ np.abs(x)).max()
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                p = w / total
                out[t0 + i, a] = p @ v
                lse[t0 + i, a] = m + np.log(total)
                e = (24 * most + 8) * u
                part = 2.0 ** -11 if dtype == "bfloat16" else u
                size = p @ np.abs(v)
                tol[t0 + i, a] = (2 * e + part) * size + (32 + n / 32) * u * (size + 16 * (p @ vd[seen, h]))
                tol_lse[t0 + i, a] = e + 4 * u * (1 + abs(lse[t0 + i, a]))
    tol += EPS[dtype] * (np.abs(out) + tol) + (2.0 ** -25 if dtype == "float16" else 1e-37)
    return out, lse, tol, tol_lse


def rotate(x, positions, turning, factor, interleaved, back=False):
    """x [n, heads, dim] (any float type) rotated, in 64 bits, with the magnitudes that its rounding scales with."""
    y = np.asarray(x, np.float64).copy()
    size = np.abs(y)
    half = len(turning)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(turning, np.float64)
    c, s = (factor * f(angle)[:, None, :] for f in (np.cos, np.sin))
    if back:
        s = -s
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = y[..., one].copy(), y[..., two].copy()
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    size[..., one], size[..., two] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, size


class Pool:
    """The bookkeeping of pages in plain Python, as the header states it."""

    def __init__(self, pages, page_size, requests, columns):
        self.page_size, self.columns = page_size, columns
        self.refs = np.zeros(pages, np.int32)
        self.table = np.full((requests, columns), -1, np.int32)
        self.held = np.zeros(requests, np.int32)

    def state(self):
        return self.refs.copy(), self.table.copy(), self.held.copy()

    def extend(self, lengths, tokens, width):
        size, n = self.page_size, len(self.held)
        refs = self.refs.copy()
        free = [p for p in range(len(refs)) if refs[p] == 0]
        slots = np.full((n, width), -1, np.int64)
        src, dst, ok = (np.full(n, v, np.int32) for v in (-1, -1, 1))
        used = 0
        for b in range(n):
            length, more = max(int(lengths[b]), 0), max(int(tokens[b]), 0)
            need = -(-(length + more) // size) if more else 0
            if need > self.columns:
                ok[b] = 0
                continue
            first = min(length // size, int(self.held[b]))
            fresh = [c for c in range(first, need) if c >= self.held[b] or refs[self.table[b, c]] > 1]
            if fresh and used + len(fresh) > len(free):
                ok[b] = 0
                used += len(fresh)  # nobody behind gets any
                continue
            for c in fresh:
                page = free[used]
                used += 1
                if c < self.held[b]:
                    old = self.table[b, c]
                    self.refs[old] -= 1
                    if c == length // size and length % size:
                        src[b], dst[b] = old, page
                self.table[b, c] = page
                self.refs[page] = 1
            self.held[b] = max(self.held[b], need)
            for t in range(min(width, more)):
                slots[b, t] = int(self.table[b, (length + t) // size]) * size + (length + t) % size
        return slots, src, dst, ok

    def fork(self, parents):
        table, held = self.table.copy(), self.held.copy()
        for b, p in enumerate(parents):
            if p == b:
                continue
            for c in range(held[b]):
                self.refs[table[b, c]] -= 1
            self.table[b] = -1
            self.held[b] = 0
            if 0 <= p < len(held):
                self.table[b, :held[p]] = table[p, :held[p]]
                self.held[b] = held[p]
                for c in range(held[p]):
                    self.refs[table[p, c]] += 1

    def free(self, lengths):
        for b, length in enumerate(lengths):
            keep = -(-max(int(length), 0) // self.page_size)
            for c in range(keep, self.held[b]):
                self.refs[self.table[b, c]] -= 1
                self.table[b, c] = -1
            self.held[b] = min(self.held[b], keep)

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(len(live)) if self.refs[p] == 0]
        far = [p for p in live if p >= len(live)]
        most = len(self.refs) // 2
        src, dst = np.full(most, -1, np.int32), np.full(most, -1, np.int32)
        src[:len(far)], dst[:len(far)] = far, holes
        for a, b in zip(far, holes):
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return src, dst, np.array([len(far)], np.int32)
