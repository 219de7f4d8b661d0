"""Plain 64-bit references of the cache operators, and builders of their test inputs."""
from __future__ import annotations

import numpy as np

TYPES = ("float32", "float16", "bfloat16")
EPS = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}  # half an ulp, relative


def quantise(x):
    """(codes int8, scales f32) of the last axis of x f32 per 32 elements, in IEEE f32 as the header defines them."""
    x = np.asarray(x, np.float32)
    dim = x.shape[-1]
    codes = np.zeros(x.shape, np.int8)
    scales = np.zeros(x.shape[:-1] + ((dim + 31) // 32,), np.float32)
    with np.errstate(all="ignore"):
        for b in range(scales.shape[-1]):
            part = x[..., 32 * b:32 * b + 32]
            mag = np.abs(part)
            amax = np.where(np.isnan(mag), np.float32(0), mag).max(-1)
            scales[..., b] = amax / np.float32(127)
            inv = np.where(amax > 0, np.float32(127) * (np.float32(1) / amax), np.float32(0))[..., None]
            y = part * inv
            codes[..., 32 * b:32 * b + 32] = np.clip(np.rint(np.where(np.isnan(y), np.float32(0), y)), -127, 127)
    return codes, scales


def values(codes, scales):
    """codes * scales in 64 bits."""
    d = np.repeat(scales.astype(np.float64), 32, -1)[..., :codes.shape[-1]]
    return codes.astype(np.float64) * d


class Host:
    """A cache on the host, and its copy on the GPU."""

    def __init__(self, rng, pages, page_size, heads, dim, layout="head", spread=0.5):
        self.page_size = page_size
        gain = np.exp(spread * rng.standard_normal(dim)).astype(np.float32)
        shape = (pages, heads, page_size, dim)
        self.kc, self.ks = quantise(rng.standard_normal(shape, np.float32) * gain)
        self.vc, self.vs = quantise(rng.standard_normal(shape, np.float32) * gain)
        self.layout = layout

    def device(self, q8mv):
        import torch

        parts = []
        for a in (self.kc, self.ks, self.vc, self.vs):
            t = torch.from_numpy(np.ascontiguousarray(a if self.layout == "head" else a.transpose(0, 2, 1, 3))).cuda()
            parts.append(t if self.layout == "head" else t.transpose(1, 2))
        return q8mv.Cache.of(*parts)

    def rows(self, slots):
        """Keys and values [n, heads, dim] of slots, in 64 bits."""
        page, place = slots // self.page_size, slots % self.page_size
        return (values(self.kc[page, :, place], self.ks[page, :, place]),
                values(self.vc[page, :, place], self.vs[page, :, place]))


def attend(host, q, table, lengths, starts, sees, scale, dtype):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits.

    ``sees(b, i, j)`` -> whether node i of request b sees its node j.  Tolerances, from the kernel's arithmetic
    (u = 2^-23, the largest error of one truncated or rounded f32 operation):
      * a score: q in two f16 parts (u) or exact, at most 8 sums of a block and 8 of the row, truncated, the row
        factor and the argument of exp2: 20 u of scale * sum |q k|; exp2 itself 4 u, its argument's own rounding
        2 u of |score - max| <= 2 sum |q k| scale.  Together e = 24 u A + 8 u with A the largest scale * sum |q k|.
      * out: the weights' error twice (numerator and sum), the second product's weights in f16 parts (u, or 2^-11
        for bf16 outputs), 16 truncated sums and one rounded sum per 32 keys: (2 e + (32 + n / 32) u + part) *
        sum p |v|, then half an ulp of the output's type.
    """
    u = 2.0 ** -23
    heads = q.shape[1]
    group = heads // host.kc.shape[1]
    out = np.zeros(q.shape)
    tol = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    tol_lse = np.zeros(q.shape[:2])
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
        for i in range(t1 - t0):
            seen = there & np.array([p < prefix or sees(b, i, int(p) - prefix) for p in pos])
            if not seen.any():
                continue
            k, v = keys[seen], vals[seen]
            for a in range(heads):
                x = q[t0 + i, a].astype(np.float64)
                s = scale * (k[:, a // group] @ x)
                most = scale * (np.abs(k[:, a // group]) @ np.abs(x)).max()
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                p = w / total
                out[t0 + i, a] = p @ v[:, a // group]
                lse[t0 + i, a] = m + np.log(total)
                e = (24 * most + 8) * u
                part = 2.0 ** -11 if dtype == "bfloat16" else u
                tol[t0 + i, a] = (2 * e + (32 + n / 32) * u + part) * (p @ np.abs(v[:, a // group]))
                tol_lse[t0 + i, a] = e + 4 * u * (1 + abs(lse[t0 + i, a]))
    tol += EPS[dtype] * (np.abs(out) + tol) + (2.0 ** -25 if dtype == "float16" else 1e-37)
    return out, lse, tol, tol_lse


def walk(e, vocab, tokens, parents, uniforms, draft=None):
    """The verification of one request as the header defines it, in Python's whole numbers.

    e [nodes, vocab] f32: exp(z - max) of each row (0 everywhere for a row with nothing left)."""
    one = 2.0 ** 40
    nodes = len(tokens)
    f32 = np.float32

    def whole(x):
        return [int(v) for v in (np.asarray(x, np.float64) * one).astype(np.int64)]

    cur, path = 0, [0]
    while True:
        w = whole(e[cur])
        total = sum(w)
        rest = list(w)
        left = total
        if draft is not None and total > 0:
            per = f32(float(one) / float(total))
            q, a, norm = draft[cur].astype(f32), f32(0), f32(1)
        accepted = None
        for i in range(cur + 1, nodes):
            if parents[i] != cur or total == 0:
                continue
            x = int(tokens[i])
            if draft is None:
                mine = rest[x] if 0 <= x < vocab else 0
                if float(f32(uniforms[i])) * float(left) < float(mine):
                    accepted = i
                    break
                left -= mine
                if 0 <= x < vocab:
                    rest[x] = 0
            else:
                if not 0 <= x < vocab:
                    continue
                num = max(f32(e[cur][x] * per) - f32(a * q[x]), f32(0))
                if f32(f32(uniforms[i]) * q[x]) * norm < num:
                    accepted = i
                    break
                a = f32(a + norm)
                res = np.maximum((e[cur] * per).astype(f32) - (a * q).astype(f32), f32(0))
                new = whole(res)
                if sum(new) == 0:
                    rest, left = list(w), total
                    break
                rest, left = new, sum(new)
                norm = f32(float(left) / one)
        if accepted is None:
            break
        cur = accepted
        path.append(cur)
    if left == 0:
        return path, -1
    want = max(0, min(int(float(f32(uniforms[0])) * float(left)), left - 1))
    upto = 0
    for i, x in enumerate(rest):
        upto += x
        if upto > want:
            return path, i
    raise AssertionError("the weights' sum")
