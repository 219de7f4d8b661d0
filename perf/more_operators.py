"""Cases, plain forms and exact values of the 4-bit key/value cache with its attention, of rotary positions and
of the pages of a cache.

A 4-bit cache holds, for each token slot and kv head, codes 0 .. 15 and an f16 scale per 32 of them, for keys and
for values: code c stands for (c - 8) d.  A row of codes has 16 * B bytes, B the least of 2, 3, 4, 6, 8 blocks that
hold the head; byte i of a block has its elements 2 i (low half) and 2 i + 1, and a row keeps units of 4 bytes (keys)
or 2 bytes (values) of all its blocks side by side.
"""
from __future__ import annotations

import math
import random
from fractions import Fraction

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
SIZE = {"float32": 4, "float16": 2, "bfloat16": 2}
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def listed():
    return [
        # one decode step of sixteen sequences: keys and values of one layer go into the cache, latency counts
        dict(name="write_step", op="write", n=16, heads=8, dim=128, page=16, pages=512, dtype="bfloat16", layout="head"),
        # a prompt of 7B-class heads written at once, with slots that padding left out, and read back
        dict(name="write_prompt", op="write", n=8190, heads=32, dim=128, page=64, pages=160, dtype="bfloat16",
             layout="token"),
        # the single-token step of a short 7B-class sequence: 32 heads, each with its own keys
        dict(name="attend_step", op="attend", batch=1, nodes=1, heads=32, group=1, dim=128, page=16, low=511, high=511,
             dtype="float32", tree=False, empty=False, layout="head"),
        # a serving batch, one token each, grouped heads, lengths from short to long
        dict(name="attend_batch", op="attend", batch=64, nodes=1, heads=8, group=8, dim=128, page=16, low=180, high=8100,
             dtype="bfloat16", tree=False, empty=False, layout="head"),
        # two very long sequences, what four bits are for: the cache's length is all the work
        dict(name="attend_long", op="attend", batch=2, nodes=1, heads=8, group=4, dim=128, page=64, low=300001,
             high=524287, dtype="float16", tree=False, empty=False, layout="head"),
        # trees of 31 drafted tokens for sixteen requests
        dict(name="attend_tree", op="attend", batch=16, nodes=31, heads=8, group=4, dim=128, page=32, low=700, high=5000,
             dtype="bfloat16", tree=True, empty=True, layout="head"),
        # a decode step of 32 sequences far into a scaled context: q rotated, k rotated and written with v, 4 bits
        dict(name="rotary_step", op="rotary", n=32, heads=8, group=4, dim=128, rot=128, inter=False, scaling="yarn",
             bits=4, page=16, pages=512, top=131072, dtype="bfloat16"),
        # a prompt, the same in one call, to the 8-bit cache
        dict(name="rotary_prompt", op="rotary", n=8192, heads=8, group=4, dim=128, rot=128, inter=False, scaling="",
             bits=8, page=64, pages=160, top=8192, dtype="bfloat16"),
        # queries alone: neighbouring pairs, part of an odd head, positions beyond a million, and the way back (the gradient)
        dict(name="rotary_part", op="rotate", n=5003, heads=12, dim=80, rot=32, inter=True, scaling="linear", top=1 << 21,
             dtype="float32"),
        # one prompt forked into four samples that each get a token: the last page is copied for each
        dict(name="fork_step", op="fork", prompts=3, samples=4, tokens=1, low=37, high=300, page=16, pages=600, cols=64,
             heads=8, dim=128, bits=4),
        # 16 prompts into 8 samples each, five more tokens a sample, all layers in one cache (its heads are layers * heads)
        dict(name="fork_beams", op="fork", prompts=16, samples=8, tokens=5, low=900, high=4000, page=32, pages=4096,
             cols=256, heads=128, dim=128, bits=4),
        # a pool with holes, after many requests have left, made dense again
        dict(name="compact", op="compact", requests=96, low=200, high=2400, page=16, pages=16384, cols=256, heads=16,
             dim=128, bits=4),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("write", "attend", "attend", "attend", "attend", "rotary", "rotary", "rotate", "fork", "fork", "compact"))
    dim = rng.choice((64, 80, 96, 112, 128, 128, 128, 192, 256))
    heads = rng.choice((1, 2, 4, 8, 8, 10, 32))
    page = rng.choice((1, 8, 16, 16, 24, 32, 64, 100, 256))
    dtype = rng.choice(("float32", "bfloat16", "bfloat16", "float16"))
    layout = rng.choice(("head", "token"))
    if op == "write":
        n = _spread(rng, 1, min(8190, 8190 * 32 * 128 // (heads * dim)))
        return dict(op=op, n=n, heads=heads, dim=dim, page=page, pages=-(-n // page) + rng.randrange(1, 40), dtype=dtype,
                    layout=layout)
    if op in ("rotary", "rotate"):
        rot = rng.choice((dim, dim, dim // 2, 32, 2 * rng.randrange(1, dim // 2 + 1)))
        case = dict(op=op, n=_spread(rng, 1, 8192 * 8 // max(heads, 8)), heads=heads, group=rng.choice((1, 2, 4)), dim=dim,
                    rot=rot, inter=rng.random() < 0.4, scaling=rng.choice(("", "linear", "ntk", "yarn", "bands")),
                    bits=rng.choice((4, 8)), page=page, top=_spread(rng, 4000, 1 << 21), dtype=dtype)
        case["pages"] = -(-case["n"] // page) + rng.randrange(1, 40)
        return case
    if op in ("fork", "compact"):
        page = rng.choice((8, 16, 16, 24, 32, 64))
        case = dict(op=op, low=_spread(rng, 1, 700), high=0, page=page, pages=0, cols=0, heads=rng.choice((2, 8, 31, 64)), dim=dim,
                    bits=rng.choice((4, 4, 8)))
        case["high"] = case["low"] + _spread(rng, 1, 2000)
        if op == "fork":
            case.update(prompts=_spread(rng, 1, 16), samples=rng.randrange(1, 9), tokens=rng.choice((1, 1, 2, 5, 17, 40)))
            rows = case["prompts"] * case["samples"]
            case["cols"] = -(-(case["high"] + case["tokens"]) // page) + rng.randrange(0, 9)
            case["pages"] = case["prompts"] * case["cols"] + rows * (2 + case["tokens"] // page) + rng.randrange(0, 60)
        else:
            case.update(requests=_spread(rng, 1, 64))
            case["cols"] = -(-case["high"] // page) + rng.randrange(0, 9)
            case["pages"] = case["requests"] * case["cols"] * rng.choice((1, 2)) + rng.randrange(0, 60)
        # a pool of a gigabyte at most
        while case["pages"] * case["page"] * case["heads"] * case["dim"] > 2 ** 30 and case["heads"] > 1:
            case["heads"] //= 2
        return case
    while True:
        case = dict(op="attend", batch=_spread(rng, 1, 64), nodes=rng.choice((1, 1, 1, 1, 2, 5, 8, 17, 31, 33)),
                    heads=heads, group=rng.choice((1, 2, 3, 4, 5, 8)), dim=dim, page=page, low=0, high=0,
                    dtype=dtype, tree=rng.random() < 0.6, empty=False, layout=layout)
        case["high"] = _spread(rng, 16, 200000)
        case["low"] = rng.choice((1, max(case["high"] // 8, 1), case["high"]))
        case["empty"] = case["tree"] and rng.random() < 0.3
        w, top = work(case), work(listed()[5])
        if w["flops"] <= top["flops"] and w["bytes"] <= 6 * top["bytes"]:
            return case


def _blocks(dim):
    return next(b for b in (2, 3, 4, 6, 8) if 32 * b >= dim)


def _columns(dim):  # of scales
    return {2: 2, 3: 4, 4: 4, 6: 8, 8: 8}[_blocks(dim)]


def _row_bytes(case):  # a token's keys and values in one head
    dim = case["dim"]
    if case.get("bits", 4) == 8:
        return 2 * (dim + 4 * -(-dim // 32))
    return 2 * (dim // 2 + 2 * -(-dim // 32))


def _lengths(case, count):
    """From the case alone, so that its work is known."""
    r = random.Random("%d %d %d" % (count, case["low"], case["high"]))
    got = [r.randint(case["low"], case["high"]) for _ in range(count)]
    got[0] = case["high"]
    if case.get("empty"):
        got[-1] = 0
    return got


def work(case):
    op, dim = case["op"], case["dim"]
    heads = case["heads"]
    row = heads * _row_bytes(case)
    if op == "attend":
        keys = [p + case["nodes"] for p in _lengths(case, case["batch"])]
        rows = case["batch"] * case["nodes"] * heads * case["group"]
        return {"bytes": sum(keys) * row + 2 * rows * dim * SIZE[case["dtype"]] + sum(-(-k // case["page"]) for k in keys) * 4,
                "flops": 4 * sum(keys) * case["nodes"] * heads * case["group"] * dim}
    if op in ("fork", "compact"):
        moved, size = len(_moved(case)), case["page"]
        entries = case["pages"] + case.get("requests", case.get("prompts", 0) * (1 + case.get("samples", 0))) * case["cols"]
        # each page moved is read and written, then read back and written in 16 bits
        return {"bytes": moved * size * (3 * row + 4 * heads * dim) + 8 * entries, "flops": 2 * moved * size * heads * dim}
    n, size = case["n"], SIZE[case["dtype"]]
    if op == "write":
        # written, and read back in the same type
        return {"bytes": n * (4 * heads * dim * size + 2 * row + 16), "flops": 8 * n * heads * dim}
    if op == "rotary":
        # q in and out, k and v in, rows out; rows in and k and v out as they are read back
        return {"bytes": n * heads * dim * size * (2 * case["group"] + 4) + n * (2 * row + 24),
                "flops": n * heads * (3 * case["rot"] * (case["group"] + 1) + 8 * dim)}
    # there and back
    return {"bytes": n * (4 * heads * dim * size + 16), "flops": 6 * n * heads * case["rot"]}


# ---------------------------------------------------------------- the formats

def _cut(x):  # [..., dim] -> [..., blocks, 32]
    dim, blocks = x.shape[-1], _blocks(x.shape[-1])
    return torch.nn.functional.pad(x, (0, 32 * blocks - dim)).unflatten(-1, (blocks, 32))


def _quantise4(x, unit):
    """Packed codes and scales of the last axis of x (f32)."""
    y = _cut(x)
    high, low = y.amax(-1), y.amin(-1)
    d = (torch.where(-low > high, low, high) * -0.125).half()
    f = d.float()
    inv = torch.where(f != 0, 1.0 / f, torch.zeros_like(f))
    c = (torch.round(y * inv.unsqueeze(-1)) + 8).clamp(0, 15).to(torch.uint8)
    b = c[..., 0::2] | (c[..., 1::2] << 4)
    b = b.unflatten(-1, (16 // unit, unit)).transpose(-3, -2).flatten(-3).contiguous()
    return b, torch.nn.functional.pad(d, (0, _columns(x.shape[-1]) - d.shape[-1]))


def _values4(codes, scales, unit, dim, dtype=torch.float32):
    """[..., dim] of packed codes and scales."""
    blocks = _blocks(dim)
    b = codes.unflatten(-1, (16 // unit, blocks, unit)).transpose(-3, -2).flatten(-2)
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2).to(dtype) - 8
    return (c * scales[..., :blocks].to(dtype).unsqueeze(-1)).flatten(-2)[..., :dim]


def _quantise8(x):
    dim = x.shape[-1]
    blocks = -(-dim // 32)
    y = torch.nn.functional.pad(x, (0, 32 * blocks - dim)).unflatten(-1, (blocks, 32))
    amax = y.abs().amax(-1)
    inv = torch.where(amax > 0, 127.0 * (1.0 / amax), torch.zeros_like(amax))
    codes = torch.round(y * inv.unsqueeze(-1)).to(torch.int8)
    return codes.flatten(-2)[..., :dim].contiguous(), amax / 127.0


def _values8(codes, scales, dtype=torch.float32):
    return codes.to(dtype) * scales.to(dtype).repeat_interleave(32, -1)[..., :codes.shape[-1]]


def _unpack(case, parts, at, which, dtype=torch.float32):
    """Rows of keys (0) or values (1) picked by an index of pages (and places)."""
    codes, scales = parts[2 * which][at], parts[2 * which + 1][at]
    if case.get("bits", 4) == 8:
        return _values8(codes, scales, dtype)
    return _values4(codes, scales, 2 if which else 4, case["dim"], dtype)


def _values(g, shape, dim):
    """Keys or values as layers give them: normal, with some channels much larger than the rest."""
    x = torch.randn(*shape, dim, generator=g, device=DEV)
    return x.mul_(torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV)))


def _cache(g, case, pages, filled=True):
    """k codes, k scales, v codes, v scales as [pages, heads, page, ...]; `filled` from values, else any codes."""
    token = case.get("layout") == "token"
    shape = (pages, case["page"], case["heads"]) if token else (pages, case["heads"], case["page"])
    dim, parts = case["dim"], []
    for unit in (4, 2):
        if filled:
            # some gigabytes of values at a time
            step = max(1, (1 << 28) // max(1, shape[1] * shape[2] * dim))
            some = [_quantise4(_values(g, (min(step, pages - i), *shape[1:]), dim), unit) for i in range(0, pages, step)]
            codes, scales = (torch.cat(p) for p in zip(*some)) if len(some) > 1 else some[0]
        elif case["bits"] == 8:
            codes = torch.randint(-127, 128, (*shape, dim), generator=g, device=DEV, dtype=torch.int8)
            scales = torch.rand(*shape, -(-dim // 32), generator=g, device=DEV) * 0.03 + 0.001
        else:
            codes = torch.randint(0, 256, (*shape, 16 * _blocks(dim)), generator=g, device=DEV, dtype=torch.uint8)
            scales = (torch.rand(*shape, _columns(dim), generator=g, device=DEV) * 0.3 + 0.01).half()
        if token:
            codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
        parts += [codes, scales]
    return parts


def _package():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def _own_cache(case, parts):
    if case.get("bits", 4) == 8:
        return _package().Cache.of(*parts)
    return _package().Cache4.of(*parts, case["dim"])


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    return {"write": _prepare_write, "attend": _prepare_attend, "rotary": _prepare_rotary, "rotate": _prepare_rotary,
            "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, g, s)


def _prepare_write(case, g, s):
    s["parts"] = _cache(g, case, case["pages"])
    s["slots"] = torch.randperm(case["pages"] * case["page"], generator=g, device=DEV)[:case["n"]].contiguous()
    kv = _values(g, (case["n"], 2 * case["heads"]), case["dim"]).to(TYPES[case["dtype"]])
    s["k"], s["v"] = kv[:, :case["heads"]], kv[:, case["heads"]:]  # the two halves of one projection
    if case["n"] > 100:
        s["slots"][::97] = -1  # padding
    if own:
        s["cache"] = _own_cache(case, s["parts"])
    return s


def _prepare_attend(case, g, s):
    batch, nodes, page = case["batch"], case["nodes"], case["page"]
    prefixes = _lengths(case, batch)
    need = [-(-(p + nodes) // page) for p in prefixes]
    pages = sum(need) + 3
    s["parts"] = _cache(g, case, pages)
    order = torch.randperm(pages, generator=g, device=DEV).int().tolist()
    table = np.zeros((batch, max(need)), dtype=np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    s["table"] = torch.from_numpy(table).to(DEV)
    s["lengths"] = torch.tensor(prefixes, dtype=torch.int32, device=DEV)
    heads = case["heads"] * case["group"]
    s["q"] = (torch.randn(batch * nodes, heads, case["dim"], generator=g, device=DEV) * 0.8).to(TYPES[case["dtype"]])
    s["mask"] = None
    if case["tree"]:
        i = torch.arange(nodes, device=DEV)
        back = torch.rand(batch, nodes, generator=g, device=DEV) * torch.clamp(i, max=6)
        parents = (i - 1 - back.floor().long().clamp(min=0)).clamp(min=-1)
        sees = torch.eye(nodes, dtype=torch.bool, device=DEV).expand(batch, nodes, nodes).clone()
        for j in range(1, nodes):
            sees[:, j] |= sees[torch.arange(batch, device=DEV), parents[:, j].clamp(min=0)]
        if case["empty"]:
            sees[-1, -1] = False  # a row that pads the last request, which has no prefix
        s["sees"] = sees
        words = -(-nodes // 32)
        bits = torch.nn.functional.pad(sees, (0, 32 * words - nodes)).view(batch * nodes, words, 32).long()
        packed = (bits << torch.arange(32, device=DEV)).sum(-1)
        s["mask"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int().contiguous()
    if own:
        s["cache"] = _own_cache(case, s["parts"])
        s["plan"] = _package().TreeAttention4(heads, case["heads"], case["dim"], batch, batch * nodes)
    return s


BASE, FACTOR, ORIGINAL = 10000.0, 8.0, 4096


def _frequencies(case):
    """Of each pair, in radians a position, and the factor of cos and sin: the usual ones, or scaled for contexts
    FACTOR times the original."""
    rot, kind = case["rot"], case["scaling"]
    base = BASE * FACTOR ** (rot / (rot - 2)) if kind == "ntk" and rot > 2 else BASE
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    factor = 1.0
    if kind == "linear":
        freq = [f / FACTOR for f in freq]
    elif kind == "yarn":
        # pairs that turn more than 32 times within the original context stay, those below once are interpolated
        at = [rot * math.log(ORIGINAL / (t * 2 * math.pi)) / (2 * math.log(BASE)) for t in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        freq = [f * (1 - r) + f / FACTOR * r for f, r in zip(freq, ramp)]
        factor = 0.1 * math.log(FACTOR) + 1.0
    elif kind == "bands":
        # by the turns within the original context: more than 4 stay, less than 1 are divided
        keep = [min(max((ORIGINAL * f / (2 * math.pi) - 1.0) / 3.0, 0.0), 1.0) for f in freq]
        freq = [f * k + f / FACTOR * (1 - k) for f, k in zip(freq, keep)]
    return freq, factor


def _prepare_rotary(case, g, s):
    n, heads = case["n"], case["heads"]
    dtype = TYPES[case["dtype"]]
    s["positions"] = torch.randint(case["top"], (n,), generator=g, device=DEV)
    freq, factor = _frequencies(case)
    turns = [round(Fraction(f) / (2 * PI) * 2 ** 64) % 2 ** 64 for f in freq]
    s["turns"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=DEV)
    s["factor"] = torch.tensor(factor, dtype=torch.float32, device=DEV)
    scaling = {"": None, "linear": dict(kind="linear", factor=FACTOR), "ntk": dict(kind="ntk", factor=FACTOR),
               "yarn": dict(kind="yarn", factor=FACTOR, original=ORIGINAL),
               "bands": dict(kind="bands", factor=FACTOR, original=ORIGINAL)}[case["scaling"]]
    if own:
        s["rotary"] = _package().Rotary(case["dim"], case["rot"], base=BASE, interleaved=case["inter"], scaling=scaling)
    if case["op"] == "rotate":
        s["q"] = torch.randn(n, heads, case["dim"], generator=g, device=DEV).to(dtype)
        return s
    mine = heads * case["group"]
    qkv = _values(g, (n, mine + 2 * heads), case["dim"]).to(dtype)  # one projection
    s["q"], s["k"], s["v"] = qkv.split([mine, heads, heads], 1)
    s["parts"] = _cache(g, case, case["pages"], filled=False)
    s["slots"] = torch.randperm(case["pages"] * case["page"], generator=g, device=DEV)[:n].contiguous()
    if n > 100:
        s["slots"][::97] = -1
    if own:
        s["cache"] = _own_cache(case, s["parts"])
    return s


def _prompt_pages(case):
    """The lengths of the prompts, and the pages of each: some of the pool in a mixed order."""
    lengths = _lengths(case, case["prompts"])
    need = [-(-p // case["page"]) for p in lengths]
    order = list(range(case["pages"]))
    random.Random("%d %d" % (case["pages"], sum(lengths))).shuffle(order)
    got, at = [], 0
    for c in need:
        got.append(order[at:at + c])
        at += c
    return lengths, got


def _moved(case):
    """Pages that get copied: the destinations, ascending in the order in which they are taken."""
    page = case["page"]
    if case["op"] == "compact":
        live = {p for row in _live(case) for p in row}
        return sorted(set(range(len(live))) - live)
    lengths, got = _prompt_pages(case)
    free = sorted(set(range(case["pages"])) - {p for row in got for p in row})
    taken, at = [], 0
    for p, row in zip(lengths, got):
        for _ in range(case["samples"]):
            first = len(row) - (1 if p % page else 0)
            count = -(-(p + case["tokens"]) // page) - first
            if p % page:
                taken.append(free[at])
            at += count
    return taken


def _prepare_fork(case, g, s):
    prompts, samples, page = case["prompts"], case["samples"], case["page"]
    rows = prompts * (1 + samples)
    lengths, got = _prompt_pages(case)
    table = np.full((rows, case["cols"]), -1, dtype=np.int32)
    held = np.zeros(rows, dtype=np.int32)
    refs = np.zeros(case["pages"], dtype=np.int32)
    for b, row in enumerate(got):
        table[b, :len(row)], held[b] = row, len(row)
        refs[row] = 1
    s["parents"] = torch.tensor(list(range(prompts)) + [b for b in range(prompts) for _ in range(samples)],
                                dtype=torch.int32, device=DEV)
    s["lengths"] = torch.tensor(lengths + [lengths[b] for b in range(prompts) for _ in range(samples)],
                                dtype=torch.int32, device=DEV)
    s["tokens"] = torch.tensor([0] * prompts + [case["tokens"]] * (rows - prompts), dtype=torch.int32, device=DEV)
    s["kept"] = torch.tensor(lengths + [0] * (rows - prompts), dtype=torch.int32, device=DEV)
    return _prepare_pool(case, g, s, refs, table, held)


def _live(case):
    """The pages of each request that is still there; every third shares the first of the one before it."""
    r = random.Random("%d %d %d" % (case["requests"], case["pages"], case["high"]))
    order = list(range(case["pages"]))
    r.shuffle(order)
    lengths = _lengths(case, case["requests"])
    got, at = [], 0
    for p in lengths:
        c = -(-p // case["page"])
        got.append(order[at:at + c])
        at += c
    for b in range(2, len(got), 3):
        share = min(len(got[b]), len(got[b - 1])) // 2
        got[b][:share] = got[b - 1][:share]
    return got


def _prepare_compact(case, g, s):
    got = _live(case)
    table = np.full((len(got), case["cols"]), -1, dtype=np.int32)
    held = np.zeros(len(got), dtype=np.int32)
    refs = np.zeros(case["pages"], dtype=np.int32)
    for b, row in enumerate(got):
        table[b, :len(row)], held[b] = row, len(row)
        refs[row] += 1
    return _prepare_pool(case, g, s, refs, table, held)


def _prepare_pool(case, g, s, refs, table, held):
    s["start"] = [torch.from_numpy(x).to(DEV) for x in (refs, table, held)]
    s["parts"] = _cache(g, case, case["pages"], filled=False)
    dst = np.array(_moved(case), dtype=np.int64)
    # the slots of the pages that get copied, looked at afterwards
    s["look"] = torch.from_numpy((dst[:, None] * case["page"] + np.arange(case["page"])).reshape(-1)).to(DEV)
    if own:
        s["cache"] = _own_cache(case, s["parts"])
        s["pool"] = _package().Pages(case["pages"], case["page"], len(held), case["cols"])
        for mine, start in zip((s["pool"].refs, s["pool"].table, s["pool"].held), s["start"]):
            mine.copy_(start)
    else:
        s["refs"], s["table"], s["held"] = (x.clone() for x in s["start"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    case = s["case"]
    op = case["op"]
    if op == "attend":
        return s["plan"](s["q"], s["cache"], s["table"], s["lengths"], mask=s["mask"], lse=True)
    if op == "write":
        s["cache"].write(s["k"], s["v"], s["slots"])
        return s["cache"].read(s["slots"], dtype=s["k"].dtype)
    if op == "rotary":
        q = s["rotary"].write(s["cache"], s["q"], s["k"], s["v"], s["positions"], s["slots"])
        return q, *s["cache"].read(s["slots"], dtype=s["k"].dtype)
    if op == "rotate":
        y = s["rotary"](s["q"], s["positions"])
        return y, s["rotary"](y, s["positions"], inverse=True)
    pool, cache = s["pool"], s["cache"]
    if op == "fork":
        pool.fork(s["parents"])
        slots, src, dst, ok = pool.extend(s["lengths"], s["tokens"], case["tokens"])
        cache.copy_pages(src, dst)
        k, v = cache.read(s["look"], dtype=torch.bfloat16)
        pool.free(s["kept"])
        return slots, src, dst, ok, pool.refs, pool.table, pool.held, k, v
    for mine, start in zip((pool.refs, pool.table, pool.held), s["start"]):
        mine.copy_(start)
    src, dst, count = pool.compact()
    cache.copy_pages(src, dst, count)
    return src, dst, count, pool.refs, pool.table, pool.held, *cache.read(s["look"], dtype=torch.bfloat16)


def _run_plain(s):
    return {"attend": _attend, "write": _write, "rotary": _rotary, "rotate": _rotate, "fork": _fork,
            "compact": _compact}[s["case"]["op"]](s)


def _store(s, slots, rows):
    """k and v rows (f32) to their slots."""
    page, case = s["case"]["page"], s["case"]
    use = slots >= 0
    at = slots[use]
    for which, x in enumerate(rows):
        x = x[use]
        c, d = _quantise8(x) if case.get("bits", 4) == 8 else _quantise4(x, 2 if which else 4)
        s["parts"][2 * which][at // page, :, at % page] = c
        s["parts"][2 * which + 1][at // page, :, at % page] = d


def _read(s, slots, dtype):
    """Keys and values of the slots, [n, heads, dim]; a slot below zero gives zeros."""
    page, at = s["case"]["page"], slots.clamp(min=0)
    got = []
    for which in range(2):
        x = _unpack(s["case"], s["parts"], (at // page, slice(None), at % page), which)
        got.append(torch.where(slots.view(-1, 1, 1) >= 0, x, torch.zeros_like(x)).to(dtype))
    return tuple(got)


def _write(s):
    _store(s, s["slots"], (s["k"].float(), s["v"].float()))
    return _read(s, s["slots"], s["k"].dtype)


def _angles(s):
    """cos and sin [n, 1, pairs]: the turn of a position is a whole number of 2^-64, whose product wraps as turns do."""
    turn = (s["positions"].view(-1, 1) * s["turns"]).double() * (2 * math.pi / 2.0 ** 64)
    return tuple((f(turn).float() * s["factor"]).unsqueeze(1) for f in (torch.cos, torch.sin))


def _turned(case, x, c, sn):
    """x in 32 bits, rotated."""
    rot = case["rot"]
    y = x.float().clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one] = a * c - b * sn
    y[..., two] = b * c + a * sn
    return y


def _rotate(s):
    c, sn = _angles(s)
    y = _turned(s["case"], s["q"], c, sn).to(s["q"].dtype)
    return y, _turned(s["case"], y, c, -sn).to(s["q"].dtype)


def _rotary(s):
    c, sn = _angles(s)
    q = _turned(s["case"], s["q"], c, sn).to(s["q"].dtype)
    _store(s, s["slots"], (_turned(s["case"], s["k"], c, sn), s["v"].float()))
    return q, *_read(s, s["slots"], s["k"].dtype)


def _attend(s):
    case = s["case"]
    batch, nodes, heads, group, dim = (case[k] for k in ("batch", "nodes", "heads", "group", "dim"))
    table = s["table"].long()

    def whole(which):  # [batch, heads, positions, dim] of every request, in 32 bits
        return _unpack(case, s["parts"], table, which).transpose(1, 2).flatten(2, 3)

    keys = whole(0)
    q = s["q"].float().view(batch, nodes, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, heads, nodes * group, dim)
    scores = torch.matmul(q, keys.transpose(-1, -2)).view(batch, heads, nodes, group, -1) / math.sqrt(dim)
    del keys
    at = torch.arange(scores.shape[-1], device=DEV) - s["lengths"].long().view(-1, 1)  # place among the drafts
    i = torch.arange(nodes, device=DEV)
    sees = s["sees"] if s["mask"] is not None else (i.view(1, -1) <= i.view(-1, 1)).expand(batch, nodes, nodes)
    among = torch.gather(sees, 2, at.clamp(0, nodes - 1).view(batch, 1, -1).expand(batch, nodes, -1))
    seen = (at < 0).unsqueeze(1) | (among & (at < nodes).unsqueeze(1))
    scores.masked_fill_(~seen.view(batch, 1, nodes, 1, -1), float("-inf"))
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights.view(batch, heads, nodes * group, -1), whole(1))
    out = out.view(batch, heads, nodes, group, dim) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).reshape(batch * nodes, heads * group, dim)
    return out.to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(batch * nodes, heads * group)


def _count(refs, pages, by):
    """Adds `by` to the counts of pages (whole numbers: in any order); those below zero are skipped."""
    use = pages >= 0
    refs.index_add_(0, pages.clamp(min=0).long(), use.to(refs.dtype) * by)


def _copy(s, src, dst):
    use = (src >= 0) & (dst >= 0)
    a, b = src[use].long(), dst[use].long()
    for part in s["parts"]:
        part[b] = part[a]


def _free_rows(s, lengths):
    """Requests keep the pages of their first `lengths` tokens."""
    keep = (lengths.long().clamp(min=0) + s["case"]["page"] - 1) // s["case"]["page"]
    col = torch.arange(s["table"].shape[1], device=DEV)
    gone = (col >= keep.view(-1, 1)) & (col < s["held"].view(-1, 1))
    _count(s["refs"], torch.where(gone, s["table"], torch.full_like(s["table"], -1)).view(-1), -1)
    s["table"].masked_fill_(gone, -1)
    s["held"].copy_(torch.minimum(s["held"], keep.int()))


def _fork(s):
    case, page = s["case"], s["case"]["page"]
    refs, table, held = s["refs"], s["table"], s["held"]
    rows, cols = table.shape
    row = torch.arange(rows, device=DEV)
    # each request becomes what its parent was
    parents = s["parents"].long()
    changed = (parents != row).view(-1, 1)
    new = torch.where(parents.view(-1, 1) >= 0, table[parents.clamp(min=0)], torch.full_like(table, -1))
    new_held = torch.where(parents >= 0, held[parents.clamp(min=0)], torch.zeros_like(held))
    none = torch.full_like(table, -1)
    _count(refs, torch.where(changed, new, none).view(-1), 1)
    _count(refs, torch.where(changed, table, none).view(-1), -1)
    table.copy_(torch.where(changed, new, table))
    held.copy_(new_held)
    # pages for more tokens: fresh ones past those held, and in place of shared ones that would be written
    length, tokens = s["lengths"].long(), s["tokens"].long().clamp(min=0)
    first = torch.minimum(length // page, held.long())
    need = torch.where(tokens > 0, (length + tokens + page - 1) // page, torch.zeros_like(length))
    col = torch.arange(cols, device=DEV)
    span = (col >= first.view(-1, 1)) & (col < need.view(-1, 1)) & (need <= cols).view(-1, 1)
    mine = col < held.view(-1, 1)
    shared = mine & (refs[table.clamp(min=0).long()] > 1)
    fresh = span & (~mine | shared)
    amount = fresh.sum(-1)
    ends = amount.cumsum(0)
    empty = refs == 0
    ok = (need <= cols) & ((amount == 0) | (ends <= empty.sum()))
    fresh &= ok.view(-1, 1)
    # the free pages, lowest first
    nth = torch.where(empty, empty.long().cumsum(0) - 1, torch.full_like(refs, len(refs)).long())
    order = torch.zeros(len(refs) + 1, dtype=torch.int32, device=DEV)
    order.scatter_(0, nth, torch.arange(len(refs), dtype=torch.int32, device=DEV))
    at = (ends - amount).view(-1, 1) + fresh.long().cumsum(-1) - 1
    page_of = order[at.clamp(0, len(refs))]
    part = fresh & shared & (col == (length // page).view(-1, 1)) & (length % page != 0).view(-1, 1)
    src = torch.where(part, table, none).amax(-1)
    dst = torch.where(part, page_of, none).amax(-1)
    old = torch.where(fresh & shared, table, none).view(-1)
    table.copy_(torch.where(fresh, page_of, table))
    _count(refs, old, -1)
    _count(refs, torch.where(fresh, page_of, none).view(-1), 1)
    held.copy_(torch.where(ok, torch.maximum(held, need.int()), held))
    t = torch.arange(case["tokens"], device=DEV)
    where = length.view(-1, 1) + t
    there = torch.gather(table, 1, (where // page).clamp(max=cols - 1)).long()
    slots = torch.where((t < tokens.view(-1, 1)) & ok.view(-1, 1), there * page + where % page, torch.full_like(where, -1))
    _copy(s, src, dst)
    k, v = _read(s, s["look"], torch.bfloat16)
    _free_rows(s, s["kept"])
    return slots, src, dst, ok.int(), refs, table, held, k, v


def _compact(s):
    for mine, start in zip((s["refs"], s["table"], s["held"]), s["start"]):
        mine.copy_(start)
    refs, table, held = s["refs"], s["table"], s["held"]
    pages = len(refs)
    number = torch.arange(pages, dtype=torch.int32, device=DEV)
    live = refs > 0
    dense = live.sum()
    hole, far = ~live & (number < dense), live & (number >= dense)
    src, dst = (torch.full((pages + 1,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    for pick, into in ((far, src), (hole, dst)):  # the i-th goes to place i, the rest behind the end
        nth = torch.where(pick, pick.long().cumsum(0) - 1, torch.full_like(number, pages).long())
        into.scatter_(0, nth, number)
    count = far.sum().int().view(1)
    most = pages // 2
    src, dst = src[:most], dst[:most]
    use = torch.arange(most, device=DEV) < count
    # where each page is now
    now = torch.cat((number, number[:1]))
    now.scatter_(0, torch.where(use, src, torch.full_like(src, pages)).long(), dst)
    mine = torch.arange(table.shape[1], device=DEV) < held.view(-1, 1)
    table.copy_(torch.where(mine, now[table.clamp(min=0).long()], table))
    refs.copy_(torch.where(number < dense, refs, torch.zeros_like(refs)).index_add_(
        0, dst.clamp(min=0).long(), torch.where(use, s["start"][0][src.clamp(min=0).long()], torch.zeros_like(src))))
    _copy(s, src, dst)
    return src, dst, count, refs, table, held, *_read(s, s["look"], torch.bfloat16)


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_rows(case, parts, slots):
    """Keys and values of slots in 64 bits, nibble by nibble."""
    page, dim, got = case["page"], case["dim"], []
    e = torch.arange(dim, device=DEV)
    for which in range(2):
        codes, scales = (p[slots // page, :, slots % page] for p in parts[2 * which:2 * which + 2])
        if case.get("bits", 4) == 8:
            c = codes.double()
        else:
            unit, i = (2 if which else 4), e % 32
            byte = codes[..., unit * (i // 2 // unit * _blocks(dim) + e // 32) + i // 2 % unit].long()
            c = ((byte >> (4 * (e % 2))) % 16 - 8).double()
        got.append(c * scales.double()[..., e // 32])
    return got


def _exact_stored(case, x):
    """What a row reads back as after it was written, 64 bits but for the format's own rounding of the scale."""
    y = torch.zeros_like(x)
    for b in range(0, x.shape[-1], 32):
        part = x[..., b:b + 32]
        if case.get("bits", 4) == 8:
            step = part.abs().amax(-1, keepdim=True) / 127
            y[..., b:b + 32] = torch.where(step > 0, torch.round(part / step) * step, part)
        else:
            high, low = part.amax(-1, keepdim=True), part.amin(-1, keepdim=True)
            step = (torch.where(-low > high, low, high) / -8).half().double()
            y[..., b:b + 32] = torch.where(step != 0, torch.round(part / step).clamp(-8, 7) * step, torch.zeros_like(part))
    return y


def _exact_turned(case, x, positions, back=False):
    rot = case["rot"]
    freq, factor = _frequencies(case)
    y = x.double().clone()
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
        angle = positions.double() * f
        c, sn = (factor * torch.cos(angle)).view(-1, 1), (factor * torch.sin(angle)).view(-1, 1)
        if back:
            sn = -sn
        y[..., a] = x[..., a].double() * c - x[..., b].double() * sn
        y[..., b] = x[..., a].double() * sn + x[..., b].double() * c
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fork", "compact"):
        # whole numbers aside, the pages' values: those of the page that each was copied from
        moved = len(s["look"]) // case["page"]
        if op == "fork":
            lengths, got = _prompt_pages(case)
            src = [row[-1] for p, row in zip(lengths, got) for _ in range(case["samples"]) if p % case["page"]]
        else:
            refs = s["start"][0].cpu().numpy()
            live = np.flatnonzero(refs)
            src = live[live >= len(live)]
        assert len(src) == moved
        at = np.asarray(src, dtype=np.int64).reshape(-1, 1) * case["page"] + np.arange(case["page"])
        slots = torch.from_numpy(at.reshape(-1)).to(DEV)
        if len(slots) * case["heads"] * case["dim"] > 1 << 29:
            return None
        k, v = _exact_rows(case, s["parts"], slots)
        return (None,) * (7 if op == "fork" else 6) + (k, v)
    if op == "write":
        got = [_exact_stored(case, x.double()) for x in (s["k"], s["v"])]
        for y in got:
            y[s["slots"] < 0] = 0
        return tuple(got)
    if op == "rotate":
        # the way back starts from what the way there is rounded to
        y = _exact_turned(case, s["q"], s["positions"])
        return y, _exact_turned(case, y.to(s["q"].dtype), s["positions"], back=True)
    if op == "rotary":
        q, k = (_exact_turned(case, s[x], s["positions"]) for x in "qk")
        got = [_exact_stored(case, k), _exact_stored(case, s["v"].double())]
        for y in got:
            y[s["slots"] < 0] = 0
        return (q, *got)
    batch, nodes, group, dim, page = (case[k] for k in ("batch", "nodes", "group", "dim", "page"))
    prefixes = _lengths(case, batch)
    if sum(prefixes) * case["heads"] * dim > 1 << 31 or sum(prefixes) * case["heads"] * case["group"] * nodes > 1 << 28:
        return None
    outs, sums = [], []
    for b, prefix in enumerate(prefixes):
        j = torch.arange(prefix + nodes, device=DEV)
        keys, values = _exact_rows(case, s["parts"], s["table"][b].long()[j // page] * page + j % page)
        q = s["q"][b * nodes:(b + 1) * nodes].double()
        sees = torch.ones(nodes, prefix + nodes, dtype=torch.bool, device=DEV)
        sees[:, prefix:] = s["sees"][b] if s["mask"] is not None else torch.ones(nodes, nodes, device=DEV).tril().bool()
        for h in range(case["heads"]):
            mine = q[:, h * group:(h + 1) * group].reshape(nodes * group, dim)
            score = mine @ keys[:, h].T / math.sqrt(dim)
            score = torch.where(sees.repeat_interleave(group, 0), score, torch.full_like(score, -torch.inf))
            lse = torch.logsumexp(score, -1)
            weight = torch.where(lse.unsqueeze(-1) > -torch.inf, torch.exp(score - lse.unsqueeze(-1)), torch.zeros_like(score))
            outs.append((weight @ values[:, h]).view(nodes, group, dim))
            sums.append(lse.view(nodes, group))
    heads = case["heads"]
    out = torch.stack(outs).view(batch, heads, nodes, group, dim).transpose(1, 2).reshape(batch * nodes, heads * group, dim)
    lse = torch.stack(sums).view(batch, heads, nodes, group).transpose(1, 2).reshape(batch * nodes, heads * group)
    return out, lse
