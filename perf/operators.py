"""Cases, plain forms and exact values of the cache operators: write, read and move of a Q8_0 key/value
cache, attention of a tree of drafted tokens over it, and the verification of drafted tokens.

A cache holds, for each of ``pages * page`` token slots and each kv head, ``dim`` int8 codes and one f32
scale per 32 of them (the last block may be partial), for keys and for values.  ``layout`` "head" keeps a
page's tokens of one head together ([pages, heads, page, dim]), "token" a token's heads.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
SIZE = {"float32": 4, "float16": 2, "bfloat16": 2}
ONE = float(2 ** 40)  # the whole-number weight of a row's most likely token


def listed():
    return [
        # one decode step of eight sequences: keys and values of one layer go in, latency counts
        dict(name="write_step", op="write", n=8, heads=8, dim=128, page=16, pages=512, dtype="float32",
             layout="head"),
        # a prompt of 7B-class heads written at once, with slots that padding left out
        dict(name="write_prompt", op="write", n=8190, heads=32, dim=128, page=64, pages=160, dtype="bfloat16",
             layout="token"),
        # a few rows looked at in full precision
        dict(name="read_rows", op="read", n=67, heads=8, dim=80, page=24, pages=64, dtype="float32", layout="head"),
        # a long shared prefix handed to a program that wants 16-bit keys and values
        dict(name="read_prefix", op="read", n=32768, heads=8, dim=128, page=32, pages=1100, dtype="bfloat16",
             layout="head"),
        # the accepted path of four requests, one layer
        dict(name="move_path", op="move", batch=4, path=5, heads=8, dim=128, page=16, pages=256, layout="head"),
        # 64 requests, all 32 layers of a model with 8 kv heads in one cache (its heads are layers * heads)
        dict(name="move_layers", op="move", batch=64, path=9, heads=256, dim=128, page=16, pages=640,
             layout="head"),
        # the single-token step of a short 7B-class sequence: 32 heads, each with its own keys
        dict(name="attend_step", op="attend", batch=1, nodes=1, heads=32, group=1, dim=128, page=16, low=511,
             high=511, dtype="float32", tree=False, empty=False, layout="head"),
        # a serving batch, one token each, grouped heads, lengths from short to long
        dict(name="attend_batch", op="attend", batch=32, nodes=1, heads=8, group=8, dim=128, page=16, low=180,
             high=8100, dtype="bfloat16", tree=False, empty=False, layout="head"),
        # two very long sequences, few rows: the cache's length is all the work
        dict(name="attend_long", op="attend", batch=2, nodes=1, heads=8, group=8, dim=128, page=64, low=200001,
             high=262143, dtype="float32", tree=False, empty=False, layout="token"),
        # trees of 31 drafted tokens for sixteen requests
        dict(name="attend_tree", op="attend", batch=16, nodes=31, heads=8, group=4, dim=128, page=32, low=700,
             high=5000, dtype="bfloat16", tree=True, empty=True, layout="head"),
        # five drafted tokens in a chain, sampled from a draft model whose probabilities are at hand
        dict(name="verify_chain", op="verify", batch=2, nodes=6, vocab=128256, dtype="float32", drafts=True,
             chain=True, greedy=False),
        # trees of 24 most likely tokens for 32 requests
        dict(name="verify_tree", op="verify", batch=32, nodes=24, vocab=128256, dtype="float32", drafts=False,
             chain=False, greedy=False),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("write", "read", "move", "attend", "attend", "attend", "verify", "verify"))
    dim = rng.choice((64, 80, 96, 112, 128, 128, 192, 256))
    heads = rng.choice((1, 2, 4, 8, 8, 10, 32))
    page = rng.choice((1, 8, 16, 24, 32, 64, 100, 256))
    dtype = rng.choice(("float32", "bfloat16", "float16"))
    layout = rng.choice(("head", "token"))
    if op in ("write", "read"):
        n = _spread(rng, 1, min(8190, 8190 * 32 * 128 // (heads * dim)))
        return dict(op=op, n=n, heads=heads, dim=dim, page=page, pages=-(-n // page) + rng.randrange(1, 40),
                    dtype=dtype, layout=layout)
    if op == "move":
        batch, path = _spread(rng, 1, 64), rng.randrange(1, 17)
        heads = rng.choice((2, 8, 31, 64, 128))
        return dict(op=op, batch=batch, path=path, heads=heads, dim=dim, page=page,
                    pages=-(-2 * batch * path // page) + rng.randrange(1, 40), layout=layout)
    if op == "verify":
        dtype = rng.choice(("float32", "float32", "bfloat16"))
        drafts = rng.random() < 0.4
        return dict(op=op, batch=_spread(rng, 1, 32), nodes=rng.randrange(2, 8 if drafts else 25),
                    vocab=_spread(rng, 1000, 128256), dtype=dtype, drafts=drafts, chain=drafts or rng.random() < 0.3,
                    greedy=rng.random() < 0.2)
    while True:
        case = dict(op="attend", batch=_spread(rng, 1, 32), nodes=rng.choice((1, 1, 1, 2, 5, 8, 17, 31, 33)),
                    heads=heads, group=rng.choice((1, 2, 3, 4, 5, 8)), dim=dim, page=page, low=0, high=0,
                    dtype=dtype, tree=rng.random() < 0.6, empty=False, layout=layout)
        case["high"] = _spread(rng, 16, 100000)
        case["low"] = rng.choice((1, case["high"] // 8, case["high"]))
        case["empty"] = case["tree"] and rng.random() < 0.3
        w, top = work(case), work(listed()[9])
        if w["flops"] <= top["flops"] and w["bytes"] <= 8 * top["bytes"]:
            return case


def _prefixes(case):
    """Tokens before the drafts, per request: from the case alone, so that its work is known."""
    r = random.Random("%d %d %d" % (case["batch"], case["low"], case["high"]))
    got = [r.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    got[0] = case["high"]
    if case["empty"]:
        got[-1] = 0
    return got


def work(case):
    op = case["op"]
    if op == "verify":
        # the root's row and two more of each request are needed on this data
        rows = case["batch"] * min(3, case["nodes"])
        per = SIZE[case["dtype"]] + (4 if case["drafts"] else 0)
        return {"bytes": rows * case["vocab"] * per + case["batch"] * case["nodes"] * 16,
                "flops": 4 * rows * case["vocab"]}
    dim, heads = case["dim"], case["heads"]
    row = 2 * heads * (dim + 4 * -(-dim // 32))  # bytes of a token's keys and values
    if op == "attend":
        keys = [p + case["nodes"] for p in _prefixes(case)]
        rows = case["batch"] * case["nodes"] * heads * case["group"]
        return {"bytes": sum(keys) * row + 2 * rows * dim * SIZE[case["dtype"]] + sum(-(-k // case["page"]) for k in keys) * 4,
                "flops": 4 * sum(keys) * case["nodes"] * heads * case["group"] * dim}
    if op == "move":
        n = case["batch"] * case["path"]
        # the move reads and writes each row, the read back reads it and writes it in 32 bits
        return {"bytes": n * (3 * row + 8 * heads * dim + 24), "flops": 2 * n * heads * dim}
    n, wide = case["n"], 2 * heads * dim * SIZE[case["dtype"]]
    if op == "write":
        # written, and read back in the same type
        return {"bytes": n * (2 * wide + 2 * row + 16), "flops": 8 * n * heads * dim}
    return {"bytes": n * (wide + row + 8), "flops": 2 * n * heads * dim}


# ---------------------------------------------------------------- inputs

def _quantise(x):
    """Codes and scales of the last axis of x (f32), per 32: d = amax / 127, c = round(x * (127 / amax))."""
    dim = x.shape[-1]
    blocks = -(-dim // 32)
    y = torch.nn.functional.pad(x, (0, 32 * blocks - dim)).unflatten(-1, (blocks, 32))
    amax = y.abs().amax(-1)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    codes = torch.round(y * inv.unsqueeze(-1)).to(torch.int8)
    return codes.flatten(-2)[..., :dim].contiguous(), amax / 127.0


def _values(g, shape, dim):
    """Keys or values as layers give them: normal, with some channels much larger than the rest."""
    x = torch.randn(*shape, dim, generator=g, device=DEV)
    gain = torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))
    return x.mul_(gain)


def _cache(g, case, pages):
    shape = (pages, case["heads"], case["page"]) if case["layout"] == "head" else (pages, case["page"], case["heads"])
    parts = []
    for _ in range(2):
        codes, scales = _quantise(_values(g, shape, case["dim"]))
        if case["layout"] == "token":
            codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
        parts += [codes, scales]
    return parts  # k codes, k scales, v codes, v scales, as [pages, heads, page, ...] views


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op == "verify":
        return _prepare_verify(case, g, s)
    if op == "attend":
        return _prepare_attend(case, g, s)
    s["parts"] = _cache(g, case, case["pages"])
    places = case["pages"] * case["page"]
    order = torch.randperm(places, generator=g, device=DEV)
    if op == "move":
        n = case["batch"] * case["path"]
        s["src"] = order[:n].view(case["batch"], case["path"]).contiguous()
        s["dst"] = order[n:2 * n].view(case["batch"], case["path"]).contiguous()
        if case["path"] > 2:  # paths of several lengths: the rest is padding
            s["src"][::3, -1] = -1
            s["dst"][::3, -1] = -1
    else:
        s["slots"] = order[:case["n"]].contiguous()
        if op == "write":
            kv = _values(g, (case["n"], 2 * case["heads"]), case["dim"]).to(TYPES[case["dtype"]])
            s["k"], s["v"] = kv[:, :case["heads"]], kv[:, case["heads"]:]  # the two halves of one projection
            if case["n"] > 100:
                s["slots"][::97] = -1  # padding
    if own:
        s["cache"] = _package().Cache.of(*s["parts"])
    return s


def _parents(g, case):
    """A parent below each node's own index; a chain, or a tree that grows near its newest nodes."""
    nodes = case["nodes"]
    i = torch.arange(nodes, device=DEV)
    if case.get("chain", False) or not case.get("tree", True):
        return (i - 1).expand(case["batch"], nodes).contiguous()
    back = torch.rand(case["batch"], nodes, generator=g, device=DEV) * torch.clamp(i, max=6)
    return torch.where(i > 0, i - 1 - back.floor().long().clamp(min=0), torch.full_like(i, -1)).clamp(min=-1)


def _prepare_attend(case, g, s):
    batch, nodes, page = case["batch"], case["nodes"], case["page"]
    prefixes = _prefixes(case)
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
        parents = _parents(g, case)
        sees = torch.eye(nodes, dtype=torch.bool, device=DEV).expand(batch, nodes, nodes).clone()
        for i in range(1, nodes):
            up = parents[:, i].clamp(min=0)
            sees[:, i] |= sees[torch.arange(batch, device=DEV), up]
        if case["empty"]:
            sees[-1, -1] = False  # a row that pads the last request, which has no prefix
        s["sees"] = sees
        words = -(-nodes // 32)
        bits = torch.nn.functional.pad(sees, (0, 32 * words - nodes)).view(batch * nodes, words, 32).long()
        packed = (bits << torch.arange(32, device=DEV)).sum(-1)
        s["mask"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int().contiguous()
    if own:
        s["cache"] = _package().Cache.of(*s["parts"])
        s["plan"] = _package().TreeAttention(heads, case["heads"], case["dim"], batch, batch * nodes)
    return s


def _prepare_verify(case, g, s):
    batch, nodes, vocab = case["batch"], case["nodes"], case["vocab"]
    logits = torch.randn(batch, nodes, vocab, generator=g, device=DEV) * 2.2
    parents = _parents(g, case)
    rows = torch.arange(batch, device=DEV)
    tokens = torch.zeros(batch, nodes, dtype=torch.long, device=DEV)
    s["drafts"] = None
    if case["drafts"]:
        # the draft model is near the target, and each node's token was drawn from it
        near = logits + 0.7 * torch.randn(batch, nodes, vocab, generator=g, device=DEV)
        drafts = torch.softmax(near, -1)
        for i in range(1, nodes):
            tokens[:, i] = torch.multinomial(drafts[rows, parents[:, i]], 1, generator=g)[:, 0]
        s["drafts"] = drafts.view(batch * nodes, vocab)
    else:
        # drafted tokens are likely ones: about 6 of 10 for a node's first child, less for its others
        level = math.log(vocab) + 2.42
        for i in range(1, nodes):
            tokens[:, i] = torch.randint(vocab, (batch,), generator=g, device=DEV)
            first = (parents[:, :i] == parents[:, i:i + 1]).sum(-1) == 0
            logits[rows, parents[:, i], tokens[:, i]] = level + torch.where(first, 0.6, -0.9)
    s["logits"] = logits.view(batch * nodes, vocab).to(TYPES[case["dtype"]])
    s["tokens"], s["parents"] = tokens.int().view(-1), parents.int().view(-1).contiguous()
    s["uniforms"] = torch.rand(batch * nodes, generator=g, device=DEV)
    s["temperature"] = 0.6 + 0.5 * torch.rand(batch, generator=g, device=DEV)
    if case["greedy"]:
        s["temperature"][::2] = 0.0
    if own:
        s["plan"] = _package().TreeVerify(batch, batch * nodes, vocab)
    return s


# ---------------------------------------------------------------- one pass

def _package():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    op = s["case"]["op"]
    if op == "attend":
        return s["plan"](s["q"], s["cache"], s["table"], s["lengths"], mask=s["mask"], lse=True)
    if op == "verify":
        return s["plan"](s["logits"], s["tokens"], s["parents"], s["uniforms"], temperature=s["temperature"],
                         draft_probs=s["drafts"])
    cache = s["cache"]
    if op == "write":
        cache.write(s["k"], s["v"], s["slots"])
        return cache.read(s["slots"], dtype=s["k"].dtype)
    if op == "move":
        cache.move(s["src"], s["dst"])
        return cache.read(s["dst"].view(-1), dtype=torch.float32)
    return cache.read(s["slots"], dtype=TYPES[s["case"]["dtype"]])


def _run_plain(s):
    op = s["case"]["op"]
    if op == "attend":
        return _attend(s)
    if op == "verify":
        return _verify(s)
    page = s["case"]["page"]
    if op == "write":
        use = s["slots"] >= 0
        slots = s["slots"][use]
        for x, codes, scales in ((s["k"], *s["parts"][:2]), (s["v"], *s["parts"][2:])):
            c, d = _quantise(x[use].float())
            codes[slots // page, :, slots % page] = c
            scales[slots // page, :, slots % page] = d
        return _read(s, s["slots"], s["k"].dtype)
    if op == "move":
        src, dst = s["src"].view(-1), s["dst"].view(-1)
        src, dst = src[src >= 0], dst[dst >= 0]
        for part in s["parts"]:
            part[dst // page, :, dst % page] = part[src // page, :, src % page]
        return _read(s, s["dst"].view(-1), torch.float32)
    return _read(s, s["slots"], TYPES[s["case"]["dtype"]])


def _read(s, slots, dtype):
    """Keys and values of the slots, [n, heads, dim]; a slot below zero gives zeros."""
    page, at = s["case"]["page"], slots.clamp(min=0)
    got = []
    for codes, scales in (s["parts"][:2], s["parts"][2:]):
        c, d = codes[at // page, :, at % page].float(), scales[at // page, :, at % page]
        x = c * d.repeat_interleave(32, -1)[..., :c.shape[-1]]
        got.append(torch.where(slots.view(-1, 1, 1) >= 0, x, torch.zeros_like(x)).to(dtype))
    return tuple(got)


def _attend(s):
    case = s["case"]
    batch, nodes, heads, group, dim = (case[k] for k in ("batch", "nodes", "heads", "group", "dim"))
    table = s["table"].long()

    def whole(codes, scales):  # [batch, heads, positions, dim] of every request, in 32 bits
        x = codes[table].float()
        x *= scales[table].repeat_interleave(32, -1)[..., :dim]
        return x.transpose(1, 2).flatten(2, 3)

    keys = whole(*s["parts"][:2])
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
    out = torch.matmul(weights.view(batch, heads, nodes * group, -1), whole(*s["parts"][2:]))
    out = out.view(batch, heads, nodes, group, dim) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).reshape(batch * nodes, heads * group, dim)
    return out.to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(batch * nodes, heads * group)


def _verify(s):
    case = s["case"]
    batch, nodes, vocab = case["batch"], case["nodes"], case["vocab"]
    t = s["temperature"]
    inv = torch.where(t > 0, 1.0 / t, torch.ones_like(t)).view(-1, 1, 1)
    z = s["logits"].float().view(batch, nodes, vocab) * inv
    z = torch.where(torch.isnan(z), torch.full_like(z, float("-inf")), z)
    top = z.amax(-1, keepdim=True)
    e = torch.where(z == top, torch.ones_like(z), torch.exp(z - top))
    best = torch.zeros_like(e).scatter_(2, torch.argmax((z == top).to(torch.int8), -1, keepdim=True), 1.0)
    e = torch.where((t > 0).view(-1, 1, 1), e, best)
    e = torch.where(top > float("-inf"), e, torch.zeros_like(e))  # a row with nothing left has no weight
    del z, best
    w = (e * ONE).long()  # whole numbers: their sums do not depend on an order
    total = w.sum(-1)
    rows = torch.arange(batch, device=DEV)
    tokens, parents = s["tokens"].view(batch, nodes).long(), s["parents"].view(batch, nodes).long()
    u = s["uniforms"].view(batch, nodes)
    at = torch.zeros(batch, dtype=torch.long, device=DEV)
    path = torch.full((batch, nodes), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    count = torch.zeros(batch, dtype=torch.int32, device=DEV)
    drafts = s["drafts"].view(batch, nodes, vocab) if s["drafts"] is not None else None
    if drafts is None:
        mass = total[:, 0].clone()
    else:
        less, norm = torch.zeros(batch, device=DEV), torch.ones(batch, device=DEV)
        per = (ONE / total.double()).float()
        open_ = torch.ones(batch, dtype=torch.bool, device=DEV)
        rest = w[:, 0].clone()
    for i in range(1, nodes):
        tested = parents[:, i] == at
        token = tokens[:, i]
        if drafts is None:
            mine = w[rows, at, token]
            taken = tested & (u[:, i].double() * mass.double() < mine.double())
            refused = tested & ~taken
            w[rows, at, token] = torch.where(refused, torch.zeros_like(mine), mine)
            mass = torch.where(refused, mass - mine, mass)
        else:
            q = drafts[rows, at, token]
            p = e[rows, at, token] * per[rows, at]
            left = (p - less * q).clamp(min=0)
            taken = tested & open_ & (u[:, i] * q * norm < left)
            refused = tested & open_ & ~taken
            more = less + norm
            some = e[rows, at] * per[rows, at].view(-1, 1)
            some = ((some - more.view(-1, 1) * drafts[rows, at]).clamp(min=0) * ONE).long()
            weight = some.sum(-1)
            empty = refused & (weight == 0)
            go = refused & ~empty
            less = torch.where(go, more, less)
            norm = torch.where(go, (weight.double() / ONE).float(), norm)
            rest = torch.where(go.view(-1, 1), some, torch.where(empty.view(-1, 1), w[rows, at], rest))
            open_ = open_ & ~empty
        at = torch.where(taken, torch.full_like(at, i), at)
        count += taken.int()
        path[rows, count.long()] = torch.where(taken, torch.full_like(count, i), path[rows, count.long()])
        if drafts is None:
            mass = torch.where(taken, total[:, i], mass)
        else:
            less = torch.where(taken, torch.zeros_like(less), less)
            norm = torch.where(taken, torch.ones_like(norm), norm)
            open_ = open_ | taken
            rest = torch.where(taken.view(-1, 1), w[:, i], rest)
    rest = w[rows, at] if drafts is None else rest
    sums = rest.cumsum(-1)
    all_ = sums[:, -1]
    want = torch.minimum((u[:, 0].double() * all_.double()).long(), all_ - 1)
    token = torch.searchsorted(sums, want.unsqueeze(1), right=True).squeeze(1)
    token = torch.where(all_ > 0, token, torch.full_like(token, -1)).int()
    return path.view(-1), count, token


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    page, dim = case["page"], case["dim"]
    block = torch.arange(dim, device=DEV) // 32

    def rows(codes, scales, slots):
        c, d = codes[slots // page, :, slots % page].double(), scales[slots // page, :, slots % page].double()
        return c * d[..., block]

    if case["op"] == "write":
        got = []
        for x in (s["k"], s["v"]):
            x = x.double()
            y = torch.zeros_like(x)
            for b in range(-(-dim // 32)):
                part = x[..., 32 * b:32 * b + 32]
                step = part.abs().amax(-1, keepdim=True) / 127
                y[..., 32 * b:32 * b + 32] = torch.where(step > 0, torch.round(part / step) * step, part)
            y[s["slots"] < 0] = 0
            got.append(y)
        return tuple(got)
    if case["op"] in ("read", "move"):
        slots = (s["slots"] if case["op"] == "read" else s["src"].view(-1))
        got = []
        for pair in (s["parts"][:2], s["parts"][2:]):
            y = rows(*pair, slots.clamp(min=0))
            y[slots < 0] = 0
            got.append(y)
        return tuple(got)
    batch, nodes, group = case["batch"], case["nodes"], case["group"]
    outs, sums = [], []
    for b, prefix in enumerate(_prefixes(case)):
        j = torch.arange(prefix + nodes, device=DEV)
        slots = s["table"][b].long()[j // page] * page + j % page
        keys, values = rows(*s["parts"][:2], slots), rows(*s["parts"][2:], slots)
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
