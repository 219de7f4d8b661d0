"""Decoding with draft trees, end to end: a small decoder with Q8_0 weights and a paged Q8_0 cache.

    python examples/speculative_decode.py [--requests 8] [--tokens 128] [--temperature 0.0]

A step drafts a tree of tokens after each request's newest one, runs the model once over all trees
(``matvec`` for the products, ``Cache.write`` and ``TreeAttention`` for the keys and values), lets
``TreeVerify`` decide what is kept and brings the accepted path's rows together with ``Cache.move``.
Nothing in it waits for the host, so the whole step is captured as one CUDA graph.  The weights are
random (layers with small outputs, so that drafts made without them are often right); greedy tokens
are compared with those of one-token steps.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import q8_matrix_vector_gb300 as q8mv

CHAIN = (-1,)                      # one token at a time
TREE = (-1, 0, 0, 1, 1, 2, 3, 6)   # each node's parent: three drafts deep, two wide, and a fourth


def q8_weights(rng, K, N, size):
    """Random Q8_0 weights [K, N]: the output of a unit row is about ``size``."""
    codes = torch.from_numpy(rng.integers(-127, 128, size=(K, N), dtype=np.int8)).cuda()
    scale = size / (127 / 3 ** 0.5 * K ** 0.5)
    return codes, torch.full((q8mv.num_blocks(K), N), scale, device="cuda")


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Model:
    def __init__(self, seed=0, layers=2, dim=512, heads=8, kv_heads=2, head_dim=64, hidden=1024, vocab=2048):
        rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.embed = torch.from_numpy(rng.standard_normal((vocab, dim)).astype(np.float32)).cuda()
        self.layers = [dict(qkv=q8_weights(rng, dim, (heads + 2 * kv_heads) * head_dim, 1.0),
                            out=q8_weights(rng, heads * head_dim, dim, 0.3),
                            up=q8_weights(rng, dim, hidden, 1.0), down=q8_weights(rng, hidden, dim, 0.3))
                       for _ in range(layers)]
        self.head = q8_weights(rng, dim, vocab, 4.0)
        half = head_dim // 2
        self.turns = 10000.0 ** (-torch.arange(half, device="cuda") / half)

    def rotate(self, x, position):
        """Rotary position of [rows, heads, head_dim]."""
        angle = (position[:, None] * self.turns)[:, None]
        a, b = x.chunk(2, -1)
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    def logits(self, tokens, position, slots, attend, caches):
        """Of rows of tokens whose keys and values go to ``slots``; attend(q, cache) is their attention."""
        x = self.embed[tokens]
        cut = [self.heads, self.kv_heads, self.kv_heads]
        for w, cache in zip(self.layers, caches):
            q, k, v = q8mv.matvec(norm(x), *w["qkv"]).view(len(x), -1, self.head_dim).split(cut, 1)
            cache.write(self.rotate(k, position), v, slots)
            y = attend(self.rotate(q, position), cache)
            x = q8mv.matvec(y.reshape(len(x), -1), *w["out"], residual=x)
            x = q8mv.matvec(q8mv.matvec(norm(x), *w["up"], act="silu"), *w["down"], residual=x)
        return q8mv.matvec(norm(x), *self.head)

    def followers(self, wide):
        """The drafts: for each token the likeliest next ones, by the model without its layers."""
        every = q8mv.matvec(norm(self.embed), *self.head)
        return every.topk(wide, -1).indices.to(torch.int32)


class Decoder:
    """Requests that are decoded together, with the same tree each."""

    def __init__(self, model, prompts, tokens, parents=TREE, temperature=0.0, page=16, seed=1):
        B, T = len(prompts), len(parents)
        self.model, self.T = model, T
        dev = dict(device="cuda")
        lengths = [len(p) for p in prompts]
        self.limit = max(lengths) + tokens + T  # positions a request may use
        cols = -(-(self.limit + T) // page)
        order = torch.randperm(B * cols, generator=torch.Generator().manual_seed(seed))
        self.page, self.table = page, order.view(B, cols).to(torch.int32).cuda()
        self.caches = [q8mv.Cache(B * cols, page, model.kv_heads, model.head_dim) for _ in model.layers]
        self.attention = q8mv.TreeAttention(model.heads, model.kv_heads, model.head_dim, B, max(sum(lengths), B * T))
        self.verify = q8mv.TreeVerify(B, B * T, model.vocab)

        # the tree: a node's depth, which of its parent's followers it is, and whom it sees
        depth, rank, sees = [0], [0], [1]
        for i in range(1, T):
            depth.append(depth[parents[i]] + 1)
            rank.append(sum(parents[j] == parents[i] for j in range(1, i)))
            sees.append(sees[parents[i]] | 1 << i)
        assert T <= 31 and depth == sorted(depth), "nodes in order of depth, at most 31"
        self.parents, self.rank = parents, rank
        self.followers = model.followers(max(rank) + 1)
        self.depth = torch.tensor(depth, **dev)
        self.parent_of = torch.tensor(list(parents) * B, dtype=torch.int32, **dev)
        self.mask = torch.tensor(sees * B, dtype=torch.int32, **dev).view(B * T, 1)
        self.at = torch.arange(T, **dev)

        # the state: cached tokens, the newest one (not cached yet), all tokens, uniforms still to be used
        self.lengths = torch.zeros(B, dtype=torch.int32, **dev)
        self.text = torch.zeros(B, self.limit + T + 2, dtype=torch.int32, **dev)
        self.temperature = torch.full((B,), temperature, **dev)
        self.uniforms = torch.rand(tokens + 1, B * T, generator=torch.Generator("cuda").manual_seed(seed), **dev)
        self.steps = torch.zeros(1, dtype=torch.int64, **dev)
        self.newest = self.prompt(prompts)

    def slots(self, position):
        """Slots of positions [requests, n]; -1 for positions below 0."""
        page = self.table.gather(1, (position.clamp(min=0) // self.page).long()).long()
        return torch.where(position >= 0, page * self.page + position.clamp(min=0) % self.page, -1)

    def prompt(self, prompts):
        """Caches the prompts, of any lengths, in one pass; the first new token of each."""
        starts = np.cumsum([0] + [len(p) for p in prompts])
        request = np.repeat(np.arange(len(prompts)), np.diff(starts))
        position = np.arange(starts[-1]) - starts[request]
        rows = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in
                (np.concatenate(prompts).astype(np.int64), position, request)]
        tokens, position, request = rows
        starts_d = torch.from_numpy(starts.astype(np.int32)).cuda()
        slots = self.table[request, position // self.page].long() * self.page + position % self.page
        logits = self.model.logits(tokens, position, slots.contiguous(), lambda q, cache: self.attention(
            q, cache, self.table, self.lengths, starts=starts_d), self.caches)
        self.text[request, position] = tokens.to(torch.int32)
        self.lengths.copy_(starts_d.diff())
        last = logits[starts_d[1:].long() - 1]
        alone = self.parent_of[:: self.T].contiguous()
        u = torch.rand(len(prompts), generator=torch.Generator("cuda").manual_seed(0), device="cuda")
        newest = self.verify(last, alone, alone, u, temperature=self.temperature)[2]
        self.text.scatter_(1, self.lengths.long()[:, None], newest[:, None])
        return newest

    def step(self):
        """One pass of the model: every request goes on by 1 to its tree's depth + 1 tokens."""
        B, T = len(self.lengths), self.T
        tokens = [self.newest]
        for i in range(1, T):
            tokens.append(self.followers[tokens[self.parents[i]].long(), self.rank[i]])
        tokens = torch.stack(tokens, 1)
        before = self.lengths[:, None]
        logits = self.model.logits(tokens.view(-1).long(), (before + self.depth).view(-1), self.slots(before + self.at).view(-1),
                                   lambda q, cache: self.attention(q, cache, self.table, self.lengths, mask=self.mask),
                                   self.caches)
        uniforms = self.uniforms[self.steps].view(-1)
        path, count, newest = self.verify(logits, tokens.view(-1), self.parent_of, uniforms, temperature=self.temperature)
        path = path.view(B, T)
        kept = path >= 0
        src, dst = self.slots(torch.where(kept, before + path, -1)), self.slots(torch.where(kept, before + self.at, -1))
        for cache in self.caches:
            cache.move(src, dst)
        # the accepted tokens' text, then the next one; what is not kept goes to the last column
        spare = self.text.shape[1] - 1
        self.text.scatter_(1, torch.where(kept, before + self.at, spare).long(), tokens.gather(1, path.clamp(min=0).long()))
        self.lengths.add_(count + 1)
        self.text.scatter_(1, self.lengths.long()[:, None], newest[:, None])
        self.newest.copy_(newest)
        self.steps.add_(1)

    def capture(self):
        """The step as a CUDA graph; its buffers stay with the decoder."""
        state = [self.lengths, self.text, self.newest, self.steps]
        saved = [t.clone() for t in state]
        side = torch.cuda.Stream()  # plans and allocations, before the capture
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        for t, s in zip(state, saved):
            t.copy_(s)
        return self.graph.replay

    def run(self, tokens):
        """Steps until every request has ``tokens`` new ones: (texts, steps, seconds)."""
        first = self.lengths.clone()
        step = self.capture()
        torch.cuda.synchronize()
        t0, steps, least, most = time.perf_counter(), 0, 0, int(first.max())
        # a step adds 1 to T tokens: the next look at the device when the slowest may be done or the fastest at its limit
        while least < tokens and most + self.T <= self.limit:
            for _ in range(min(max(1, (tokens - least) // self.T), (self.limit - most) // self.T)):
                step()
                steps += 1
            least, most = int((self.lengths - first).min()), int(self.lengths.max())
        seconds = time.perf_counter() - t0
        if self.attention.check():
            raise RuntimeError("a wait in the attention kernel ran out")
        ends = self.lengths.tolist()
        return [self.text[b, :n + 1].tolist() for b, n in enumerate(ends)], steps, seconds


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--temperature", type=float, default=0.0)
    args = ap.parse_args()
    rng = np.random.default_rng(3)
    model = Model()
    prompts = [rng.integers(0, model.vocab, size=int(n)) for n in rng.integers(1, 200, size=args.requests)]
    Decoder(model, prompts, 16).run(16)  # warm-up
    texts = {}
    for name, parents in (("one token a step", CHAIN), ("draft trees", TREE)):
        out, steps, seconds = Decoder(model, prompts, args.tokens, parents, args.temperature).run(args.tokens)
        new = sum(len(t) - len(p) for t, p in zip(out, prompts))
        texts[name] = out
        print(f"{name:18s} {steps} steps, {new} tokens: {new / steps / len(prompts):.2f} a request and step, "
              f"{seconds / steps * 1e6:.0f} us a step, {new / seconds:.0f} tokens/s")
    if args.temperature <= 0:
        same = all(x[:n] == y[:n] for x, y in zip(*texts.values()) for n in [min(len(x), len(y))])
        print("same tokens" if same else "different tokens")
        return 0 if same else 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
