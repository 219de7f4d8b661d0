"""Several samples of each prompt, decoded together over a 4-bit cache whose pages they share.

    python examples/parallel_sampling.py [--prompts 4] [--samples 8] [--tokens 64] [--bits 4]

The prompts run once.  ``Pages.fork`` lets every sample hold its prompt's pages; ``Pages.extend`` gives a sample a
page of its own, and ``copy_pages`` its contents, when it first writes to a shared one.  ``Rotary.write`` rotates
q and k and writes k and v to the cache in one call, ``TreeAttention4`` attends over it.  Nothing in a step waits
for the host, so it is captured as one CUDA graph.  The weights are random.
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


def q8_weights(rng, K, N, size):
    """Random Q8_0 weights [K, N]: the output of a unit row is about ``size``."""
    codes = torch.from_numpy(rng.integers(-127, 128, size=(K, N), dtype=np.int8)).cuda()
    scale = size / (127 / 3 ** 0.5 * K ** 0.5)
    return codes, torch.full((q8mv.num_blocks(K), N), scale, device="cuda")


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Sampler:
    """``samples`` continuations of each prompt."""

    def __init__(self, prompts, samples, tokens, bits=4, page=16, seed=0, layers=2, dim=512, heads=8, kv_heads=2,
                 head_dim=64, hidden=1024, vocab=2048):
        rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.embed = torch.from_numpy(rng.standard_normal((vocab, dim)).astype(np.float32)).cuda()
        self.layers = [dict(qkv=q8_weights(rng, dim, (heads + 2 * kv_heads) * head_dim, 1.0),
                            out=q8_weights(rng, heads * head_dim, dim, 0.3),
                            up=q8_weights(rng, dim, hidden, 1.0), down=q8_weights(rng, hidden, dim, 0.3))
                       for _ in range(layers)]
        self.head = q8_weights(rng, dim, vocab, 4.0)
        self.rotary = q8mv.Rotary(head_dim, scaling=dict(kind="yarn", factor=4.0, original=1024))

        P = len(prompts)
        rows = self.rows = P * samples
        lengths = [len(p) for p in prompts]
        columns = -(-(max(lengths) + tokens + 1) // page)
        # every prompt once, and of each sample what is its own
        pages = sum(-(-n // page) for n in lengths) + rows * (-(-(tokens + 1) // page) + 1)
        kind, attention = (q8mv.Cache4, q8mv.TreeAttention4) if bits == 4 else (q8mv.Cache, q8mv.TreeAttention)
        self.caches = [kind(pages, page, kv_heads, head_dim) for _ in self.layers]
        self.pool = q8mv.Pages(pages, page, rows, columns)
        self.attention = attention(heads, kv_heads, head_dim, rows, max(sum(lengths), rows))

        dev = dict(device="cuda")
        self.lengths = torch.zeros(rows, dtype=torch.int32, **dev)
        self.one = torch.ones(rows, dtype=torch.int32, **dev)
        self.text = torch.zeros(rows, tokens + 2, dtype=torch.int64, **dev)
        self.uniforms = torch.rand(tokens + 2, rows, generator=torch.Generator("cuda").manual_seed(seed), **dev)
        self.steps = torch.zeros(1, dtype=torch.int64, **dev)
        self.prompt(prompts, samples)

    def forward(self, tokens, positions, slots, starts):
        """Logits of rows of tokens; their keys and values go to ``slots``."""
        x = self.embed[tokens]
        cut = [self.heads, self.kv_heads, self.kv_heads]
        for w, cache in zip(self.layers, self.caches):
            q, k, v = q8mv.matvec(norm(x), *w["qkv"]).view(len(x), -1, self.head_dim).split(cut, 1)
            q = self.rotary.write(cache, q, k, v, positions, slots)
            y = self.attention(q, cache, self.pool.table, self.lengths, starts=starts)
            x = q8mv.matvec(y.reshape(len(x), -1), *w["out"], residual=x)
            x = q8mv.matvec(q8mv.matvec(norm(x), *w["up"], act="silu"), *w["down"], residual=x)
        return q8mv.matvec(norm(x), *self.head)

    def draw(self, logits):
        """A token of each sample, by its uniform of this step."""
        sums = torch.softmax(logits, -1).cumsum(-1)
        u = self.uniforms.index_select(0, self.steps)[0]
        token = torch.searchsorted(sums, u.view(-1, 1) * sums[:, -1:], right=True).clamp(max=self.vocab - 1)
        self.text.index_copy_(1, self.steps, token)
        self.steps.add_(1)

    def prompt(self, prompts, samples):
        P, counts = len(prompts), [len(p) for p in prompts]
        first = torch.zeros(self.rows, dtype=torch.int32)
        first[:P] = torch.tensor(counts)
        slots, _, _, ok = self.pool.extend(self.lengths, first.cuda(), max(counts))
        assert ok.all()
        slots = torch.cat([slots[b, :n] for b, n in enumerate(counts)])
        positions = torch.cat([torch.arange(n) for n in counts]).cuda()
        starts = torch.tensor(np.concatenate([[0], np.cumsum(counts), [sum(counts)] * (self.rows - P)]), dtype=torch.int32).cuda()
        logits = self.forward(torch.tensor([t for p in prompts for t in p], device="cuda"), positions, slots, starts)
        # row b * samples + i becomes the i-th sample of prompt b: all rows at once
        parent = torch.arange(self.rows, device="cuda") // samples
        self.pool.fork(parent.int())
        self.lengths.copy_(first.cuda()[parent])
        self.draw(logits[starts[1:P + 1].long() - 1][parent])

    def step(self):
        """One token of every sample."""
        slots, src, dst, _ = self.pool.extend(self.lengths, self.one, 1)
        for cache in self.caches:
            cache.copy_pages(src, dst)
        newest = self.text.index_select(1, self.steps - 1).view(-1)
        logits = self.forward(newest, self.lengths.long(), slots.view(-1), None)
        self.lengths.add_(self.one)
        self.draw(logits)

    def run(self, tokens):
        """[rows, tokens + 1] int64, by a captured step."""
        self.step()  # plans and the caching allocator's blocks, before the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        for _ in range(tokens - 1):
            graph.replay()
        torch.cuda.synchronize()
        return self.text[:, :tokens + 1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--samples", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--bits", type=int, default=4, choices=(4, 8))
    a = ap.parse_args()
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, 2048, size=int(n)).tolist() for n in rng.integers(100, 400, a.prompts)]
    s = Sampler(prompts, a.samples, a.tokens, bits=a.bits)
    t0 = time.perf_counter()
    s.run(a.tokens)
    dt = time.perf_counter() - t0
    held, used = int(s.pool.held.sum()), int((s.pool.refs > 0).sum())
    print(f"{s.rows} samples of {a.prompts} prompts, {a.tokens} tokens each, {a.bits} bits: {s.rows * a.tokens / dt:.0f} tokens/s; "
          f"{used} pages where samples of their own would hold {held}")


if __name__ == "__main__":
    main()
