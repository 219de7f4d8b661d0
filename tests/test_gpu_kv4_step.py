"""The operators one after another, as a serving program runs them: prompts, samples forked from them, drafts that are
given back, a pool made dense; what attention gives is checked against 64 bits at every step."""
import numpy as np
import pytest

import kv4_ref as ref
import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


class Text:
    """What a request's cache has to hold: codes and scales of its tokens, in order, as a host of the references reads them."""

    def __init__(self, bits, heads, dim):
        self.bits, self.heads, self.dim = bits, heads, dim
        self.k, self.v = [], []

    def add(self, k, v):
        self.k.append(k)
        self.v.append(v)

    def copy(self, n=None):
        other = Text(self.bits, self.heads, self.dim)
        other.k, other.v = list(self.k[:n]), list(self.v[:n])
        return other


class Host:
    """The texts of all requests as one cache with a page a token."""

    def __init__(self, texts):
        self.page_size, self.heads, self.dim = 1, texts[0].heads, texts[0].dim
        self.bits = texts[0].bits
        module = ref if self.bits == 4 else kv_ref
        self.module = module
        ks, vs = [x for t in texts for x in t.k], [x for t in texts for x in t.v]
        self.kc, self.ks = (np.stack(a)[:, :, None] for a in zip(*(module.quantise(x) for x in ks)))
        self.vc, self.vs = (np.stack(a)[:, :, None] for a in zip(*(module.quantise(x) for x in vs)))
        at = np.cumsum([0] + [len(t.k) for t in texts])
        self.table = np.full((len(texts), max(len(t.k) for t in texts)), -1, np.int32)
        for b in range(len(texts)):
            self.table[b, :at[b + 1] - at[b]] = np.arange(at[b], at[b + 1])

    def _values(self, codes, scales):
        return ref.values(codes, scales, self.dim) if self.bits == 4 else kv_ref.values(codes, scales)

    def rows(self, slots):
        return self._values(self.kc[slots, :, 0], self.ks[slots, :, 0]), self._values(self.vc[slots, :, 0], self.vs[slots, :, 0])

    def steps(self, slots):
        return [np.abs(np.repeat(s[slots, :, 0].astype(np.float64), 32, -1)[..., :self.dim]) for s in (self.ks, self.vs)]


@pytest.mark.parametrize("bits,dim,rot,interleaved,dtype", [(4, 128, 128, False, "bfloat16"), (4, 80, 32, True, "float32"),
                                                            (4, 64, 64, False, "float16"), (8, 128, 64, False, "bfloat16")])
def test_a_serving_program(q8mv, bits, dim, rot, interleaved, dtype):
    import torch

    rng = np.random.default_rng(dim)
    heads, group, page, cols, requests = 2, 3, 8, 30, 6
    kind, attention = (q8mv.Cache4, q8mv.TreeAttention4) if bits == 4 else (q8mv.Cache, q8mv.TreeAttention)
    cache = kind(140, page, heads, dim)
    pool = q8mv.Pages(140, page, requests, cols)
    rotary = q8mv.Rotary(dim, rot, interleaved=interleaved, scaling=dict(kind="yarn", factor=4.0, original=64))
    attend = attention(heads * group, heads, dim, requests, requests * 70)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    texts = [Text(bits, heads, dim) for _ in range(requests)]

    def step(tokens, masks=None):
        """`tokens` more of each request, seen as a chain or by masks; all stay in the cache."""
        lengths = [len(t.k) for t in texts]
        width = max(tokens)
        slots, src, dst, ok = pool.extend(ints(lengths), ints(tokens), width)
        cache.copy_pages(src, dst)
        assert ok.all()
        rows = sum(tokens)
        starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
        x = torch.from_numpy(rng.standard_normal((rows, heads * (group + 2), dim)).astype(np.float32)).cuda().to(getattr(torch, dtype))
        q, k, v = x.split([heads * group, heads, heads], 1)
        pos = np.concatenate([n + np.arange(t) for n, t in zip(lengths, tokens)]).astype(np.int64)
        flat = torch.cat([slots[b, :t] for b, t in enumerate(tokens)])
        at = torch.from_numpy(pos).cuda()
        turned = rotary.write(cache, q, k, v, at, flat)
        # the keys as they are quantised: turned, in 32 bits
        k32, v32 = rotary(k.float(), at).cpu().numpy(), v.float().cpu().numpy()
        for b in range(requests):
            for i in range(starts[b], starts[b + 1]):
                texts[b].add(k32[i], v32[i])
        mask = None
        if masks is not None:
            bits_of = np.zeros((rows, 1), np.uint32)
            for b in range(requests):
                for i in range(tokens[b]):
                    bits_of[starts[b] + i, 0] = sum(int(masks[b][i, j]) << j for j in range(tokens[b]))
            mask = torch.from_numpy(bits_of.view(np.int32)).cuda()
        out, lse = attend(turned, cache, pool.table, ints(lengths), starts=torch.from_numpy(starts).cuda(), mask=mask, lse=True)
        host = Host(texts)
        sees = (lambda b, i, j: j <= i) if masks is None else (lambda b, i, j: bool(masks[b][i, j]))
        reference = ref.attend if bits == 4 else kv_ref.attend
        want = reference(host, turned.float().cpu().numpy(), host.table, np.array(lengths), starts, sees, 1 / np.sqrt(dim), dtype)
        for got, w, tol in ((out, want[0], want[2]), (lse, want[1], want[3])):
            got = got.float().cpu().numpy().astype(np.float64)
            empty = np.isneginf(w)
            assert np.array_equal(np.isneginf(got), empty)
            assert (np.abs(np.where(empty, 0, got) - np.where(empty, 0, w)) <= tol).all()

    step([37, 1, 64, 0, 0, 0])                      # prompts
    pool.fork(ints([0, 1, 2, 0, 2, 2]))             # samples
    texts = [texts[p].copy() for p in (0, 1, 2, 0, 2, 2)]
    for _ in range(3):
        step([1] * 6)                               # a token each: pages are copied once
    drafts = [5, 3, 7, 1, 2, 6]
    step(drafts, [np.tril(rng.random((t, t)) < 0.6) | np.eye(t, dtype=bool) for t in drafts])
    kept = [len(t.k) - d + 1 for t, d in zip(texts, drafts)]  # only the first draft of each was right
    pool.free(ints(kept))
    texts = [t.copy(n) for t, n in zip(texts, kept)]
    step([1] * 6)
    pool.fork(ints([5, 5, 0, 3, -1, 2]))            # beams change places, one ends
    texts = [texts[p].copy() for p in (5, 5, 0, 3)] + [Text(bits, heads, dim), texts[2].copy()]
    step([1, 1, 2, 1, 20, 1])                       # and another prompt takes its place
    cache.copy_pages(*pool.compact())
    assert int((pool.refs > 0).sum()) == int((pool.refs[:int((pool.refs > 0).sum())] > 0).sum())
    step([2, 1, 1, 1, 1, 3])
    pool.free(ints([0] * 6))
    assert not pool.refs.any()
