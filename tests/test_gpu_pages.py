"""Pages of a cache against the plain bookkeeping of kv4_ref.Pool: whole numbers, all equal."""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


class Pair:
    """A pool on the GPU and its plain counterpart, which have to stay alike."""

    def __init__(self, q8mv, pages, page, requests, columns):
        self.gpu, self.host = q8mv.Pages(pages, page, requests, columns), ref.Pool(pages, page, requests, columns)

    def ints(self, x):
        import torch

        return torch.from_numpy(np.asarray(x, np.int32)).cuda()

    def same(self, *pairs):
        for got, want in (*pairs, *zip((self.gpu.refs, self.gpu.table, self.gpu.held), self.host.state())):
            assert np.array_equal(got.cpu().numpy(), want)

    def extend(self, lengths, tokens, width):
        got = self.gpu.extend(self.ints(lengths), self.ints(tokens), width)
        want = self.host.extend(lengths, tokens, width)
        self.same(*zip(got, want))
        return want

    def fork(self, parents):
        self.gpu.fork(self.ints(parents))
        self.host.fork(parents)
        self.same()

    def free(self, lengths):
        self.gpu.free(self.ints(lengths))
        self.host.free(lengths)
        self.same()

    def compact(self):
        got = self.gpu.compact()
        self.same(*zip(got, self.host.compact()))


@pytest.mark.parametrize("pages,page,requests,columns", [(1, 1, 1, 1), (2, 16, 1, 2), (40, 16, 5, 12), (300, 1, 7, 60),
                                                         (1000, 7, 33, 40), (5000, 16, 70, 90), (70001, 24, 600, 130)])
def test_a_life_of_requests(q8mv, pages, page, requests, columns):
    """Random growth, forks, frees and compactions, with shortages, until every path has been taken."""
    rng = np.random.default_rng(pages)
    pair = Pair(q8mv, pages, page, requests, columns)
    lengths = np.zeros(requests, np.int64)
    for step in range(12 if pages < 10000 else 5):
        tokens = rng.integers(0, max(2, min(columns * page, 3 * page * pages // requests // 4 + 3)), requests)
        tokens[rng.random(requests) < 0.3] = 0
        if step % 4 == 3:
            tokens[rng.integers(requests)] = columns * page + 1  # more than its columns
            tokens[rng.integers(requests)] = -3
        _, _, _, ok = pair.extend(lengths, tokens, int(rng.integers(0, 80)))
        lengths = np.where(ok == 1, lengths + np.maximum(tokens, 0), lengths)
        parents = np.arange(requests)
        some = rng.random(requests) < 0.4
        parents[some] = rng.integers(-1, requests, some.sum())
        pair.fork(parents)
        lengths = np.where(parents >= 0, lengths[np.maximum(parents, 0)], 0)
        # one more token each, next to shared pages
        _, _, _, ok = pair.extend(lengths, np.ones(requests, int), 1)
        lengths = lengths + ok
        if step % 2:
            keep = np.where(rng.random(requests) < 0.5, lengths, (lengths * rng.random(requests)).astype(np.int64))
            keep[rng.random(requests) < 0.2] = -1
            pair.free(keep)
            lengths = np.maximum(np.minimum(lengths, keep), 0)
        if step % 3 == 2:
            pair.compact()
    pair.free(np.zeros(requests, int))
    assert not pair.host.refs.any()
    pair.compact()


def test_a_long_prompt(q8mv):
    pair = Pair(q8mv, 900, 16, 3, 600)
    pair.extend([0, 0, 0], [5000, 33, 8000], 8000)
    pair.extend([5000, 33, 8000], [100, 0, 3], 100)


def test_forks_copy_on_write(q8mv):
    """Beams that swap places, share a partial page and write to it; reserved pages that are shared."""
    pair = Pair(q8mv, 64, 8, 6, 8)
    pair.extend([0] * 6, [13, 8, 0, 0, 0, 0], 13)
    pair.fork([0, 1, 0, 0, 1, -1])
    slots, src, dst, ok = pair.extend([13, 8, 13, 13, 8, 0], [1] * 6, 1)
    assert (src >= 0).tolist() == [True, False, True, True, False, False]
    pair.fork([3, 2, 1, 0, 4, 9])  # all at once
    pair.extend([14, 14, 9, 14, 9, 0], [40, 0, 0, 0, 0, 0], 40)
    pair.free([14, 14, 9, 14, 9, 0])
    pair.extend([14, 14, 9, 14, 9, 0], [5, 0, 0, 0, 0, 0], 5)
    # pages beyond the length are held, shared by a fork, and each writes its own
    pair.fork([0, 0, 2, 3, 4, 5])
    pair.extend([14, 14, 9, 14, 9, 0], [5, 5, 0, 0, 0, 0], 5)


def test_shortage_is_in_order(q8mv):
    pair = Pair(q8mv, 5, 4, 4, 8)
    _, _, _, ok = pair.extend([0] * 4, [8, 20, 4, 0], 4)
    assert ok.tolist() == [1, 0, 0, 1]
    _, _, _, ok = pair.extend([8, 0, 0, 0], [0, 12, 0, 4], 4)
    assert ok.tolist() == [1, 1, 1, 0]


def test_lengths_near_the_end_of_31_bits(q8mv):
    pair = Pair(q8mv, 16, 65536, 2, 8)
    _, _, _, ok = pair.extend([2 ** 31 - 1, 0], [2 ** 31 - 1, 65537], 2)
    assert ok.tolist() == [0, 1]


def test_a_table_with_numbers_that_are_no_pages(q8mv):
    """They are not followed: nothing is counted for them, and a write gets a fresh page."""
    import torch

    pool = q8mv.Pages(8, 4, 2, 4)
    pool.table.copy_(torch.tensor([[99, -5, 3, -1], [2 ** 31 - 1, 1, -1, -1]], dtype=torch.int32))
    pool.held.copy_(torch.tensor([3, 2], dtype=torch.int32))
    pool.refs[3], pool.refs[1] = 1, 1
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, src, dst, ok = pool.extend(ints([6, 4]), ints([1, 1]), 1)
    assert ok.tolist() == [1, 1] and src.tolist() == [-1, -1] and slots[:, 0].tolist() == [2, 4]
    pool.fork(ints([0, 0]))
    assert pool.refs.tolist() == [2, 0, 0, 2, 0, 0, 0, 0]
    pool.free(ints([0, 0]))
    assert not pool.refs.any()


@pytest.mark.parametrize("bits", [4, 8])
def test_contents_follow(q8mv, bits):
    """What each request reads through its table is what was written for it, whatever moved in between."""
    import torch

    rng = np.random.default_rng(bits)
    requests, page, cols = 6, 4, 16
    pool = q8mv.Pages(90, page, requests, cols)
    caches = [(q8mv.Cache4 if bits == 4 else q8mv.Cache)(90, page, 2, 64, layout=layout) for layout in ("head", "token")]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    text = [[] for _ in range(requests)]  # a row is its number, which both formats hold exactly up to a scale
    written = 0

    def copy(*moves):
        for c in caches:
            c.copy_pages(*moves)

    def check():
        for b, want in enumerate(text):
            if not want:
                continue
            at = torch.arange(len(want), device="cuda")
            slots = pool.table[b].long()[at // page] * page + at % page
            for c in caches:
                k, v = c.read(slots)
                assert k[:, 0, 0].tolist() == want and v[:, 1, 63].tolist() == [-x for x in want]

    for step in range(30):
        lengths = [len(t) for t in text]
        tokens = [int(t) for t in rng.integers(0, 6, requests)]
        tokens = [min(t, cols * page - n) for t, n in zip(tokens, lengths)]
        slots, src, dst, ok = pool.extend(ints(lengths), ints(tokens), 5)
        copy(src, dst)
        rows = torch.zeros(requests, 5, 2, 64, device="cuda")
        for b in range(requests):
            if ok[b]:
                for t in range(tokens[b]):
                    written += 1
                    # seven numbers' worth of steps of 2^-k: the largest magnitude is held exactly
                    rows[b, t] = float(written)
                    text[b].append(float(written))
        # a constant block's largest value is its own top: (0 - 8) d = top exactly for f16-sized numbers
        for c in caches:
            c.write(rows.view(-1, 2, 64), -rows.view(-1, 2, 64), slots.view(-1))
        if bits == 8:
            text = [[float(np.float32(127) * np.float32(np.float32(x) / np.float32(127))) for x in t] for t in text]
        check()
        if step % 3 == 1:
            parents = [int(p) for p in rng.integers(0, requests, requests)]
            pool.fork(ints(parents))
            text = [list(text[p]) for p in parents]
            check()
        if step % 4 == 2:
            keep = [int(rng.integers(0, len(t) + 1)) for t in text]
            pool.free(ints(keep))
            text = [t[:n] for t, n in zip(text, keep)]
            check()
        if step % 5 == 3:
            copy(*pool.compact())
            check()


def test_a_captured_step(q8mv):
    """fork, extend and the copies as one graph, replayed on changing state."""
    import torch

    pool, plain = q8mv.Pages(300, 8, 6, 20), ref.Pool(300, 8, 6, 20)
    cache = q8mv.Cache4(300, 8, 2, 64)
    lengths = torch.zeros(6, dtype=torch.int32, device="cuda")
    tokens, parents = torch.ones_like(lengths), torch.arange(6, dtype=torch.int32, device="cuda")
    pool.extend(lengths, tokens, 1)  # warm
    for t in (pool.refs, pool.held):
        t.zero_()
    pool.table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.fork(parents)
        slots, src, dst, ok = pool.extend(lengths, tokens, 4)
        cache.copy_pages(src, dst)
    rng = np.random.default_rng(0)
    host_lengths = np.zeros(6, int)
    for _ in range(12):
        p, t = rng.integers(0, 6, 6), rng.integers(0, 5, 6)
        parents.copy_(torch.from_numpy(p.astype(np.int32)))
        host_lengths = host_lengths[p]
        lengths.copy_(torch.from_numpy(host_lengths.astype(np.int32)))
        tokens.copy_(torch.from_numpy(t.astype(np.int32)))
        graph.replay()
        plain.fork(p)
        want = plain.extend(host_lengths, t, 4)
        for a, b in (*zip((slots, src, dst, ok), want), *zip((pool.refs, pool.table, pool.held), plain.state())):
            assert np.array_equal(a.cpu().numpy(), b)
        host_lengths = host_lengths + t


def test_refusals(q8mv):
    import torch

    pool = q8mv.Pages(8, 4, 2, 4)
    good = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pool.extend(good[:1], good, 1)
    with pytest.raises(TypeError):
        pool.extend(good.long(), good, 1)
    with pytest.raises(ValueError):
        pool.extend(good, good, -1)
    with pytest.raises(ValueError):
        pool.fork(good.cpu())
    with pytest.raises(ValueError):
        pool.free(torch.zeros(4, dtype=torch.int32, device="cuda")[::2])
    for bad in ((0, 4, 2, 4), (8, 0, 2, 4), (8, 4, 0, 4), (8, 4, 2, 0), (2 ** 29, 4, 2, 4), (8, 65537, 2, 4),
                (8, 4, 65535, 2 ** 24)):
        with pytest.raises(q8mv.Q8mvError):
            q8mv.Pages(*bad)
    cache = q8mv.Cache(4, 16, 1, 64)
    with pytest.raises(ValueError):
        cache.copy_pages(good, good[:1])
    with pytest.raises(TypeError):
        cache.copy_pages(good, good.long())
    with pytest.raises(TypeError):
        cache.copy_pages(good, good, torch.zeros(1, device="cuda"))


def test_more_requests_than_a_cluster_keeps(q8mv):
    """Amounts of more than 512 requests a CTA go through the workspace."""
    rng = np.random.default_rng(5)
    n = 5000
    pair = Pair(q8mv, 9000, 4, n, 6)
    lengths = np.zeros(n, int)
    for _ in range(3):
        tokens = rng.integers(0, 9, n)
        _, _, _, ok = pair.extend(lengths, tokens, 8)
        lengths = np.where(ok == 1, lengths + tokens, lengths)
        parents = np.arange(n)
        parents[rng.random(n) < 0.2] = rng.integers(n)
        pair.fork(parents)
        lengths = lengths[parents]
    pair.compact()


def test_a_captured_cluster(q8mv):
    import torch

    pool, plain = q8mv.Pages(40000, 8, 20, 40), ref.Pool(40000, 8, 20, 40)
    lengths = torch.zeros(20, dtype=torch.int32, device="cuda")
    tokens = torch.full_like(lengths, 100)
    pool.refs[:39000] = 1  # held by nobody here
    plain.refs[:39000] = 1
    pool.extend(lengths, torch.zeros_like(lengths), 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pool.extend(lengths, tokens, 70)  # (and slots by a kernel of their own)
        moves = pool.compact()
    host = np.zeros(20, int)
    for _ in range(3):
        graph.replay()
        want = plain.extend(host, [100] * 20, 70)
        want_moves = plain.compact()
        for a, b in (*zip(out, want), *zip(moves, want_moves), *zip((pool.refs, pool.table, pool.held), plain.state())):
            assert np.array_equal(a.cpu().numpy(), b)
        host += 100
        lengths.add_(tokens)
