"""Draft-tree attention over the Q8_0 cache against the 64-bit reference (tolerances derived in kv_ref.attend)."""
import numpy as np
import pytest

import kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


class Case:
    """Requests with their own lengths and trees over one cache."""

    def __init__(self, q8mv, seed, lengths, nodes, heads=2, group=2, dim=64, page=16, dtype="float32", layout="head",
                 tree=True, cols=None, words=None):
        import torch

        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.nodes, self.tree = dtype, nodes, tree
        self.lengths = np.array(lengths, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        rows = int(self.starts[-1])
        need = [-(-(max(p, 0) + t) // page) for p, t in zip(lengths, nodes)]
        self.host = ref.Host(rng, sum(need) + 2, page, heads, dim, layout)
        order = rng.permutation(sum(need) + 2)
        self.table = np.full((len(nodes), cols if cols is not None else max(max(need), 1)), -1, np.int32)
        at = 0
        for b, c in enumerate(need):
            c = min(c, self.table.shape[1])
            self.table[b, :c] = order[at:at + c]
            at += c
        self.q = torch.from_numpy(rng.standard_normal((rows, heads * group, dim)).astype(np.float32)).cuda()
        self.q = self.q.to(getattr(torch, dtype))
        self.seen = [rng.random((t, t)) < 0.5 for t in nodes]
        self.words = words if words is not None else -(-max(max(nodes), 1) // 32)
        mask = np.zeros((rows, self.words), np.uint32)
        for b, t in enumerate(nodes):
            for i, j in zip(*np.nonzero(self.seen[b])):
                if j < 32 * self.words:
                    mask[self.starts[b] + i, j // 32] |= np.uint32(1 << (j % 32))
        self.mask = torch.from_numpy(mask.view(np.int32)).cuda() if tree else None
        self.plan = q8mv.TreeAttention(heads * group, heads, dim, len(nodes), max(rows, 1))
        self.q8mv = q8mv

    def sees(self, b, i, j):
        return bool(self.seen[b][i, j]) and j < 32 * self.words if self.tree else j <= i

    def device(self):
        import torch

        self.cache = self.host.device(self.q8mv)
        self.args = [torch.from_numpy(a).cuda() for a in (self.table, self.lengths, self.starts)]

    def run(self, **more):
        if not hasattr(self, "cache"):
            self.device()
        table, lengths, starts = self.args
        return self.plan(self.q, self.cache, table, lengths, starts=starts, mask=self.mask, lse=True, **more)

    def check(self, got=None, scale=None):
        out, lse = got if got is not None else self.run()
        scale = scale if scale is not None else self.host.kc.shape[3] ** -0.5
        want, want_lse, tol, tol_lse = ref.attend(self.host, self.q.float().cpu().numpy(), self.table, self.lengths,
                                                  self.starts, self.sees, scale, self.dtype)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(out).all()
        bad = ~(np.abs(out - want) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], float(np.max(np.abs(out - want) / tol)))
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(lse), none)
        assert np.all(np.abs(lse[~none] - want_lse[~none]) <= tol_lse[~none])
        assert not out[none].any()


def wide(q8mv, seed, lengths, nodes, heads=2, group=2, page=16, **more):
    """A case whose tables reach far enough, in columns without pages, for the tensor-memory path."""
    tiles = heads * len(nodes) * -(-(-(-sum(nodes) // len(nodes)) * group) // 16)  # of 16 rows, for 128 keys of reach
    cols = max(-(-4096 // tiles) * 128 // page + 1, *(-(-(max(n, 0) + t) // page) for n, t in zip(lengths, nodes)), 1)
    return Case(q8mv, seed, lengths, nodes, heads=heads, group=group, page=page, cols=cols, **more)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("layout,page", [("head", 16), ("token", 7)])
def test_types_and_head_sizes(q8mv, dtype, dim, layout, page):
    Case(q8mv, dim, [0, 37, 300], [3, 1, 9], dim=dim, dtype=dtype, layout=layout, page=page).check()


@pytest.mark.parametrize("group", [1, 3, 8, 16, 21])
@pytest.mark.parametrize("nodes", [[1, 1], [5, 0, 12], [33, 2], [70]])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_groups_and_trees(q8mv, group, nodes, dtype):
    Case(q8mv, group, [41 * (b + 1) for b in range(len(nodes))], nodes, heads=3, group=group, dim=32, dtype=dtype).check()


@pytest.mark.parametrize("length", [0, 1, 30, 31, 32, 33, 63, 64, 95, 126, 127, 128, 129, 255, 256, 700])
@pytest.mark.parametrize("tree", [True, False])
def test_lengths_around_the_tiles(q8mv, length, tree):
    for nodes in (1, 4, 37):
        Case(q8mv, length, [length], [nodes], heads=1, group=3, dim=48, page=5, tree=tree).check()


@pytest.mark.parametrize("page", [1, 3, 32, 100, 1024])
def test_pages_that_end_inside_a_tile(q8mv, page):
    Case(q8mv, page, [257, 90], [6, 6], dim=64, page=page, dtype="bfloat16").check()


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("dim", [48, 64, 112, 128, 256])
@pytest.mark.parametrize("heads,group,nodes", [(4, 2, [1, 3, 0, 2]), (8, 1, [5, 1, 1, 8]), (4, 8, [1, 1, 1, 1])])
def test_heads_side_by_side(q8mv, dtype, dim, heads, group, nodes):
    """A token's heads next to each other, eight query rows at most."""
    Case(q8mv, dim, [0, 35, 64, 500], nodes, heads=heads, group=group, dim=dim, dtype=dtype, layout="token", page=9).check()


def test_heads_side_by_side_in_a_long_table(q8mv):
    """Tables that reach far, of which little is used: the shape for long sequences at short lengths."""
    for dim, dtype, heads, group, nodes in ((64, "float32", 4, 2, [1, 3, 0, 2]), (128, "bfloat16", 8, 1, [5, 1, 1, 8]),
                                            (80, "float16", 4, 8, [1, 1, 1, 1]), (256, "float32", 4, 1, [2, 2, 8, 1]),
                                            (128, "float32", 12, 1, [1, 4, 6, 2])):
        c = Case(q8mv, dim, [0, 35, 64, 3000], nodes, heads=heads, group=group, dim=dim, dtype=dtype, layout="token", page=9,
                 cols=80000)
        c.check()


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("dim", [80, 96, 160, 192, 224])
def test_heads_that_end_before_their_layout(q8mv, dtype, dim):
    """Heads of fewer blocks than the layout that they share: by heads side by side, 8 rows and 16."""
    Case(q8mv, dim, [0, 35, 64, 900], [1, 3, 0, 2], heads=4, group=2, dim=dim, dtype=dtype, layout="token", page=9, cols=80000).check()
    Case(q8mv, dim, [7, 3000], [2, 1], heads=3, group=2, dim=dim, dtype=dtype).check()
    Case(q8mv, dim, [7, 500], [5, 9], heads=3, group=2, dim=dim, dtype=dtype).check()


def test_heads_side_by_side_cut_between_ctas(q8mv):
    Case(q8mv, 7, [20001], [1], heads=4, group=2, dim=64, page=64, tree=False, layout="token").check()
    Case(q8mv, 8, [9000, 20011, 1, 5, 3000], [2, 1, 1, 2, 1], heads=8, group=4, dim=128, page=32, dtype="bfloat16",
         layout="token", cols=9000).check()


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("layout,page", [("head", 16), ("token", 7)])
def test_wide_trees(q8mv, dim, layout, page):
    """More than 32 bf16 query rows a request, and tables that reach far: the tensor-memory path."""
    wide(q8mv, dim, [300, 0, 5, 1000], [40, 0, 33, 70], heads=2, group=2, dim=dim, page=page, dtype="bfloat16",
         layout=layout).check()


@pytest.mark.parametrize("length", [0, 1, 15, 16, 90, 112, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("tree", [True, False])
def test_wide_trees_around_the_tiles(q8mv, length, tree):
    for nodes in (34, 129, 150):
        wide(q8mv, length, [length], [nodes], heads=1, group=1, dim=64, page=5, dtype="bfloat16", tree=tree).check()


def test_wide_trees_cut_between_ctas(q8mv):
    wide(q8mv, 1, [20001], [35], heads=1, group=2, dim=64, page=64, dtype="bfloat16").check()
    wide(q8mv, 2, [9000, 20011, 1, 5, 13000], [40, 33, 50, 35, 41], heads=2, group=4, dim=128, page=32,
         dtype="bfloat16").check()
    wide(q8mv, 3, [90] * 60, [40] * 60, heads=3, group=1, dim=128, page=16, dtype="bfloat16").check()


def test_wide_trees_the_same_bits_again(q8mv):
    import torch

    c = wide(q8mv, 4, [3000, 700, 0], [50, 90, 36], heads=4, group=1, dim=128, dtype="bfloat16")
    a = c.run()
    for _ in range(20):
        for x, y in zip(a, c.run()):
            assert torch.equal(x, y)
    assert c.plan.check() == 0
    c.check(a)


def test_wide_trees_and_what_is_not_seen(q8mv):
    """Rows that see nothing; NaN, infinities and huge scales in unseen nodes and unused places."""
    import torch

    c = wide(q8mv, 5, [33, 140, 0], [40, 45, 50], heads=2, group=1, dim=64, dtype="bfloat16")
    for b in range(3):
        c.seen[b][:, 2] = False
        c.seen[b][:, 37] = False
    c.seen[2][5] = False
    mask = np.zeros((135, 2), np.uint32)
    for b, t in enumerate(c.nodes):
        for i, j in zip(*np.nonzero(c.seen[b])):
            mask[c.starts[b] + i, j // 32] |= np.uint32(1 << (j % 32))
    c.mask = torch.from_numpy(mask.view(np.int32)).cuda()
    c.check()
    used = np.zeros(c.host.kc.shape[0] * 16, bool)
    for b, (p, t) in enumerate(zip(c.lengths, c.nodes)):
        for j in [*range(p), *(p + i for i in range(t) if i not in (2, 37))]:
            used[c.table[b, j // 16] * 16 + j % 16] = True
    for bad in (np.nan, np.inf, -np.inf, 3e38, 1e30):
        for a in (c.host.ks, c.host.vs):
            flat = a.reshape(a.shape[0], a.shape[1], 16, -1)
            for s in np.flatnonzero(~used):
                flat[s // 16, :, s % 16] = bad
        c.device()
        c.check()
    c.table[0, 1] = 10 ** 9
    c.table[1, 0] = -5
    c.device()
    c.check()


def test_wide_trees_and_seen_values_that_are_not_finite(q8mv):
    import torch

    c = wide(q8mv, 6, [20], [40], heads=1, group=1, dim=64, dtype="bfloat16", tree=False)
    slot = c.table[0, 50 // 16] * 16 + 50 % 16  # node 30
    c.host.vs[slot // 16, :, slot % 16] = np.nan
    out, _ = c.run()
    assert torch.isfinite(out[:30]).all() and torch.isnan(out[30:]).all()


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_wide_trees_with_scales_of_any_size(q8mv, size):
    c = wide(q8mv, 7, [200], [40], dim=64, dtype="bfloat16")
    c.host.vs *= np.float32(size)
    c.check()
    c = wide(q8mv, 8, [200], [40], dim=64, dtype="bfloat16")
    c.host.ks *= np.float32(size)
    c.q = (c.q * (1 / size)).to(c.q.dtype)
    c.check()


def test_wide_trees_strided_rows(q8mv):
    import torch

    c = wide(q8mv, 9, [300], [40], heads=2, group=2, dim=128, dtype="bfloat16")
    want = c.run()
    outs = torch.full((40, 4, 140), 7.0, device="cuda", dtype=torch.bfloat16)
    got = c.run(out=outs[:, :, 5:133])
    assert torch.equal(got[0], want[0])
    assert bool((outs[:, :, :5] == 7).all()) and bool((outs[:, :, 133:] == 7).all())


@pytest.mark.parametrize("scale", [30.0, -30.0])
def test_wide_trees_large_scores(q8mv, scale):
    """Scores hundreds apart: where one key has all of a row's weight (the next below e^-40), out is its value within
    the two roundings of a value (f16 in the product, bf16 at the end), measured by the row's largest value."""
    c = wide(q8mv, 12, [300], [40], heads=2, group=2, dim=128, dtype="bfloat16")
    out, lse = (x.double().cpu().numpy() for x in c.run(scale=scale))
    pos = np.arange(340)
    keys, values = c.host.rows(c.table[0, pos // 16].astype(np.int64) * 16 + pos % 16)
    q = c.q.double().cpu().numpy()
    alone = 0
    for i in range(40):
        seen = np.array([j < 300 or c.sees(0, i, int(j) - 300) for j in pos])
        for a in range(4):
            s = np.where(seen, scale * (keys[:, a // 2] @ q[i, a]), -np.inf)
            first, second = np.argsort(-s)[:2]
            assert abs(lse[i, a] - s[first]) <= 1e-6 * abs(scale) * np.abs(keys[:, a // 2] * q[i, a]).sum(-1).max() + 1
            if s[first] - s[second] > 40:
                alone += 1
                v = values[first, a // 2]
                assert np.all(np.abs(out[i, a] - v) <= (2.0 ** -11 + 2.0 ** -8) * np.abs(v).max())
    assert alone > 40


def test_a_wait_that_runs_out_is_reported_and_the_plan_goes_on(q8mv):
    c = wide(q8mv, 10, [3000, 100], [40, 50], heads=2, group=2, dim=128, dtype="bfloat16")
    c.check()
    c.plan.set_wait(1)  # nanosecond: the first wait that has to wait runs out
    c.run()
    assert c.plan.check() == 1
    c.plan.set_wait(0)
    assert c.plan.check() == 0
    c.check()
    with pytest.raises(q8mv.Q8mvError):
        c.plan.set_wait(11 * 10 ** 9)


def test_items_cut_between_ctas(q8mv):
    """Few heads, long sequences: many CTAs share an item, and a CTA has two parts."""
    Case(q8mv, 1, [40001], [1], heads=1, group=2, dim=64, page=64, tree=False).check()
    Case(q8mv, 2, [9000, 20011, 1, 5, 13000], [2, 1, 1, 3, 1], heads=2, group=4, dim=128, page=32, dtype="bfloat16").check()


def test_many_requests(q8mv):
    rng = np.random.default_rng(5)
    nodes = rng.integers(0, 4, 400).tolist()
    Case(q8mv, 5, rng.integers(0, 90, 400).tolist(), nodes, heads=2, group=1, dim=32, page=8).check()


def test_the_same_bits_again_and_on_another_stream(q8mv):
    import torch

    c = Case(q8mv, 11, [5000, 777], [3, 8], heads=4, dim=128)
    a = c.run()
    b = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d = c.run()
    s.synchronize()
    for x, y, z in zip(a, b, d):
        assert torch.equal(x, y) and torch.equal(x, z)
    c.check(a)


def test_rows_that_see_nothing(q8mv):
    import torch

    c = Case(q8mv, 21, [0, 50, 0], [4, 3, 40], heads=2)
    c.seen[0][:] = False
    c.seen[2][7] = False
    c.mask = c.mask.clone()
    c.mask[0:4] = 0
    c.mask[7 + 7] = 0
    out, lse = c.run()
    c.check((out, lse))
    assert not out[:4].any() and torch.isneginf(lse[:4]).all() and torch.isneginf(lse[14]).all()


def test_a_mask_with_fewer_words_than_nodes(q8mv):
    Case(q8mv, 22, [10, 0], [70, 40], words=1).check()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_what_is_not_seen_has_no_effect(q8mv, dtype):
    """NaN, infinities and huge scales in unseen nodes, unused places and pages outside the cache."""
    import torch

    c = Case(q8mv, 31, [33, 64], [6, 5], heads=2, dtype=dtype)
    for b in range(2):
        c.seen[b][:, 2] = False
        c.seen[b][:, 4] = False
    mask = np.zeros((11, 1), np.uint32)
    for b, t in enumerate(c.nodes):
        for i, j in zip(*np.nonzero(c.seen[b])):
            mask[c.starts[b] + i, 0] |= np.uint32(1 << j)
    c.mask = torch.from_numpy(mask.view(np.int32)).cuda()
    want = c.run()
    c.check(want)
    used = np.zeros(c.host.kc.shape[0] * 16, bool)
    for b, (p, t) in enumerate(zip(c.lengths, c.nodes)):
        for j in [*range(p), *(p + i for i in range(t) if i not in (2, 4))]:
            used[c.table[b, j // 16] * 16 + j % 16] = True
    for bad in (np.nan, np.inf, -np.inf, 3e38, 1e30):
        for a in (c.host.ks, c.host.vs):
            flat = a.reshape(a.shape[0], a.shape[1], 16, -1)
            for s in np.flatnonzero(~used):
                flat[s // 16, :, s % 16] = bad
        c.device()
        for x, y in zip(c.run(), want):
            assert torch.equal(x, y), bad
    # pages outside the cache are not seen, wherever they point
    c.table[0, 1] = 10 ** 9
    c.table[1, 0] = -5
    c.device()
    c.check()


def test_seen_values_that_are_not_finite_reach_their_rows_only(q8mv):
    import torch

    c = Case(q8mv, 32, [20], [4], heads=1, group=1, tree=True)
    c.seen[0][:] = np.tril(np.ones((4, 4), bool))
    c.mask = torch.tensor([[1], [3], [7], [15]], dtype=torch.int32, device="cuda")
    slot = c.table[0, 22 // 16] * 16 + 22 % 16  # node 2
    c.host.vs[slot // 16, :, slot % 16] = np.nan
    out, _ = c.run()
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2:]).all()


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_scales_of_any_size(q8mv, size):
    c = Case(q8mv, 33, [200], [4], dim=64)
    c.host.vs *= np.float32(size)
    c.check()
    c = Case(q8mv, 34, [200], [4], dim=64)
    c.host.ks *= np.float32(size)
    c.q = c.q * (1 / size)
    c.check()


def test_large_scores(q8mv):
    """Scores far apart: the softmax is one key."""
    c = Case(q8mv, 35, [300], [4], dim=128)
    c.check(c.run(scale=20.0), scale=20.0)


def test_negative_lengths_and_short_tables(q8mv):
    c = Case(q8mv, 41, [-7, 200], [5, 3], page=16, cols=4)  # positions past 64 have no page
    c.check()
    c = Case(q8mv, 42, [10], [2], cols=0)
    out, _ = c.run()
    assert not out.any()


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_strided_queries_and_outputs(q8mv, dtype):
    import torch

    c = Case(q8mv, 51, [77, 30], [3, 4], heads=2, group=2, dim=64, dtype=dtype)
    want = c.run()
    big = torch.zeros(7, 9 * 64 + 3, device="cuda", dtype=c.q.dtype)
    view = torch.as_strided(big, (7, 4, 64), (9 * 64 + 3, 2 * 64, 1), 1)
    view.copy_(c.q)
    c.q = view
    outs = torch.full((7, 4, 100), 7.0, device="cuda", dtype=view.dtype)
    got = c.run(out=outs[:, :, 5:69])
    assert got[0].data_ptr() == outs[:, :, 5:69].data_ptr()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert bool((outs[:, :, :5] == 7).all()) and bool((outs[:, :, 69:] == 7).all())


def test_offsets_past_32_bits(q8mv):
    """A cache whose codes and scales pass 2^32 bytes: the same rows at its start and at its end."""
    import torch

    heads, dim, page = 8, 128, 64
    pages = (2 ** 32 + 2 ** 28) // (heads * dim * page)
    cache = q8mv.Cache(pages, page, heads, dim)
    n = 130
    k, v = torch.randn(n, heads, dim, device="cuda"), torch.randn(n, heads, dim, device="cuda")
    far = pages * page - n
    low, high = torch.arange(n, device="cuda"), torch.arange(far, far + n, device="cuda")
    cache.write(k, v, low)
    cache.write(k, v, high)
    for x, y in zip(cache.read(low), cache.read(high)):
        assert torch.equal(x, y)
    plan = q8mv.TreeAttention(16, heads, dim, 2, 2)
    first = far // page + 1  # whole pages at the end
    shift = first * page - far
    cache.move(torch.arange(far, far + n - shift, device="cuda"), torch.arange(far + shift, far + n, device="cuda").flip(0))
    cache.write(k[:n - shift], v[:n - shift], torch.arange(first * page, first * page + n - shift, device="cuda"))
    table = torch.tensor([[0, 1, 2], [first, first + 1, first + 2]], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, dim, device="cuda").expand(2, 16, dim)
    lengths = torch.full((2,), n - shift - 1, dtype=torch.int32, device="cuda")
    out = plan(q, cache, table, lengths)
    assert torch.equal(out[0], out[1]) and torch.isfinite(out).all() and out.any()


def test_a_plan_serves_smaller_calls_and_none(q8mv):
    import torch

    c = Case(q8mv, 61, [100, 40], [5, 6])
    c.plan = q8mv.TreeAttention(4, 2, 64, 9, 200)
    c.check()
    none = torch.empty(0, 4, 64, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = c.plan(none, c.cache, torch.empty(0, 3, **i32), torch.empty(0, **i32))
    assert out.shape == (0, 4, 64)


def test_refusals(q8mv):
    import torch

    c = Case(q8mv, 71, [100, 40], [5, 6])
    c.device()
    table, lengths, starts = c.args
    with pytest.raises(TypeError):
        c.plan(c.q.double(), c.cache, table, lengths, starts=starts)
    with pytest.raises(ValueError):
        c.plan(c.q[:, :2], c.cache, table, lengths, starts=starts)
    with pytest.raises(ValueError):
        c.plan(c.q.cpu(), c.cache, table, lengths, starts=starts)
    with pytest.raises(TypeError):
        c.plan(c.q, c.cache, table.long(), lengths, starts=starts)
    with pytest.raises(ValueError):
        c.plan(c.q, c.cache, table[:1], lengths, starts=starts)
    with pytest.raises(ValueError):
        c.plan(c.q, c.cache, table, lengths)  # 11 rows over 2 requests
    with pytest.raises(ValueError):
        c.plan(c.q, c.cache, table, lengths, starts=starts[:2])
    with pytest.raises(ValueError):
        c.plan(c.q, c.cache, table, lengths, starts=starts, mask=c.mask[:3])
    with pytest.raises(ValueError):
        c.plan(c.q, c.cache, table, lengths, starts=starts, out=torch.empty_like(c.q).half())
    with pytest.raises(q8mv.Q8mvError):  # another head size than the plan's
        c.plan(c.q, q8mv.Cache(2, 16, 2, 32), table, lengths, starts=starts)
    small = q8mv.TreeAttention(4, 2, 64, 1, 11)
    with pytest.raises(q8mv.Q8mvError):  # more requests than planned
        small(c.q, c.cache, table, lengths, starts=starts)
    small = q8mv.TreeAttention(4, 2, 64, 2, 10)
    with pytest.raises(q8mv.Q8mvError):  # more rows than planned
        small(c.q, c.cache, table, lengths, starts=starts)
