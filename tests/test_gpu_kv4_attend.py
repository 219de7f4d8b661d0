"""Draft-tree attention over the Q4_0 cache against the 64-bit reference (tolerances derived in kv4_ref.attend)."""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


class Case:
    """Requests with their own lengths and trees over one cache."""

    def __init__(self, q8mv, seed, lengths, nodes, heads=2, group=2, dim=64, page=16, dtype="float32", layout="head",
                 tree=True, cols=None, words=None, density=0.5):
        import torch

        rng = self.rng = np.random.default_rng(seed)
        self.dtype, self.nodes, self.tree, self.dim = dtype, nodes, tree, dim
        self.lengths = np.array(lengths, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.rows = rows = int(self.starts[-1])
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
        self.seen = [rng.random((t, t)) < density for t in nodes]
        self.words = words if words is not None else -(-max(max(nodes), 1) // 32)
        mask = np.zeros((rows, self.words), np.uint32)
        for b, t in enumerate(nodes):
            for i, j in zip(*np.nonzero(self.seen[b])):
                if j < 32 * self.words:
                    mask[self.starts[b] + i, j // 32] |= np.uint32(1 << (j % 32))
        self.mask = torch.from_numpy(mask.view(np.int32)).cuda() if tree else None
        self.plan = q8mv.TreeAttention4(heads * group, heads, dim, len(nodes), max(rows, 1))
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
        out, lse = self.run() if got is None else got
        want = ref.attend(self.host, self.q.float().cpu().numpy(), self.table, self.lengths, self.starts, self.sees,
                          1 / np.sqrt(self.dim) if scale is None else scale, self.dtype)
        for x, y, tol, what in ((out, want[0], want[2], "out"), (lse, want[1], want[3], "lse")):
            x = x.float().cpu().numpy().astype(np.float64)
            empty = np.isneginf(y)
            assert np.array_equal(np.isneginf(x), empty), what
            err = np.abs(np.where(empty, 0, x) - np.where(empty, 0, y))
            assert (err <= tol).all(), (what, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_single_tokens_of_all_heads(q8mv, dtype, dim, group):
    Case(q8mv, dim + group, [0, 1, 31, 32, 33, 127, 128, 129, 300], [1] * 9, group=group, dim=dim, dtype=dtype,
         tree=False).check()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 80, 128, 192])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("nodes", [[5, 0, 17, 1], [33, 2, 40, 31], [70, 3, 0, 64]])
def test_trees(q8mv, dtype, dim, layout, nodes):
    Case(q8mv, dim + nodes[0], [200, 0, 64, 5], nodes, group=3, dim=dim, dtype=dtype, layout=layout, page=24).check()


@pytest.mark.parametrize("page", [1, 5, 16, 100, 256])
def test_pages_of_any_size(q8mv, page):
    Case(q8mv, page, [333, 16, 1], [3, 1, 9], dim=96, page=page, dtype="bfloat16").check()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_chains_and_masks_that_leave_nothing(q8mv, dtype):
    Case(q8mv, 1, [0, 0, 7], [6, 1, 2], tree=False, dtype=dtype).check()
    Case(q8mv, 2, [0, 0, 3], [6, 1, 2], density=0.0, dtype=dtype).check()
    Case(q8mv, 3, [10, 0], [40, 40], words=1, dtype=dtype).check()  # bits past the words are 0
    Case(q8mv, 4, [-5, 40], [3, 3], dtype=dtype).check()


def test_tables_that_end_early_and_pages_that_are_not_there(q8mv):
    c = Case(q8mv, 5, [400, 90], [4, 4], cols=6, dim=128, dtype="bfloat16")
    c.table[0, 2], c.table[1, 1] = -1, 2 ** 30
    c.check()
    c = Case(q8mv, 6, [50, 90], [1, 1], dim=128, tree=False)
    c.table[0] = -7  # nothing is seen at all
    c.check()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_long_sequences_are_cut_and_joined(q8mv, dtype):
    # one request's keys over all CTAs: parts are joined in two levels
    Case(q8mv, 7, [30000], [1], heads=1, group=4, dim=128, dtype=dtype, tree=False, page=64).check()
    Case(q8mv, 8, [9000, 3, 2500], [1, 2, 9], heads=3, group=2, dim=64, dtype=dtype, page=32).check()


def test_what_is_not_seen_does_not_matter(q8mv):
    """Infinite and NaN scales, of keys and values, in masked and absent places."""
    import torch

    c = Case(q8mv, 9, [70, 33], [6, 4], dim=128, dtype="float32")
    for b in range(2):
        # node 1 is seen by nobody
        c.seen[b][:, 1] = False
    mask = c.mask.cpu().numpy().view(np.uint32) & ~np.uint32(2)
    c.mask = torch.from_numpy(mask.view(np.int32)).cuda()
    c.device()
    for b, value in ((0, np.inf), (1, np.nan)):
        for pos in (int(c.lengths[b]) + 1, int(c.lengths[b]) + c.nodes[b]):
            if pos // 16 < c.table.shape[1] and c.table[b, pos // 16] >= 0:
                at = (int(c.table[b, pos // 16]), slice(None), pos % 16)
                for s in (c.cache.k_scales, c.cache.v_scales):
                    s[at] = value
    c.check(c.run())


def test_a_seen_value_that_is_not_finite_shows(q8mv):
    import torch

    c = Case(q8mv, 10, [40, 40], [1, 1], dim=64, tree=False)
    c.device()
    c.cache.v_scales[int(c.table[1, 1]), 1, 3] = float("inf")
    out, _ = c.run()
    bad = torch.isnan(out)
    assert not bad[0].any() and not bad[1, :2].any() and bad[1, 2:].all()


def test_strides_scales_and_rows_behind_the_last(q8mv):
    import torch

    c = Case(q8mv, 11, [100, 40], [3, 2], heads=2, group=3, dim=80, dtype="bfloat16")
    wide = torch.full((c.rows + 3, 9, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(c.rows, 7, 83, dtype=torch.bfloat16, device="cuda")
    q[:, 1:, 2:82] = c.q
    c.q = q[:, 1:, 2:82]
    for scale in (0.25, -0.1, 0.0):
        out = wide[:c.rows, 2:8, 5:85]
        got, lse = c.run(out=out, scale=scale)
        c.check((got, lse), scale=scale)
    rest = wide.clone()
    rest[:c.rows, 2:8, 5:85] = 7
    assert (rest == 7).all()
    # starts that leave the last rows to nobody
    starts = c.args[2].clone()
    starts[2] = 4
    mine = torch.full((c.rows, 6, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    c.plan(c.q, c.cache, c.args[0], c.args[1], starts=starts, mask=c.mask, out=mine)
    assert (mine[4] == 7).all() and not (mine[3] == 7).any()


def test_queries_of_any_size(q8mv):
    import torch

    c = Case(q8mv, 12, [60, 60, 60], [1, 1, 1], dim=64, tree=False)
    c.q[0] *= 1e-30
    c.q[1] *= 1e3
    c.q[2, 1:] = 0
    c.check()
    for dtype in ("float16", "bfloat16"):
        c = Case(q8mv, 13, [60, 60], [1, 1], dim=64, tree=False, dtype=dtype)
        c.q[0] *= 2.0 ** -14
        c.check()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_same_bits_again_in_a_graph_and_on_another_stream(q8mv, dtype):
    import torch

    c = Case(q8mv, 14, [5000, 3, 700, 64], [1, 8, 3, 20], heads=4, group=4, dim=128, dtype=dtype)
    out, lse = c.run()
    for _ in range(3):
        again = c.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = c.run()
    side.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = c.run()
    for _ in range(3):
        held[0].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, held[0]) and torch.equal(lse, held[1])
    # other lengths under the same graph
    c.args[1].copy_(torch.tensor([1, 2, 3, 4], dtype=torch.int32))
    graph.replay()
    c.lengths = np.array([1, 2, 3, 4], np.int32)
    c.check(held)


def test_two_plans_at_once(q8mv):
    import torch

    cases = [Case(q8mv, 20 + i, [3000, 50], [1, 7], heads=2, group=4, dim=128, dtype="bfloat16") for i in range(2)]
    want = [c.run()[0].clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run()[0])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_refusals(q8mv):
    import torch

    c = Case(q8mv, 15, [20, 20], [2, 2], dim=64)
    c.device()
    table, lengths, starts = c.args
    with pytest.raises(TypeError):
        c.plan(c.q, q8mv.Cache(4, 16, 2, 64), table, lengths)
    with pytest.raises(TypeError):
        q8mv.TreeAttention(4, 2, 64, 2, 8)(c.q, c.cache, table, lengths)
    with pytest.raises(ValueError):
        c.plan(c.q[:, :2], c.cache, table, lengths)
    with pytest.raises(TypeError):
        c.plan(c.q.double(), c.cache, table, lengths)
    with pytest.raises(ValueError):
        c.plan(c.q[:3], c.cache, table, lengths)
    with pytest.raises(ValueError):
        c.plan(c.q, c.cache, table[:1], lengths)
    with pytest.raises(q8mv.Q8mvError):
        q8mv.TreeAttention4(4, 2, 64, 1, 8)(c.q, c.cache, table, lengths)
    with pytest.raises(q8mv.Q8mvError):
        q8mv.TreeAttention4(4, 2, 128, 2, 8)(torch.zeros(4, 4, 128, device="cuda"), c.cache, table, lengths)
    with pytest.raises(q8mv.Q8mvError):
        q8mv.TreeAttention4(5, 2, 64, 2, 8)
    with pytest.raises(q8mv.Q8mvError):
        q8mv.TreeAttention4(4, 2, 72, 2, 8)
    assert c.plan(c.q[:0], c.cache, table, lengths).shape == (0, 4, 64)


def wide(q8mv, seed, lengths, nodes, **more):
    """A case that 128 rows at a time take: more than 32 bf16 rows a request, and a table that reaches far."""
    return Case(q8mv, seed, lengths, nodes, dtype="bfloat16", cols=131072 // more.get("page", 16), **more)


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("nodes,group", [([40, 0, 33, 64], 3), ([31, 31], 4), ([200, 7], 2)])
def test_128_rows_at_a_time(q8mv, dim, layout, nodes, group):
    lengths = [700, 3, 129, 0][:len(nodes)]
    wide(q8mv, dim + nodes[0], lengths, nodes, group=group, dim=dim, layout=layout, page=32).check()


def test_128_rows_cut_over_many_ctas(q8mv):
    c = wide(q8mv, 31, [5000, 1300], [31, 31], heads=3, group=4, dim=128, page=16)
    c.check()
    out, lse = c.run()
    for _ in range(3):
        again = c.run()
        assert (out == again[0]).all() and (lse == again[1]).all()
    assert c.plan.check() == 0


def test_128_rows_of_nothing_and_of_what_is_not_finite(q8mv):
    import torch

    wide(q8mv, 32, [0, 0], [40, 40], dim=128, density=0.0).check()
    wide(q8mv, 33, [300, 0], [40, 40], dim=96, tree=False).check()
    c = wide(q8mv, 34, [300, 60], [40, 40], dim=128)
    for b in range(2):
        c.seen[b][:, 1] = False
    mask = c.mask.cpu().numpy().view(np.uint32)
    mask[:, 0] &= ~np.uint32(2)
    c.mask = torch.from_numpy(mask.view(np.int32)).cuda()
    c.device()
    for b, value in ((0, np.inf), (1, np.nan)):
        pos = int(c.lengths[b]) + 1
        for s in (c.cache.k_scales, c.cache.v_scales):
            s[int(c.table[b, pos // 16]), :, pos % 16] = value
    c.check(c.run())
    # a prefix key that everyone sees
    c.cache.v_scales[int(c.table[0, 2]), 1, 3] = float("inf")
    out, _ = c.run()
    assert torch.isnan(out[:40, 2:]).all() and not torch.isnan(out[:40, :2]).any() and not torch.isnan(out[40:]).any()


def test_128_rows_strided(q8mv):
    import torch

    c = wide(q8mv, 35, [200, 70], [36, 40], heads=2, group=3, dim=80)
    q = torch.zeros(c.rows, 7, 83, dtype=torch.bfloat16, device="cuda")
    q[:, 1:, 2:82] = c.q
    c.q = q[:, 1:, 2:82]
    out = torch.full((c.rows + 1, 8, 85), 7.0, dtype=torch.bfloat16, device="cuda")
    got = c.run(out=out[:c.rows, 1:7, 3:83], scale=-0.2)
    c.check(got, scale=-0.2)
    out[:c.rows, 1:7, 3:83] = 7
    assert (out == 7).all()


def test_a_wait_that_runs_out_is_reported(q8mv):
    """A bound of one nanosecond: the call ends, the plan says so, and its next call is as ever."""
    c = wide(q8mv, 36, [3000, 1300], [31, 31], heads=3, group=4, dim=128)
    want = [x.clone() for x in c.run()]
    assert c.plan.check() == 0
    c.plan.set_wait(1)
    c.run()
    assert c.plan.check() in (0, 1)  # (a wait may be over before its bound is looked at)
    assert c.plan.check() == 0
    c.plan.set_wait(0)
    again = c.run()
    assert (want[0] == again[0]).all() and (want[1] == again[1]).all() and c.plan.check() == 0


def side_by_side(q8mv, seed, lengths, nodes, **more):
    """A case that four heads a CTA take: a token's heads side by side, a table that reaches far, at most 8 rows."""
    return Case(q8mv, seed, lengths, nodes, layout="token", cols=2 ** 20 // more.get("page", 16), **more)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("heads,group,nodes", [(4, 8, [1, 1, 1, 0]), (8, 1, [3, 1, 0, 8]), (4, 3, [2, 2, 1, 3])])
def test_four_heads_a_cta(q8mv, dtype, dim, heads, group, nodes):
    side_by_side(q8mv, dim + group, [300, 1, 77, 0], nodes, heads=heads, group=group, dim=dim, dtype=dtype, page=24).check()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_four_heads_a_cta_cut_over_many(q8mv, dtype):
    c = side_by_side(q8mv, 41, [9000, 40], [1, 2], heads=4, group=2, dim=128, dtype=dtype, page=64)
    c.check()
    out, lse = c.run()
    for _ in range(3):
        again = c.run()
        assert (out == again[0]).all() and (lse == again[1]).all()


def test_four_heads_a_cta_masks_and_what_is_not_finite(q8mv):
    import torch

    side_by_side(q8mv, 42, [0, 0], [3, 3], heads=4, group=2, dim=128, density=0.0).check()
    c = side_by_side(q8mv, 43, [100, 30], [4, 4], heads=8, group=1, dim=96, dtype="bfloat16")
    for b in range(2):
        c.seen[b][:, 1] = False
    mask = c.mask.cpu().numpy().view(np.uint32) & ~np.uint32(2)
    c.mask = torch.from_numpy(mask.view(np.int32)).cuda()
    c.device()
    for b, value in ((0, np.inf), (1, np.nan)):
        pos = int(c.lengths[b]) + 1
        for s in (c.cache.k_scales, c.cache.v_scales):
            s[int(c.table[b, pos // 16]), :, pos % 16] = value
    c.check(c.run())


@pytest.mark.parametrize("nodes", [[1, 1], [40, 40]])
def test_tables_without_columns(q8mv, nodes):
    Case(q8mv, 44, [30, 0], nodes, cols=0, dim=128, dtype="bfloat16").check()
