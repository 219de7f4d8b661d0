"""Forms of the draft-tree attention and of the cache that the layouts and the binding's own calls leave out."""
import ctypes

import numpy as np
import pytest

import kv_ref as ref
from test_gpu_kv_attend import Case, q8mv, wide  # noqa: F401

pytestmark = pytest.mark.gpu


def side_by_side(q8mv, seed, lengths, nodes, heads, dim, page, **more):  # noqa: F811
    """A case whose tables reach far enough, in columns without pages, for a head a warp: 0.5 GB of keys and values."""
    per = len(nodes) * heads * (2 * dim + 8 * -(-dim // 32)) * page  # bytes of a column
    return Case(q8mv, seed, lengths, nodes, heads=heads, dim=dim, page=page, layout="token", cols=-(-500000000 // per) + 1, **more)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 160, 256])
@pytest.mark.parametrize("heads,group,nodes", [(4, 2, [1, 3, 0, 2]), (8, 1, [5, 1, 1, 8]), (4, 8, [1, 1, 1, 1])])
def test_a_head_a_warp(q8mv, dtype, dim, heads, group, nodes):  # noqa: F811
    side_by_side(q8mv, dim, [0, 35, 64, 500], nodes, heads, dim, 9, group=group, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_head_a_warp_cut_between_ctas(q8mv, dtype):  # noqa: F811
    side_by_side(q8mv, 7, [20001], [1], 4, 64, 64, group=2, tree=False, dtype=dtype).check()
    side_by_side(q8mv, 8, [9000, 0, 3000], [2, 8, 1], 8, 112, 32, group=1, dtype=dtype).check()


def test_a_head_a_warp_and_what_is_not_seen(q8mv):  # noqa: F811
    """NaN, infinities and huge scales in unused places; pages outside the cache."""
    import torch

    c = side_by_side(q8mv, 9, [33, 64], [2, 3], 4, 48, 16, group=1, tree=False)
    want = c.run()
    c.check(want)
    used = np.zeros(c.host.kc.shape[0] * 16, bool)
    for b, (p, t) in enumerate(zip(c.lengths, c.nodes)):
        for j in range(p + t):
            used[c.table[b, j // 16] * 16 + j % 16] = True
    for bad in (np.nan, np.inf, -np.inf, 3e38):
        for a in (c.host.ks, c.host.vs):
            for s in np.flatnonzero(~used):
                a[s // 16, :, s % 16] = bad
        c.device()
        for x, y in zip(c.run(), want):
            assert torch.equal(x, y), bad
    c.table[0, 1], c.table[1, 0] = 10 ** 9, -5
    c.device()
    c.check()


@pytest.mark.parametrize("make,dtype", [(Case, "float32"), (wide, "bfloat16")])
def test_tables_and_masks_wider_than_what_is_used(q8mv, make, dtype):  # noqa: F811
    """Rows of the table and of the mask that are parts of wider ones."""
    import torch

    from q8_matrix_vector_gb300 import kv

    c = make(q8mv, 61, [300, 20, 0], [40, 33, 50], heads=2, group=2, dim=64, dtype=dtype)
    want = c.run()
    c.check(want)
    table, lengths, starts = c.args
    batch, cols = table.shape
    rows, words = c.mask.shape
    wide_table = torch.full((batch, cols + 3), 1, dtype=torch.int32, device="cuda")
    wide_table[:, :cols] = table
    wide_mask = torch.full((rows, words + 5), -1, dtype=torch.int32, device="cuda")
    wide_mask[:, :words] = c.mask
    out, lse = torch.full_like(c.q, float("nan")), torch.full_like(want[1], float("nan"))
    row, head, _ = c.q.stride()
    args = kv.AttendArgs(c.q.data_ptr(), out.data_ptr(), lse.data_ptr(), kv._TYPES[c.q.dtype], batch, rows, row, head, row, head,
                         starts.data_ptr(), lengths.data_ptr(), wide_table.data_ptr(), cols + 3, cols, words,
                         wide_mask.data_ptr(), words + 5, 64 ** -0.5)
    assert q8mv.library().q8kv_attend(c.plan._h, c.cache._ref, ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_any_order_of_pages_heads_and_places(q8mv, order, dtype):  # noqa: F811
    """Caches that are permuted views: written, moved, read and attended."""
    import torch

    pages, heads, page, dim = 7, 4, 9, 80
    back = [order.index(i) for i in range(3)] + [3]
    parts = [torch.zeros(*(np.array([pages, heads, page])[list(order)]), n, dtype=t, device="cuda").permute(*back)
             for n, t in ((dim, torch.int8), (3, torch.float32)) * 2]
    plain, cache = q8mv.Cache(pages, page, heads, dim), q8mv.Cache.of(*parts)
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn(50, heads, dim, device="cuda", generator=g) for _ in range(2))
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:50].contiguous()
    for x in (plain, cache):
        x.write(k, v, slots)
        x.move(slots[1:6].contiguous(), slots[:5].contiguous())
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(plain, name), getattr(cache, name))
    assert all(torch.equal(a, b) for a, b in zip(plain.read(slots), cache.read(slots)))
    c = Case(q8mv, 62, [20, 3], [3, 9], heads=heads, group=2, dim=dim, page=page, dtype=dtype)
    c.device()
    whole = c.cache
    full = [torch.empty(*(np.array(t.shape[:3])[list(order)]), t.shape[3], dtype=t.dtype, device="cuda").permute(*back).copy_(t)
            for t in (whole.k_codes, whole.k_scales, whole.v_codes, whole.v_scales)]
    c.cache = q8mv.Cache.of(*full)
    c.check()


def test_two_plans_on_two_streams_at_once(q8mv):  # noqa: F811
    import torch

    cases = [wide(q8mv, 63, [3000, 700, 0], [50, 90, 36], heads=4, group=1, dim=128, dtype="bfloat16"),
             wide(q8mv, 64, [2000, 900], [40, 60], heads=4, group=1, dim=128, dtype="bfloat16"),
             Case(q8mv, 65, [9000, 20], [1, 4], heads=4, group=2, dim=128, dtype="float32")]
    first = []
    for c in cases:
        first.append(c.run())
        c.check(first[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(c.run())
    torch.cuda.synchronize()
    for want, runs in zip(first, got):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))
    assert cases[0].plan.check() == 0 and cases[1].plan.check() == 0
