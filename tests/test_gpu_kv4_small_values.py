"""Attention over values far below 1, or of very different sizes: no weight times scale may leave f16's range unnoticed."""
import numpy as np
import pytest

from kv_ref import EPS
from test_gpu_kv4_attend import Case, q8mv  # noqa: F401

pytestmark = pytest.mark.gpu


def spread(c, factor):
    """The values' scales times factor (a number, or one for each page and place), rounded to f16 again."""
    c.host.vs = (c.host.vs.astype(np.float64) * factor).astype(np.float16)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("size", [1e-2, 1e-3, 1e-4, 1e-6, 0.0, 1e3])
@pytest.mark.parametrize("more", [dict(), dict(layout="token", cols=2 ** 16, heads=4), dict(nodes=[3, 9, 1, 2], page=24),
                                  dict(dim=64, group=1), dict(dim=96), dict(dim=192), dict(dim=256)])
def test_values_of_any_size(q8mv, dtype, size, more):  # noqa: F811
    args = dict(lengths=[400, 1, 33, 130], nodes=[1, 1, 1, 1], heads=2, group=3, dim=128, dtype=dtype)
    c = Case(q8mv, 3, **{**args, **more})
    spread(c, size)
    c.check()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("more", [dict(), dict(layout="token", cols=2 ** 16, heads=4, page=16), dict(nodes=[3, 9], page=24), dict(dim=256)])
@pytest.mark.parametrize("powers", [4, 13])
def test_values_of_very_different_sizes(q8mv, dtype, more, powers):  # noqa: F811
    """Each key's values times a power of two of its own."""
    args = dict(lengths=[2000, 75], nodes=[1, 1], heads=2, group=3, dim=128, dtype=dtype)
    c = Case(q8mv, 4, **{**args, **more})
    e = c.rng.integers(-powers, min(powers, 12) + 1, c.host.vs.shape[:3] + (1,))
    spread(c, 2.0 ** e)
    c.check()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("out_of", [2.0 ** 8, 2.0 ** 15])
@pytest.mark.parametrize("more", [dict(), dict(layout="token", cols=2 ** 16, heads=4), dict(nodes=[5, 5])])
def test_one_key_of_great_values_that_hardly_weighs(q8mv, dtype, out_of, more):  # noqa: F811
    """Its scale must not push the others' contributions out of f16's range: here it is all that is not of order 1, and its
    score is 30 below the others'."""
    args = dict(lengths=[600, 300], nodes=[1, 1], heads=2, group=2, dim=64, dtype=dtype)
    c = Case(q8mv, 5, tree=False, **{**args, **more})
    rng, page = c.rng, c.host.page_size
    c.host.kc[:], c.host.ks[:] = 8, 1.0
    q = np.zeros(c.q.shape, np.float32)
    q[..., 0] = 1.0
    for b in range(2):
        for pos in rng.integers(0, c.lengths[b], 3):
            at = (c.table[b, pos // page], slice(None), pos % page)
            c.host.kc[at][:, 0] = 0  # -8
            c.host.vs[at] = np.float16(out_of)
    c.q.copy_(c.q.new_tensor(q))
    c.check(c.run(scale=30 / 8), scale=30 / 8)


PEAKED = [(1e0, 10), (1e-1, 14), (1e-2, 16), (1e-3, 13), (1e-3, 16), (1e-3, 18), (1e-4, 13), (1e-4, 16), (1e-5, 16)]
FORMS = {"8 rows": dict(), "8 rows in turn": dict(page=64), "four heads": dict(layout="token", heads=4, page=64), "16 rows": dict(nodes=[6]),
         "16 rows in turn": dict(nodes=[6], page=64), "128 rows": dict(nodes=[33], group=2)}


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("size,below", PEAKED)
@pytest.mark.parametrize("form", sorted(FORMS))
def test_a_peak_of_nothing_over_many_small_values(q8mv, dtype, size, below, form):  # noqa: F811
    """One early key of value 0 has 2^below times any other's weight; 8192 others, all of one sign, are the answer.  So many
    requests read them that a request's keys are hardly cut, so that a warp has the peak and thousands behind it.

    Tolerance, with u and e as kv4_ref.attend: the weights' errors, twice; their f16 parts; a value's way through
    sums in f32, 32 and one for each 32 keys, of values with 8 taken off; and f16's end: a weight times a scale loses
    2^-25 up to three times, with codes of up to 8, where the peak's weight is 2^8 at least, as the scales are or, below
    2^-7, as they are brought up to 1 or more.  Then half an ulp of the type."""
    import torch

    if form == "128 rows" and dtype != "bfloat16":
        pytest.skip("bf16")
    n, many = 8192, 600 if form != "128 rows" else 160
    c = Case(q8mv, 6, **{**dict(lengths=[n], nodes=[1], heads=1, group=2, dim=64, dtype=dtype, tree=False, page=24), **FORMS[form]})
    rng, heads, nodes, page = c.rng, c.host.heads, c.nodes[0], c.host.page_size
    c.host.kc[:], c.host.ks[:] = 8, 1.0
    c.host.vc[:] = rng.integers(9, 16, c.host.vc.shape)
    c.host.vs[:] = (size / 8 * rng.uniform(0.9, 1, c.host.vs.shape)).astype(np.float16)
    peak = 70
    at = (c.table[0, peak // page], slice(None), peak % page)
    c.host.kc[at][:, 0] = 12  # a score of 4 times the scale
    c.host.vs[at] = 0.0
    c.device()
    q = torch.zeros(many * nodes, *c.q.shape[1:], dtype=c.q.dtype, device="cuda")
    q[..., 0] = 1.0
    scale = below * np.log(2) / 4
    plan = q8mv.TreeAttention4(c.q.shape[1], heads, 64, many, len(q))
    got = plan(q, c.cache, c.args[0].repeat(many, 1), c.args[1].repeat(many), scale=scale)
    got = got.double().cpu().numpy().reshape(many, nodes, heads, -1, 64)

    u, part = 2.0 ** -23, 2.0 ** -11 if dtype == "bfloat16" else 2.0 ** -23
    pos = np.arange(n + nodes)
    slots = c.table[0, pos // page].astype(np.int64) * page + pos % page
    values, steps = c.host.rows(slots)[1], c.host.steps(slots)[1]
    weights = np.where(pos == peak, 2.0 ** below, 1.0)
    e = (24 * scale * (4 + 16) + 8) * u
    d = float(c.host.vs.max())
    lost = 2.0 ** -33 * (d if d < 2.0 ** -7 else 1.0)
    for node in range(nodes):
        p = weights * (pos <= n + node)
        p /= p.sum()
        for h in range(heads):
            want = p @ values[:, h]  # of one sign: its own size
            tol = (2 * e + part) * want + (32 + n / 32) * u * (want + 16 * (p @ steps[:, h])) + n * 24 * lost
            tol += EPS[dtype] * (want + tol) + (2.0 ** -25 if dtype == "float16" else 0)
            err = np.abs(got[:, node, h] - want)
            assert (err <= tol).all(), (node, h, float((err / tol).max()), float((err / want).max()))
