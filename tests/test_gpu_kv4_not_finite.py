"""A scale that is not finite makes all of a row NaN that sees its key, however little the key weighs."""
import numpy as np
import pytest

from test_gpu_kv4_attend import Case, q8mv  # noqa: F401

pytestmark = pytest.mark.gpu

SCALE = 20.0  # scores spread over hundreds, so that weights underflow

# one token of 8 rows, keys one by one (pages of 24) or 16 at a time; 16 rows; four heads a CTA; 128 rows
FORMS = {
    "8 rows": dict(lengths=[700, 90], nodes=[1, 1], heads=2, group=2, page=24),
    "8 rows in turn": dict(lengths=[700, 90], nodes=[1, 1], heads=2, group=2, page=16),
    "16 rows": dict(lengths=[700, 90], nodes=[6, 5], heads=2, group=2, page=24),
    "16 rows in turn": dict(lengths=[700, 90], nodes=[6, 5], heads=2, group=2, page=16),
    "four heads": dict(lengths=[700, 90], nodes=[1, 1], heads=4, group=2, page=16, layout="token", cols=2 ** 16),
    "128 rows": dict(lengths=[700, 90], nodes=[40, 33], heads=2, group=3, page=16, cols=8192),
}


def scores(c, row, head):
    """Of request 0's cached tokens, in 64 bits."""
    pos = np.arange(int(c.lengths[0]))
    slots = c.table[0, pos // c.host.page_size].astype(np.int64) * c.host.page_size + pos % c.host.page_size
    group = c.q.shape[1] // c.host.heads
    keys = c.host.rows(slots)[0][:, head // group]
    return SCALE * keys @ c.q[row, head].double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("dim", [64, 96, 128, 192])
def test_a_seen_scale_shows_whatever_its_key_weighs(q8mv, form, dtype, dim):  # noqa: F811
    import torch

    if form == "128 rows" and (dtype != "bfloat16" or dim > 128):
        pytest.skip("bf16 heads of up to 128")
    c = Case(q8mv, dim, dim=dim, dtype=dtype, tree=False, **FORMS[form])
    c.device()
    group = c.q.shape[1] // c.host.heads
    clean = c.run(scale=SCALE)[0]
    assert torch.isfinite(clean).all()
    # 127 powers of two below the largest, before and after it
    s = scores(c, 0, 0)
    best = int(s.argmax())
    spots = [int(s[:best].argmin())] if best else []
    spots += [best + 1 + int(s[best + 1:].argmin())] if best + 1 < len(s) else []
    assert spots and all(s[best] - s[i] > 100 for i in spots)
    rows0 = int(c.starts[1])
    for i in spots:
        at = (int(c.table[0, i // c.host.page_size]), 0, i % c.host.page_size)
        for scales in (c.cache.v_scales, c.cache.k_scales):
            for block, value in ((0, np.inf), ((dim - 1) // 32, np.nan), (0, -np.inf)):
                old = scales[at].clone()
                scales[(*at, block)] = value
                out, _ = c.run(scale=SCALE)
                scales[at] = old
                assert torch.isnan(out[:rows0, :group]).all(), (i, value)
                assert torch.equal(out[:rows0, group:], clean[:rows0, group:]) and torch.equal(out[rows0:], clean[rows0:])
    assert torch.equal(c.run(scale=SCALE)[0], clean)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("form", ["8 rows", "16 rows", "16 rows in turn", "four heads", "128 rows"])
def test_of_a_tree_only_the_nodes_that_see_it(q8mv, form, dtype):  # noqa: F811
    """A drafted node's scale: NaN for its ancestors' children that see it, and for nobody else."""
    import torch

    if form == "128 rows" and dtype != "bfloat16":
        pytest.skip("bf16")
    shape = dict(FORMS[form], nodes=[4, 3]) if form in ("8 rows", "four heads") else FORMS[form]
    c = Case(q8mv, 7, dim=128, dtype=dtype, **shape)
    c.device()
    group = c.q.shape[1] // c.host.heads
    clean = c.run(scale=SCALE)[0]
    rows0, node = int(c.starts[1]), 2
    pos = int(c.lengths[0]) + node
    at = (int(c.table[0, pos // c.host.page_size]), 0, pos % c.host.page_size)
    sees = torch.from_numpy(c.seen[0][:, node]).cuda()
    assert sees.any() and not sees.all()
    for scales in (c.cache.v_scales, c.cache.k_scales):
        old = scales[at].clone()
        scales[(*at, 1)] = np.inf
        out, _ = c.run(scale=SCALE)
        scales[at] = old
        assert torch.isnan(out[:rows0][sees][:, :group]).all()
        assert torch.equal(out[:rows0][~sees], clean[:rows0][~sees])
        assert torch.equal(out[:rows0, group:], clean[:rows0, group:]) and torch.equal(out[rows0:], clean[rows0:])
