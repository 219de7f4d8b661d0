"""The verification's exchanges over a cluster: requests that reach the first one at once, many of them at a time."""
import numpy as np
import pytest

import kv_ref as ref
from test_gpu_kv_verify import inputs, q8mv, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("vocab", [1, 3, 200])
def test_rows_that_take_no_time(q8mv, dtype, vocab):  # noqa: F811
    """More requests than fit the GPU, rows of a few logits, some CTAs without any: CTAs start while others exchange."""
    rng = np.random.default_rng(vocab)
    sizes = rng.integers(0, 4, 300).tolist()
    logits, tokens, parents, uniforms, starts = inputs(rng, sizes, vocab, dtype)
    temperature = rng.uniform(0.3, 1.5, len(sizes)).astype(np.float32)
    temperature[::5] = 0
    first = run_and_check(q8mv, logits, tokens, parents, uniforms, starts, temperature)
    for _ in range(3):
        for a, b in zip(first, run_and_check(q8mv, logits, tokens, parents, uniforms, starts, temperature)):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("vocab", [40, 5000])
def test_children_refused_in_turn_from_the_same_words(q8mv, vocab):  # noqa: F811
    """Up to 31 siblings whose tokens lie side by side: their weights leave the same sums one after another."""
    import torch

    rng = np.random.default_rng(vocab + 3)
    nodes, batch = 32, 64
    logits = torch.from_numpy(rng.standard_normal((nodes * batch, vocab)).astype(np.float32)).cuda()
    tokens = np.concatenate([np.concatenate([[0], rng.permutation(31)]) for _ in range(batch)]).astype(np.int32)
    parents = np.tile(np.array([-1] + [0] * (nodes - 1), np.int32), batch)
    starts = (np.arange(batch + 1) * nodes).astype(np.int32)
    uniforms = rng.random(nodes * batch).astype(np.float32)
    uniforms.reshape(batch, nodes)[:, 1:] = 0.999999  # refused
    for _ in range(3):
        run_and_check(q8mv, logits, tokens, parents, uniforms, starts)


def test_how_many_requests_there_are_has_to_be_known(q8mv):  # noqa: F811
    """Rows of several requests are not taken for one request's: its walk would be a wrong one without an error."""
    import torch

    rng = np.random.default_rng(16)
    logits, tokens, parents, uniforms, starts = inputs(rng, [4, 4], 100, "float32")
    t, p, u, s = (torch.from_numpy(a).cuda() for a in (tokens, parents, uniforms, starts))
    plan = q8mv.TreeVerify(2, 8, 100)
    with pytest.raises(ValueError):
        plan(logits, t, p, u)
    want = plan(logits, t, p, u, starts=s)
    for how in (dict(requests=2), dict(temperature=torch.ones(2, device="cuda"))):
        assert all(torch.equal(a, b) for a, b in zip(plan(logits, t, p, u, **how), want))
    # a plan for one request needs nothing said
    one = q8mv.TreeVerify(1, 4, 100)
    for a, b in zip(one(logits[:4], t[:4], p[:4], u[:4]), (want[0][:4], want[1][:1], want[2][:1])):
        assert torch.equal(a, b)
