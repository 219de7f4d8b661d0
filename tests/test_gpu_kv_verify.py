"""Verification of drafted tokens: whole numbers, so every result equals the walk in Python (kv_ref.walk)."""
import numpy as np
import pytest

import kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def shares(logits, temperature):
    """exp(z - max) of a request's rows as the header defines it, with CUDA's expf (torch.exp of f32)."""
    import torch

    x = logits.float()
    if temperature > 0:
        z = x * float(np.float32(1) / np.float32(temperature))
    else:
        z = x
    z = torch.where(torch.isnan(z), torch.full_like(z, -torch.inf), z)
    top = z.amax(-1, keepdim=True)
    if temperature > 0:
        e = torch.where(z == top, torch.ones_like(z), torch.exp(z - top))
    else:
        e = torch.zeros_like(z)
        for r in range(len(z)):
            e[r, int(np.flatnonzero((z[r] == top[r]).cpu().numpy())[0])] = 1
    e[(top == -torch.inf)[:, 0]] = 0
    return e.cpu().numpy()


def random_tree(rng, nodes, chain):
    return np.array([-1] + [i - 1 if chain else int(rng.integers(max(0, i - 5), i)) for i in range(1, nodes)], np.int32)


def run_and_check(q8mv, logits, tokens, parents, uniforms, starts, temperature=None, draft=None, max_rows=None):
    import torch

    rows, vocab = logits.shape
    batch = len(starts) - 1
    plan = q8mv.TreeVerify(batch, max_rows or max(rows, 1), vocab)
    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (tokens, parents, uniforms, starts)]
    t = torch.from_numpy(temperature).cuda() if temperature is not None else None
    got = plan(logits, dev[0], dev[1], dev[2], starts=dev[3], temperature=t, draft_probs=draft)
    path, count, token = (x.cpu().numpy() for x in got)
    d = draft.cpu().numpy() if draft is not None else None
    for b in range(batch):
        s = slice(starts[b], starts[b + 1])
        if starts[b] == starts[b + 1]:
            assert count[b] == 0 and token[b] == -1
            continue
        e = shares(logits[s], float(temperature[b]) if temperature is not None else 1.0)
        want, nxt = ref.walk(e, vocab, tokens[s], parents[s], uniforms[s], d[s] if d is not None else None)
        assert path[s].tolist() == want + [-1] * (starts[b + 1] - starts[b] - len(want)), b
        assert count[b] == len(want) - 1 and token[b] == nxt, (b, token[b], nxt)
    return path, count, token


def inputs(rng, sizes, vocab, dtype, chain=False, likely=True):
    import torch

    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = int(starts[-1])
    logits = rng.standard_normal((rows, vocab)).astype(np.float32) * 2
    tokens = rng.integers(0, vocab, rows).astype(np.int32)
    parents = np.concatenate([random_tree(rng, n, chain) for n in sizes if n] or [np.zeros(0, np.int32)]).astype(np.int32)
    if likely:
        for b in range(len(sizes)):
            for i in range(starts[b] + 1, starts[b + 1]):
                logits[starts[b] + parents[i], tokens[i]] = np.log(vocab) + 2
    return (torch.from_numpy(logits).cuda().to(getattr(torch, dtype)), tokens, parents,
            rng.random(rows).astype(np.float32), starts)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 5, 127, 128, 1000, 4099, 33000])
@pytest.mark.parametrize("sizes", [[1], [2, 6], [9, 0, 1, 14]])
def test_trees_without_draft_probabilities(q8mv, dtype, vocab, sizes):
    rng = np.random.default_rng(vocab + len(sizes))
    logits, tokens, parents, uniforms, starts = inputs(rng, sizes, vocab, dtype)
    temperature = rng.uniform(0.3, 1.5, len(sizes)).astype(np.float32)
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts, temperature)
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts)
    temperature[::2] = 0
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts, temperature)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", [3, 130, 5003, 140001])
@pytest.mark.parametrize("chain", [True, False])
def test_with_draft_probabilities(q8mv, dtype, vocab, chain):
    import torch

    rng = np.random.default_rng(vocab)
    sizes = [5, 8, 1, 11] if vocab < 10000 else [4, 3]
    logits, tokens, parents, uniforms, starts = inputs(rng, sizes, vocab, dtype, chain, likely=False)
    near = logits.float() + 1.0 * torch.randn(logits.shape, generator=torch.Generator("cuda").manual_seed(vocab), device="cuda")
    draft = torch.softmax(near, -1)
    p = draft.double().cpu().numpy()
    for b in range(len(sizes)):
        for i in range(starts[b] + 1, starts[b + 1]):
            row = p[starts[b] + parents[i]]
            tokens[i] = rng.choice(vocab, p=row / row.sum())
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts, np.array([0.8] * (len(sizes) - 1) + [1.3], np.float32), draft)
    # refusals at every node
    run_and_check(q8mv, logits, tokens, parents, np.full_like(uniforms, 0.999999), starts, None, draft)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("vocab", [4, 128, 5000, 33000])
@pytest.mark.parametrize("chain", [True, False])
def test_rows_that_are_brought_while_their_parents_are_summed(q8mv, dtype, vocab, chain):
    """Vocabularies in whole fours, paths along first children and beside them, with draft probabilities and without."""
    import torch

    rng = np.random.default_rng(vocab + 1)
    sizes = [9, 0, 14, 2]
    logits, tokens, parents, uniforms, starts = inputs(rng, sizes, vocab, dtype, chain)
    for u in (uniforms, np.full_like(uniforms, 1e-6), np.full_like(uniforms, 0.999999)):
        run_and_check(q8mv, logits, tokens, parents, u, starts, np.array([0.7, 1.0, 0.0, 1.2], np.float32))
    draft = torch.softmax(logits.float() + 0.3 * torch.randn(logits.shape, generator=torch.Generator("cuda").manual_seed(vocab), device="cuda"), -1)
    for u in (uniforms, np.full_like(uniforms, 1e-6), np.full_like(uniforms, 0.999999)):
        run_and_check(q8mv, logits, tokens, parents, u, starts, np.array([0.7, 1.0, 0.9, 1.2], np.float32), draft)
    # the same rows where four cannot be loaded at once
    other = torch.zeros(logits.shape[0], vocab + 3, device="cuda", dtype=logits.dtype)[:, 1:vocab + 1]
    other.copy_(logits)
    run_and_check(q8mv, other, tokens, parents, uniforms, starts)


def test_a_large_vocabulary(q8mv):
    """More logits than a lane holds in registers."""
    rng = np.random.default_rng(4)
    logits, tokens, parents, uniforms, starts = inputs(rng, [3, 2], 300007, "bfloat16")
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts)


def test_siblings_with_the_same_token_and_tokens_outside(q8mv):
    import torch

    rng = np.random.default_rng(6)
    logits = torch.zeros(6, 4, device="cuda")
    parents = np.array([-1, 0, 0, 0, 0, 0], np.int32)
    starts = np.array([0, 6], np.int32)
    for tokens in ([0, 2, 2, 1, 1, 3], [0, -1, 4, 2, 2 ** 30, 2], [0, 0, 1, 2, 3, 0]):
        for _ in range(20):
            run_and_check(q8mv, logits, np.array(tokens, np.int32), parents, rng.random(6).astype(np.float32), starts)


def test_many_children_and_many_nodes(q8mv):
    rng = np.random.default_rng(7)
    n, vocab = 300, 500
    logits, tokens, parents, uniforms, starts = inputs(rng, [n], vocab, "float32")
    parents[1:200] = 0  # 199 children of the root
    for _ in range(5):
        run_and_check(q8mv, logits, tokens, parents, rng.random(n).astype(np.float32), starts)


def test_parents_that_are_not_below_their_node(q8mv):
    """Such nodes are never reached."""
    rng = np.random.default_rng(8)
    logits, tokens, parents, uniforms, starts = inputs(rng, [6], 50, "float32")
    parents = np.array([-1, 5, -3, 0, 4, 77], np.int32)
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts)


def test_logits_that_are_not_finite(q8mv):
    import torch

    rng = np.random.default_rng(9)
    logits, tokens, parents, uniforms, starts = inputs(rng, [4, 4, 4, 4], 200, "float32")
    logits[0:4] = -torch.inf            # nothing left: no token
    logits[4, 7] = torch.inf            # certain
    logits[8:12, ::2] = -torch.inf      # a constraint on the vocabulary
    logits[12:16, 5:] = float("nan")    # counts as -inf
    logits[13, 0] = -0.0
    _, count, token = run_and_check(q8mv, logits, tokens, parents, uniforms, starts)
    assert token[0] == -1 and count[0] == 0
    t = np.zeros(4, np.float32)
    run_and_check(q8mv, logits, tokens, parents, uniforms, starts, t)


def test_extreme_uniforms(q8mv):
    rng = np.random.default_rng(10)
    logits, tokens, parents, uniforms, starts = inputs(rng, [5, 5], 1000, "float32")
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0 ** -40):
        run_and_check(q8mv, logits, tokens, parents, np.full_like(uniforms, u), starts)


@pytest.mark.parametrize("drafted", [False, True])
def test_tokens_come_out_as_the_target_would_draw_them(q8mv, drafted):
    """40,000 requests with two drafted siblings: the first token of each follows the target's probabilities."""
    import torch

    n, vocab = 40000, 7
    g = torch.Generator("cuda").manual_seed(12)
    row = torch.tensor([0.1, 1.0, -0.5, 0.3, 2.0, -3.0, 0.7], device="cuda")
    p = torch.softmax(row, -1)
    q = torch.softmax(torch.tensor([1.5, 0.2, 0.1, -1.0, 0.5, 0.0, 0.3], device="cuda"), -1)
    logits = row.expand(3 * n, vocab).contiguous()
    tokens = torch.zeros(n, 3, dtype=torch.int32, device="cuda")
    if drafted:
        tokens[:, 1:] = torch.multinomial(q.expand(n, vocab), 2, replacement=True, generator=g).int()
    else:
        tokens[:, 1], tokens[:, 2] = 4, 1
    parents = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda").repeat(n)
    uniforms = torch.rand(3 * n, generator=g, device="cuda")
    plan = q8mv.TreeVerify(n, 3 * n, vocab)
    path, count, token = plan(logits, tokens.view(-1), parents, uniforms, requests=n,
                              draft_probs=q.expand(3 * n, vocab).contiguous() if drafted else None)
    second = path.view(n, 3)[:, 1].long()
    first = torch.where(count > 0, torch.gather(tokens.long(), 1, second.clamp(min=0).unsqueeze(1))[:, 0], token.long())
    share = torch.bincount(first, minlength=vocab).double() / n
    # five standard deviations of a binomial share
    assert bool(((share - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / n).sqrt()).all()), (share, p)
    assert 0.1 < float((count > 0).double().mean()) < 0.99


def test_strides_and_alignment(q8mv):
    import torch

    rng = np.random.default_rng(13)
    logits, tokens, parents, uniforms, starts = inputs(rng, [6, 6], 1001, "float32")
    wide = torch.zeros(12, 1100, device="cuda")
    for offset in (0, 1, 2):
        view = wide[:, offset:offset + 1001]
        view.copy_(logits)
        run_and_check(q8mv, view, tokens, parents, uniforms, starts)


def test_another_stream_and_the_same_again(q8mv):
    import torch

    rng = np.random.default_rng(14)
    logits, tokens, parents, uniforms, starts = inputs(rng, [9] * 40, 20011, "bfloat16")
    plan = q8mv.TreeVerify(40, 360, 20011)
    dev = [torch.from_numpy(a).cuda() for a in (tokens, parents, uniforms)]
    a = plan(logits, *dev, requests=40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = plan(logits, *dev, requests=40)
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_refusals(q8mv):
    import torch

    rng = np.random.default_rng(15)
    logits, tokens, parents, uniforms, starts = inputs(rng, [4, 4], 100, "float32")
    t, p, u, s = (torch.from_numpy(a).cuda() for a in (tokens, parents, uniforms, starts))
    plan = q8mv.TreeVerify(2, 8, 100)
    plan(logits, t, p, u, starts=s)
    with pytest.raises(TypeError):
        plan(logits.double(), t, p, u, starts=s)
    with pytest.raises(ValueError):
        plan(logits[:, :99], t, p, u, starts=s)
    with pytest.raises(TypeError):
        plan(logits, t.long(), p, u, starts=s)
    with pytest.raises(ValueError):
        plan(logits, t, p[:7], u, starts=s)
    with pytest.raises(TypeError):
        plan(logits, t, p, u.double(), starts=s)
    with pytest.raises(ValueError):
        plan(logits, t, p, u, requests=3)
    with pytest.raises(ValueError):
        plan(logits, t, p, u, starts=s, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        plan(logits, t, p, u, starts=s, draft_probs=logits.half())
    with pytest.raises(q8mv.Q8mvError):  # more requests than planned
        plan(logits, t, p, u, requests=4)
    with pytest.raises(q8mv.Q8mvError):  # more rows than planned
        q8mv.TreeVerify(2, 7, 100)(logits, t, p, u, starts=s)
    lib = q8mv.library()
    args = __import__("q8_matrix_vector_gb300.kv", fromlist=["kv"]).VerifyArgs(
        logits.data_ptr(), 0, t.data_ptr(), p.data_ptr(), u.data_ptr(), 0, 0, t.data_ptr(), u.data_ptr(), s.data_ptr(),
        100, 0, 8, 2, 100, 0, 0)
    import ctypes
    assert lib.q8kv_verify(plan._h, ctypes.byref(args), None) == q8mv.Q8MV_ERR_INVALID_ARG  # outputs over inputs
