"""Rotary positions against 64 bits, and their fused form against the separate calls."""
import numpy as np
import pytest

import kv4_ref as ref
import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def make(rng, shape, dtype):
    import torch

    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(getattr(torch, dtype))


def close(got, want, size, dtype, turns=0.0):
    """cos and sin are rounded to f32 once and each of two products and their sum: 2^-24 each of what they round, times
    the factor's own, 5 in all; the angle in 64 bits has an error of its own, `turns`; then half an ulp of the type."""
    got = got.float().cpu().numpy().astype(np.float64)
    tol = (5 * 2.0 ** -24 + turns) * size
    tol = tol + kv_ref.EPS[dtype] * (np.abs(want) + tol) + (2.0 ** -25 if dtype == "float16" else 1e-37)
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())


SHAPES = [(64, 64), (128, 128), (80, 32), (128, 64), (96, 20), (64, 2), (18, 6), (256, 256), (576, 512)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads", [(1, 1), (37, 5), (1200, 8)])
def test_forward_and_back(q8mv, dtype, dim, rot, interleaved, n, heads):
    import torch

    rng = np.random.default_rng(dim + rot + n)
    rotary = q8mv.Rotary(dim, rot, interleaved=interleaved)
    x = make(rng, (n, heads, dim), dtype)
    pos = rng.integers(0, 5000, n)
    if n > 30:
        pos[:4] = [0, 1, 2 ** 20, -7]
    at = torch.from_numpy(pos).cuda()
    # an f64 product of up to 2^20 radians and its cosine: 2^-53 of 2^20 each, and pi's own rounding in the reduction
    angle = 2.0 ** 20 * 2.0 ** -51
    y = rotary(x, at)
    close(y, *ref.rotate(x.float().cpu().numpy(), pos, rotary.turning, 1.0, interleaved), dtype, angle)
    back = rotary(y, at, inverse=True)
    close(back, *ref.rotate(y.float().cpu().numpy(), pos, rotary.turning, 1.0, interleaved, back=True), dtype, angle)
    # in place, and to a place of its own
    z = x.clone()
    assert rotary(z, at, out=z) is z and torch.equal(z, y)
    wide = torch.full((n, heads + 1, dim + 3), 5.0, dtype=x.dtype, device="cuda")
    got = rotary(x, at, out=wide[:, 1:, 1:dim + 1])
    assert torch.equal(got, y)
    wide[:, 1:, 1:dim + 1] = 5
    assert (wide == 5).all()
    strided = torch.zeros(n, heads, dim + 3, dtype=x.dtype, device="cuda")[:, :, 1:dim + 1]
    strided.copy_(x)
    assert torch.equal(rotary(strided, at), y)


def test_the_turn_is_the_transpose(q8mv):
    """<turn(x), g> = <x, turn back(g)>, and the difference quotient of a linear map is its value."""
    import torch

    rng = np.random.default_rng(0)
    for interleaved in (False, True):
        rotary = q8mv.Rotary(64, 48, interleaved=interleaved, scaling=dict(kind="yarn", factor=4.0, original=2048))
        x, g = make(rng, (9, 3, 64), "float32"), make(rng, (9, 3, 64), "float32")
        at = torch.arange(9, device="cuda") * 911
        a = (rotary(x, at).double() * g.double()).sum()
        b = (x.double() * rotary(g, at, inverse=True).double()).sum()
        # 27 * 64 terms, each with 5 * 2^-24 of at most |x| |g| factor
        assert abs(a - b) <= 2 * 5 * 2.0 ** -24 * rotary.factor * 2 * (x.double().norm() * g.double().norm())
        h = rotary(x + g, at).double() - rotary(x, at).double()
        want = rotary(g, at).double()
        assert (h - want).abs().max() <= 20 * 2.0 ** -24 * rotary.factor * (x.abs() + g.abs()).max().double() * 2


@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=8.0), dict(kind="ntk", factor=8.0),
                                     dict(kind="yarn", factor=8.0, original=4096),
                                     dict(kind="bands", factor=8.0, original=4096)])
def test_angles_are_exact_far_away(q8mv, scaling):
    """Against whole-number turns: no position's angle loses bits."""
    from fractions import Fraction

    import torch

    rotary = q8mv.Rotary(128, scaling=scaling)
    pos = np.array([0, 1, 4095, 131071, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 40 + 12345, -(2 ** 33) - 1], np.int64)
    x = torch.zeros(len(pos), 1, 128, device="cuda")
    x[:, :, :64] = 1
    y = rotary(x, torch.from_numpy(pos).cuda()).cpu().numpy()[:, 0]
    from q8_matrix_vector_gb300.rotary import _PI
    for r, p in enumerate(pos.tolist()):
        for i, f in enumerate(rotary.turning):
            turn = Fraction(p * round(Fraction(f) / (2 * _PI) * 2 ** 64) % 2 ** 64, 2 ** 64)
            angle = float(turn if turn < Fraction(1, 2) else turn - 1) * 2 * np.pi
            for got, want in ((y[r, i], np.cos(angle)), (y[r, 64 + i], np.sin(angle))):
                # rounded to f32 and times the factor, rounded: 2^-24 each, and 2^-42 before
                want *= rotary.factor
                assert abs(got - want) <= 2 * 2.0 ** -24 * abs(want) + 2.0 ** -42 * rotary.factor, (p, i)


def test_cosines_are_those_of_64_bits(q8mv):
    """An error below 2^-42, 2^-45 on the mean, turns the rounding of a value between 1/2 and 1 once in 2^20 (2^-45 of the
    2^-25 to a midpoint), of smaller ones a little more often: a few of two million, by a unit of the last place."""
    import torch

    rotary = q8mv.Rotary(128)
    rng = np.random.default_rng(0)
    pos = rng.integers(0, 2 ** 22, 2 ** 15)
    x = torch.zeros(len(pos), 1, 128, device="cuda")
    x[:, :, :64] = 1
    got = rotary(x, torch.from_numpy(pos).cuda()).cpu().numpy()[:, 0]
    from fractions import Fraction

    from q8_matrix_vector_gb300.rotary import _PI
    units = np.array([round(Fraction(f) / (2 * _PI) * 2 ** 64) % 2 ** 64 for f in rotary.turning], np.uint64)
    with np.errstate(over="ignore"):
        turn = (pos.astype(np.uint64)[:, None] * units).view(np.int64).astype(np.float64) * (2 * np.pi / 2.0 ** 64)
    want = np.concatenate([np.cos(turn), np.sin(turn)], 1).astype(np.float32)
    off = got != want
    assert off.sum() <= 100 and (np.abs(got - want) <= np.spacing(np.abs(want)) * 1.01).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 128, True), (80, 32, False), (96, 20, False),
                                                 (112, 10, True), (192, 192, False), (256, 64, True)])
@pytest.mark.parametrize("n,heads,group", [(1, 1, 1), (67, 3, 2), (900, 8, 4)])
def test_rotating_and_writing_at_once(q8mv, bits, dtype, dim, rot, interleaved, n, heads, group):
    import torch

    rng = np.random.default_rng(n + dim)
    rotary = q8mv.Rotary(dim, rot, interleaved=interleaved)
    kind = q8mv.Cache4 if bits == 4 else q8mv.Cache
    fused, apart = (kind(n // 16 + 2, 16, heads, dim) for _ in range(2))
    qkv = make(rng, (n, heads * (group + 2), dim), dtype)
    q, k, v = qkv.split([heads * group, heads, heads], 1)
    slots = torch.from_numpy(rng.permutation((n // 16 + 2) * 16)[:n]).cuda()
    slots[::9] = -1
    at = torch.from_numpy(rng.integers(0, 100000, n)).cuda()
    got = rotary.write(fused, q, k, v, at, slots)
    assert torch.equal(got, rotary(q, at))
    # apart: the turned keys in 32 bits, so that no rounding comes between
    apart.write(rotary(k.float(), at), v.float(), slots)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(fused, name), getattr(apart, name)), name
    # in place, and without q
    other = kind(n // 16 + 2, 16, heads, dim)
    mine = qkv.clone()
    rotary.write(other, mine[:, :heads * group], mine[:, heads * group:heads * (group + 1)], mine[:, heads * (group + 1):], at,
                 slots, out=mine[:, :heads * group])
    assert torch.equal(mine[:, :heads * group], got) and torch.equal(mine[:, heads * group:], qkv[:, heads * group:])
    assert torch.equal(other.k_codes, fused.k_codes)
    other.k_codes.zero_()
    assert rotary.write(other, None, k, v, at, slots) is None and torch.equal(other.k_codes, fused.k_codes)


@pytest.mark.parametrize("bits", [4, 8])
def test_values_that_are_not_numbers(q8mv, bits):
    import torch

    kind = q8mv.Cache4 if bits == 4 else q8mv.Cache
    rotary = q8mv.Rotary(64)
    k = torch.randn(8, 1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    k[1, 0, 3], k[2, 0, 40], k[3, 0, 7] = float("nan"), float("inf"), 0.0
    k[4] = 0
    at, slots = torch.arange(8, device="cuda"), torch.arange(8, device="cuda")
    fused, apart = kind(1, 16, 1, 64), kind(1, 16, 1, 64)
    rotary.write(fused, None, k, k, at, slots)
    apart.write(rotary(k, at), k, slots)
    for name in ("k_codes", "v_codes"):
        assert torch.equal(getattr(fused, name), getattr(apart, name)), name
    for name in ("k_scales", "v_scales"):
        a, b = getattr(fused, name), getattr(apart, name)
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())), name


def test_streams_and_graphs(q8mv):
    import torch

    rotary = q8mv.Rotary(128)
    cache = q8mv.Cache4(8, 16, 2, 128)
    q, k = torch.randn(5, 4, 128, device="cuda"), torch.randn(5, 2, 128, device="cuda")
    at, slots = torch.arange(5, device="cuda"), torch.arange(5, device="cuda")
    want = rotary(q, at + 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rotary.write(cache, q, k, k, at, slots)
    at.add_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = rotary(q, at)
    side.synchronize()
    assert torch.equal(again, want)


def test_refusals(q8mv):
    import torch

    rotary = q8mv.Rotary(64)
    x, at = torch.zeros(3, 2, 64, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (dict(rotary_dim=3), dict(rotary_dim=66), dict(rotary_dim=0), dict(turning=[1.0]), dict(base=-1.0),
                dict(scaling=dict(kind="other")), dict(scaling=dict(kind="yarn", factor=2.0)),
                dict(scaling=dict(kind="linear", factor=0.0)), dict(scaling=dict(kind="linear", factor=2.0, original=1)),
                dict(turning=[float("inf")] * 32), dict(scaling=dict(kind="linear", factor=2.0), turning=[1.0] * 32)):
        with pytest.raises(ValueError):
            q8mv.Rotary(64, **bad)
    for args in ((x[0], at), (x[..., :32], at), (x, at[:2])):
        with pytest.raises(ValueError):
            rotary(*args)
    for args in ((x.double(), at), (x, at.int())):
        with pytest.raises(TypeError):
            rotary(*args)
    with pytest.raises(ValueError):
        rotary(x, at, out=x[:1].expand(3, 2, 64))
    cache = q8mv.Cache4(2, 16, 2, 64)
    with pytest.raises(ValueError):
        rotary.write(cache, x, x, x[:2], at, at)
    with pytest.raises(ValueError):
        rotary.write(cache, x.half(), x, x, at, at)
    with pytest.raises(TypeError):
        rotary.write(x, x, x, x, at, at)
    with pytest.raises(q8mv.Q8mvError):
        q8mv.Rotary(128).write(cache, None, x, x, at, at)
    assert rotary(x[:0], at[:0]).shape == (0, 2, 64)
