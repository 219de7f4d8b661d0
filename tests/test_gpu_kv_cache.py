"""Writing, reading and moving rows of the Q8_0 cache, bit for bit against the recipe in numpy."""
import numpy as np
import pytest

import kv_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def to_gpu(x, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(getattr(torch, dtype))


def as_f32(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("heads,dim,page,layout", [(1, 16, 1, "head"), (2, 80, 7, "token"), (8, 128, 16, "head"),
                                                   (3, 96, 24, "token"), (5, 256, 64, "head"), (33, 48, 5, "token")])
@pytest.mark.parametrize("n", [1, 3, 130])
def test_write_and_read_back(q8mv, dtype, heads, dim, page, layout, n):
    import torch

    rng = np.random.default_rng(n * 1000 + dim)
    pages = -(-n // page) + 2
    cache = q8mv.Cache(pages, page, heads, dim, layout=layout)
    x = rng.standard_normal((2, n, heads, dim)).astype(np.float32) * np.exp(2 * rng.standard_normal((2, n, heads, 1))).astype(np.float32)
    x[0, 0, 0, :] = 0  # a block of zeros
    k, v = to_gpu(x[0], dtype), to_gpu(x[1], dtype)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    cache.write(k, v, torch.from_numpy(slots).cuda())
    for t, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        c, d = ref.quantise(as_f32(t))
        got_c, got_d = codes.cpu().numpy(), scales.cpu().numpy()
        assert np.array_equal(got_c[slots // page, :, slots % page], c)
        assert np.array_equal(got_d[slots // page, :, slots % page], d)
        other = np.setdiff1d(np.arange(pages * page), slots)  # nothing else was touched
        assert not got_c[other // page, :, other % page].any() and not got_d[other // page, :, other % page].any()
    for out_type in ref.TYPES:
        got = cache.read(torch.from_numpy(slots).cuda(), dtype=getattr(torch, out_type))
        for t, g in zip((k, v), got):
            c, d = ref.quantise(as_f32(t))
            want = c.astype(np.float32) * np.repeat(d, 32, -1)[..., :dim]
            assert torch.equal(g.cpu(), torch.from_numpy(want).to(getattr(torch, out_type)))


def test_slots_outside_are_skipped_and_read_as_zeros(q8mv):
    import torch

    cache = q8mv.Cache(2, 4, 2, 32)
    k = torch.randn(5, 2, 32, device="cuda")
    slots = torch.tensor([3, -1, 8, 2 ** 40, 7], device="cuda")
    cache.write(k, 2 * k, slots)
    assert int((cache.k_scales != 0).sum()) == 4  # two tokens, two heads
    a, b = cache.read(slots)
    assert not a[1:4].any() and not b[1:4].any()
    assert (a[0] - k[0]).abs().max() <= 0.5 * k[0].abs().max() / 127 * 1.001
    assert (b[4] - 2 * k[4]).abs().max() <= k[4].abs().max() / 127 * 1.001


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strides_and_alignment_of_inputs(q8mv, dtype, offset):
    """k and v as views of one fused projection, at any element offset."""
    import torch

    n, heads, dim = 9, 3, 64
    buf = torch.randn(n * 700 + 8, device="cuda").to(getattr(torch, dtype))
    k = torch.as_strided(buf, (n, heads, dim), (700, dim + offset, 1), offset)
    v = torch.as_strided(buf, (n, heads, dim), (700, dim, 1), 3 * dim + 16 + offset)
    one, two = q8mv.Cache(3, 4, heads, dim), q8mv.Cache(3, 4, heads, dim)
    slots = torch.arange(n, device="cuda")
    one.write(k, v, slots)
    two.write(k.contiguous(), v.contiguous(), slots)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(two, name))
    # one row for every head: a stride of 0
    one.write(k[:, :1].expand(n, heads, dim), v, slots)
    assert torch.equal(one.k_codes[:, 0], one.k_codes[:, 2])


def test_values_that_are_not_finite(q8mv):
    import torch

    cache = q8mv.Cache(1, 4, 1, 64)
    k = torch.ones(4, 1, 64, device="cuda")
    k[0, 0, 3] = float("nan")
    k[1, 0, 40] = float("inf")
    k[2, 0, :32] = 1e-39  # 127 / amax overflows
    k[3, 0, 0] = 3.0e38
    cache.write(k, k, torch.arange(4, device="cuda"))
    c, d = ref.quantise(k.cpu().numpy())
    assert np.array_equal(cache.k_codes.cpu().numpy()[0, 0], c[:, 0])
    assert np.array_equal(cache.k_scales.cpu().numpy()[0, 0], d[:, 0])
    back = cache.read(torch.arange(4, device="cuda"))[0].cpu().numpy()[:, 0]
    assert back[0, 3] == 0 and np.all(back[0, :3] == 1)
    assert np.isnan(back[1, 32:]).all() and np.all(back[1, :32] == 1)
    assert np.isfinite(back[2:]).all()


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("dim,heads", [(128, 8), (80, 3), (16, 70)])
@pytest.mark.parametrize("path", [1, 4, 9, 20])
def test_move_in_order(q8mv, layout, dim, heads, path):
    """Paths that move up over themselves, padding, several requests."""
    import torch

    rng = np.random.default_rng(path * dim)
    page, batch = 8, 5
    span = 3 * path + 4
    host = ref.Host(rng, -(-batch * span // page), page, heads, dim, layout)
    cache = host.device(q8mv)
    src = np.full((batch, path), -1, np.int64)
    dst = np.full((batch, path), -1, np.int64)
    for b in range(batch):
        n = path if b % 2 == 0 else rng.integers(0, path + 1)
        nodes = np.sort(rng.permutation(span)[:n])
        src[b, :n] = b * span + nodes
        dst[b, :n] = b * span + np.arange(n)
    if path > 3:
        src[0] = [b0 % span for b0 in range(1, path + 1)]  # every source is the next destination
        dst[0] = range(path)
        src[2, 1] = 2 ** 35  # outside: the pair is skipped
        dst[4, 2] = -7
    cache.move(torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    slots = host.kc.shape[0] * page
    for b in range(batch):
        for s, d in zip(src[b], dst[b]):
            if 0 <= s < slots and 0 <= d < slots:
                for a in (host.kc, host.ks, host.vc, host.vs):
                    a[d // page, :, d % page] = a[s // page, :, s % page]
    for a, name in ((host.kc, "k_codes"), (host.ks, "k_scales"), (host.vc, "v_codes"), (host.vs, "v_scales")):
        assert np.array_equal(getattr(cache, name).cpu().numpy(), a), name


def test_chained_moves_backwards(q8mv):
    """A later pair reads what an earlier one wrote."""
    import torch

    rng = np.random.default_rng(3)
    host = ref.Host(rng, 4, 4, 2, 32)
    cache = host.device(q8mv)
    cache.move(torch.tensor([0, 5, 6, 7], device="cuda"), torch.tensor([5, 6, 7, 8], device="cuda"))
    k, _ = cache.read(torch.tensor([0, 5, 6, 7, 8], device="cuda"))
    for i in range(1, 5):
        assert torch.equal(k[0], k[i])


def test_empty_calls(q8mv):
    import torch

    cache = q8mv.Cache(1, 1, 1, 16)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    cache.write(torch.empty(0, 1, 16, device="cuda"), torch.empty(0, 1, 16, device="cuda"), none)
    k, v = cache.read(none)
    assert k.shape == (0, 1, 16) and v.shape == (0, 1, 16)
    cache.move(none.view(0, 0), none.view(0, 0))


def test_other_stream(q8mv):
    import torch

    cache = q8mv.Cache(64, 16, 8, 128)
    k = torch.randn(1000, 8, 128, device="cuda")
    slots = torch.randperm(1024, device="cuda")[:1000].contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cache.write(k, k, slots)
        a, b = cache.read(slots)
    s.synchronize()
    assert torch.equal(a, b) and (a - k).abs().max() <= k.abs().max() / 127


def test_refusals(q8mv):
    import torch

    cache = q8mv.Cache(2, 4, 2, 32)
    k = torch.zeros(3, 2, 32, device="cuda")
    slots = torch.arange(3, device="cuda")
    with pytest.raises(TypeError):
        cache.write(k.double(), k.double(), slots)
    with pytest.raises(TypeError):
        cache.write(k, k, slots.int())
    with pytest.raises(ValueError):
        cache.write(k, k[:2], slots)
    with pytest.raises(ValueError):
        cache.write(k, k.half(), slots)
    with pytest.raises(ValueError):
        cache.write(k.transpose(1, 2), k, slots)
    with pytest.raises(ValueError):
        cache.write(k, k, slots[:2])
    with pytest.raises(ValueError):
        cache.write(k.cpu(), k, slots)
    with pytest.raises(ValueError):
        cache.write(k, k, slots.cpu())
    with pytest.raises(ValueError):
        cache.read(torch.arange(6, device="cuda")[::2])
    with pytest.raises(TypeError):
        cache.read(slots, dtype=torch.float64)
    with pytest.raises(ValueError):
        cache.read(slots, out=(k[:2].clone(), k[:2].clone()))
    with pytest.raises(ValueError):
        cache.move(slots, slots[:2])
    with pytest.raises(ValueError):
        q8mv.Cache(2, 4, 2, 40)
    codes, scales = torch.zeros(2, 2, 4, 32, dtype=torch.int8, device="cuda"), torch.zeros(2, 2, 4, 1, device="cuda")
    with pytest.raises(TypeError):
        q8mv.Cache.of(codes, scales.half(), codes, scales)
    with pytest.raises(ValueError):
        q8mv.Cache.of(codes, scales[..., :0], codes, scales)
    with pytest.raises(ValueError):
        q8mv.Cache.of(codes.expand(2, 2, 4, 32)[:, :1].expand(2, 2, 4, 32), scales, codes, scales)
