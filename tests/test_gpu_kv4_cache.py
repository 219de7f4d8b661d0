"""Writing, reading, moving and copying rows of the Q4_0 cache: bytes and scales as the header defines them."""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def to(x, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(getattr(torch, dtype))


def host(t):
    return t.detach().float().cpu().numpy()


def check(cache, slots, codes, scales, dim, page):
    """The cache's rows at slots hold these bytes and scales (keys, values)."""
    nb = ref.blocks4(dim)
    at, place = slots // page, slots % page
    for i, (got_c, got_s) in enumerate(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))):
        assert np.array_equal(got_c.cpu().numpy()[at, :, place], ref.pack(codes[i], 2 if i else 4))
        assert np.array_equal(got_s.cpu().numpy()[at, :, place][..., :nb].view(np.uint16) & 0x7FFF,
                              scales[i].view(np.uint16) & 0x7FFF)  # (the sign of a zero says nothing)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 160, 192, 256])
@pytest.mark.parametrize("n,heads,page,layout", [(1, 1, 16, "head"), (37, 3, 7, "token"), (700, 8, 16, "head")])
def test_write_and_read_are_the_formulas(q8mv, dtype, dim, n, heads, page, layout):
    import torch

    rng = np.random.default_rng(dim + n)
    pages = -(-n // page) + 3
    cache = q8mv.Cache4(pages, page, heads, dim, layout=layout)
    k, v = (to(rng.standard_normal((n, heads, dim)).astype(np.float32) * np.exp(rng.standard_normal(dim)).astype(np.float32),
               dtype) for _ in range(2))
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    skip = rng.random(n) < 0.1
    given = torch.from_numpy(np.where(skip, rng.choice([-1, pages * page, 2 ** 40], n), slots)).cuda()
    cache.write(k, v, given)
    quant = [ref.quantise(host(x)) for x in (k, v)]
    live = ~skip
    check(cache, slots[live], [c[live] for c, _ in quant], [d[live] for _, d in quant], dim, page)
    for out in ("float32", "float16", "bfloat16"):
        got = cache.read(given, dtype=getattr(torch, out))
        for x, (c, d) in zip(got, quant):
            want = torch.from_numpy(ref.values(c, d, dim).astype(np.float32)).to(getattr(torch, out)).float().numpy()
            want[skip] = 0
            assert np.array_equal(host(x), want)
    # rows that no slot names are as they were
    rest = np.setdiff1d(np.arange(pages * page), slots[live])
    assert not cache.k_codes.cpu().numpy()[rest // page, :, rest % page].any()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_unusual_blocks(q8mv, dtype):
    import torch

    big = 3.0e38 if dtype == "float32" else 1e38
    row = np.zeros((14, 64), np.float32)
    row[1, 5] = np.nan
    row[2, :40] = np.nan
    row[3, 7] = np.inf
    row[4, 7], row[4, 8] = -np.inf, np.nan
    row[5, 3], row[5, 40] = 524160.0, 524032.0  # the first d that leaves f16, and one below
    row[6] = np.linspace(-1, 1, 64) * 2.0 ** -21  # d subnormal, and rounded to half of it or to 0
    row[7] = np.linspace(-1, 1, 64) * 2.0 ** -23
    row[8, 0], row[8, 1], row[8, 2] = 3.0, -3.0, 1.5  # two alike: the positive one is the top
    row[9, 33] = big
    row[10] = -np.arange(64)
    row[11] = 0.1 * np.arange(64)
    row[12] = np.float32(1.17e-38) * np.linspace(-1, 1, 64)
    row[13, :8] = [8, 7.5, 7.4999, -7.5, 0.5, -0.5, 1.5, -1.5]
    x = to(row[:, None], dtype)
    cache = q8mv.Cache4(1, 16, 1, 64)
    slots = np.arange(14)
    cache.write(x, x, torch.from_numpy(slots).cuda())
    c, d = ref.quantise(host(x))
    check(cache, slots, [c, c], [d, d], 64, 16)
    got = host(cache.read(torch.from_numpy(slots).cuda())[0])[:, 0]
    want = ref.values(c, d, 64)[:, 0]
    bad = ~np.isfinite(want)
    # (524032 is 2^19 in bf16's 8 bits, whose eighth, 65536, leaves f16 as well)
    assert np.array_equal(np.isnan(got), bad) and bad[3, :32].all() and bad[5, :32].all()
    assert bad[5, 32:].any() == (dtype == "bfloat16")
    assert np.array_equal(got[~bad], want[~bad].astype(np.float32))


def test_inputs_at_odd_places(q8mv):
    """Strides and alignments that no 16-byte load can take."""
    import torch

    rng = np.random.default_rng(3)
    for dtype in ("float32", "bfloat16"):
        base = to(rng.standard_normal((9, 5 * 80 + 3)).astype(np.float32), dtype)
        k = base[:, 1:1 + 2 * 80].view(9, 2, 80)
        v = base[:, 2 * 80 + 3:2 * 80 + 3 + 160].unflatten(1, (2, 80))
        cache = q8mv.Cache4(2, 8, 2, 80)
        slots = rng.permutation(16)[:9]
        cache.write(k, v, torch.from_numpy(slots).cuda())
        quant = [ref.quantise(host(x)) for x in (k, v)]
        check(cache, slots, [c for c, _ in quant], [d for _, d in quant], 80, 8)


@pytest.mark.parametrize("dim,layout", [(64, "head"), (80, "token"), (128, "head"), (192, "token"), (256, "head")])
def test_move_keeps_the_order_of_a_request(q8mv, dim, layout):
    import torch

    rng = np.random.default_rng(dim)
    h = ref.Host(rng, 6, 8, 3, dim, layout)
    cache = h.device(q8mv)
    src = np.array([[1, 2, 9, 20], [30, 31, -1, 47]])
    dst = np.array([[0, 1, 2, 48], [40, 30, 41, 31]])
    codes, scales = cache.k_codes.clone(), cache.v_scales.clone()
    cache.move(torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    for b in range(2):
        for s, t in zip(src[b], dst[b]):
            if 0 <= s < 48 and 0 <= t < 48:
                codes[t // 8, :, t % 8] = codes[s // 8, :, s % 8]
                scales[t // 8, :, t % 8] = scales[s // 8, :, s % 8]
    assert torch.equal(cache.k_codes, codes) and torch.equal(cache.v_scales.view(torch.int16), scales.view(torch.int16))


def orders(q8mv, four, dim, pages, heads, page, order):
    """A cache with random contents whose axes lie in this order in memory."""
    import torch

    g = torch.Generator("cuda").manual_seed(dim)
    parts = []
    if four:
        kinds = ((16 * ref.blocks4(dim), torch.uint8), (ref.columns4(dim), torch.float16))
    else:
        kinds = ((dim, torch.int8), (-(-dim // 32), torch.float32))
    shape = (pages, heads, page)
    back = [order.index(i) for i in range(3)]
    for _ in range(2):
        for width, dtype in kinds:
            t = torch.randint(-100, 100, (*(shape[i] for i in order), width), generator=g, device="cuda")
            t = (t.to(torch.uint8) if dtype == torch.uint8 else t.to(dtype))
            parts.append(t.permute(*back, 3))
    return q8mv.Cache4.of(*parts, dim) if four else q8mv.Cache.of(*parts)


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 192])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 5), (8, 16), (2, 1), (40, 64)])
@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (1, 0, 2), (2, 1, 0)])
def test_copies_of_pages(q8mv, four, dim, heads, page, order):
    import torch

    cache = orders(q8mv, four, dim, 12, heads, page, order)
    parts = (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)
    src = torch.tensor([1, 1, -1, 3, 12, 7, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    dst = torch.tensor([0, 4, 2, -1, 8, 9, 12, 10], dtype=torch.int32, device="cuda")
    for count in (None, 1, 0, 100, -3):
        want = [p.clone() for p in parts]
        n = len(src) if count is None else min(max(count, 0), len(src))
        for s, t in zip(src.tolist()[:n], dst.tolist()[:n]):
            if 0 <= s < 12 and 0 <= t < 12:
                for w in want:
                    w[t] = w[s]
        cache.copy_pages(src, dst, None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda"))
        for p, w in zip(parts, want):
            assert torch.equal(p, w)
        for p in parts:  # others, for the next count
            p.add_(1)


def test_many_copies(q8mv):
    """More chunks than blocks, and a list that is mostly empty."""
    import torch

    cache = orders(q8mv, True, 128, 3000, 8, 16, (0, 1, 2))
    src = torch.full((1500,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    order = torch.randperm(3000, generator=torch.Generator().manual_seed(1)).int().cuda()
    src[:1400], dst[:1400] = order[:1400], order[1500:2900]
    want = cache.v_codes.clone()
    want[dst[:1400].long()] = want[src[:1400].long()]
    cache.copy_pages(src, dst)
    assert torch.equal(cache.v_codes, want)


def test_offsets_past_32_bits(q8mv):
    """A cache of 2^32 bytes of codes and more: its last pages are written, read, attended, moved and copied."""
    import torch

    pages, page, heads, dim = 70000, 128, 8, 128  # 71.7 million rows of 64 bytes
    cache = q8mv.Cache4(pages, page, heads, dim)
    assert cache.k_codes.numel() > 2 ** 32
    g = torch.Generator("cuda").manual_seed(3)
    n = 3 * page
    k, v = (torch.randn(n, heads, dim, generator=g, device="cuda") for _ in range(2))
    last = torch.arange((pages - 3) * page, pages * page, device="cuda")
    first = torch.arange(n, device="cuda")
    small = q8mv.Cache4(3, page, heads, dim)
    for c, slots in ((cache, last), (small, first)):
        c.write(k, v, slots)
    for a, b in zip(cache.read(last), small.read(first)):
        assert torch.equal(a, b)
    q = torch.randn(1, 32, dim, generator=g, device="cuda")
    attend = q8mv.TreeAttention4(32, heads, dim, 1, 1)
    lengths = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    tables = [torch.arange(x, x + 3, dtype=torch.int32, device="cuda").view(1, 3) for x in (pages - 3, 0)]
    assert torch.equal(attend(q, cache, tables[0], lengths), attend(q, small, tables[1], lengths))
    assert not cache.k_codes[:pages - 3].any()  # nothing went anywhere else
    cache.copy_pages(tables[0].view(-1), tables[1].view(-1))
    assert torch.equal(cache.v_codes[:3], small.v_codes)
    cache.move(last[:5].clone(), torch.arange(5, device="cuda") + 10 * page)
    assert torch.equal(cache.read(torch.arange(5, device="cuda") + 10 * page)[1], small.read(first[:5].clone())[1])
    rotary = q8mv.Rotary(dim)
    for c, slots in ((cache, last), (small, first)):
        rotary.write(c, None, k, v, first, slots)
    for a, b in zip(cache.read(last), small.read(first)):
        assert torch.equal(a, b)
