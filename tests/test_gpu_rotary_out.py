"""Where the output of a rotation may lie: refused where it overlaps what is read, taken between the parts of one tensor."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

N, HEADS, KV, DIM = 37, 8, 2, 64


@pytest.fixture(scope="module")
def q8mv():
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


def make(shape, seed=0):
    import torch

    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda().bfloat16()


def positions():
    import torch

    return torch.arange(N, device="cuda") * 3


def test_apply_refuses_what_overlaps(q8mv):
    import torch

    rotary = q8mv.Rotary(DIM)
    buffer, at = make((N + 1, HEADS + 1, DIM)), positions()
    x = buffer[:N, :HEADS]
    before = buffer.clone()
    for out in (buffer[1:, :HEADS], buffer[:N, 1:], torch.as_strided(buffer, x.shape, (DIM * HEADS, DIM, 1)),
                torch.as_strided(buffer, x.shape, x.stride(), 2),  # an element further
                torch.as_strided(make((N * HEADS + N, DIM)), x.shape, (DIM, DIM, 1)),  # its own rows
                torch.as_strided(make((N * HEADS, DIM)), x.shape, (DIM * HEADS // 2, DIM, 1))):
        with pytest.raises(q8mv.Q8mvError):
            rotary(x, at, out=out)
    # the positions, in the output's first heads
    out = torch.zeros(N, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
    inside = out.view(-1)[:4 * N].view(torch.int64)
    with pytest.raises(q8mv.Q8mvError):
        rotary(x, inside, out=out)
    assert torch.equal(buffer, before)
    # what is apart is taken: other heads, other rows and itself
    want = rotary(x[:, :4].contiguous(), at)
    assert torch.equal(rotary(x[:, :4], at, out=buffer[:N, 4:8]), want)
    wide = make((N, HEADS, 2, DIM))
    want = rotary(wide[:, :, 0].contiguous(), at)
    assert torch.equal(rotary(wide[:, :, 0], at, out=wide[:, :, 1]), want)
    assert torch.equal(rotary(wide[:, :, 0], at, out=wide[:, :, 0]), want)
    one = make((1, HEADS, DIM)).expand(N, HEADS, DIM)
    assert torch.equal(rotary(one, at, out=make((N, HEADS, DIM))), rotary(one.contiguous(), at))


@pytest.mark.parametrize("kind", ["Cache", "Cache4"])
def test_write_refuses_what_overlaps(q8mv, kind):
    import torch

    rotary, cache = q8mv.Rotary(DIM), getattr(q8mv, kind)(4, 16, KV, DIM)
    slots, at = torch.arange(N, device="cuda"), positions()
    qkv = make((N, HEADS + 2 * KV, DIM), 1)
    q, k, v = qkv.split((HEADS, KV, KV), 1)
    before = qkv.clone()
    for out in (qkv[:, KV:KV + HEADS], qkv[:, 2 * KV:], torch.as_strided(qkv, q.shape, q.stride(), 2)):
        with pytest.raises(q8mv.Q8mvError):
            rotary.write(cache, q, k, v, at, slots, out=out)
    with pytest.raises(q8mv.Q8mvError):
        rotary.write(cache, make(q.shape), k, v, at, slots, out=qkv[:, 1:1 + HEADS + KV][:, -HEADS:])
    assert torch.equal(qkv, before) and not cache.k_codes.any() | cache.v_scales.any()
    # in place between k and v of the same tensor, as a separate output gives it
    want = rotary.write(cache, q, k, v, at, slots)
    codes = cache.k_codes.clone()
    other = getattr(q8mv, kind)(4, 16, KV, DIM)
    assert rotary.write(other, q, k, v, at, slots, out=q) is q
    assert torch.equal(q, want) and torch.equal(other.k_codes, codes)
    assert torch.equal(qkv[:, HEADS:], before[:, HEADS:])
