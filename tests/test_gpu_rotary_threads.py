"""One ``Rotary`` of several threads, each with a cache of its own."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["Cache", "Cache4"])
def test_threads_write_to_their_own_slots(kind):
    import torch

    import q8_matrix_vector_gb300 as q8mv

    heads, dim, pages, page, n, many = 2, 64, 4, 16, 7, 400
    rng = np.random.default_rng(0)
    rotary = q8mv.Rotary(dim)
    work = []
    for t in range(4):
        q, k, v = (torch.from_numpy(rng.standard_normal((n, h, dim)).astype(np.float32)).cuda() for h in (4, heads, heads))
        work.append((q, k, v, torch.from_numpy(rng.integers(0, 10000, n)).cuda(),
                     torch.from_numpy(rng.permutation(pages * page)[:n]).cuda()))
    alone = [getattr(q8mv, kind)(pages, page, heads, dim) for _ in work]
    turned = [rotary.write(c, *w) for c, w in zip(alone, work)]
    caches = [getattr(q8mv, kind)(pages, page, heads, dim) for _ in work]
    torch.cuda.synchronize()
    outs, go = [None] * len(work), threading.Barrier(len(work), timeout=60)

    def serve(i):
        stream = torch.cuda.Stream()
        go.wait()
        with torch.cuda.stream(stream):
            for _ in range(many):
                outs[i] = rotary.write(caches[i], *work[i])
        stream.synchronize()

    threads = [threading.Thread(target=serve, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(len(work)):
        assert torch.equal(outs[i], turned[i])
        for part in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(caches[i], part), getattr(alone[i], part)), (i, part)
