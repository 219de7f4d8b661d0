"""Caches over existing tensors: which strides are taken, and what they reach."""
import numpy as np
import pytest

import kv_ref as ref
from test_gpu_kv_attend import q8mv  # noqa: F401

pytestmark = pytest.mark.gpu


def parts(shape, dim=128):
    import torch

    return [torch.zeros(*shape, n, dtype=t, device="cuda")
            for n, t in ((dim, torch.int8), (-(-dim // 32), torch.float32)) * 2]


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_an_expanded_axis_is_refused(q8mv, axis):  # noqa: F811
    """One row that stands for eight: they would be eight places of memory that has one."""
    shape = [1, 1, 1]
    shape[axis] = 8
    with pytest.raises(ValueError):
        q8mv.Cache.of(*(t.expand(*shape, t.shape[3]) for t in parts([1, 1, 1])))
    # beside axes that are whole
    whole = [3, 3, 3]
    whole[axis] = 1
    shape = [n if n > 1 else 8 for n in whole]
    with pytest.raises(ValueError):
        q8mv.Cache.of(*(t.expand(*shape, t.shape[3]) for t in parts(whole)))
    q8mv.Cache.of(*parts([1, 1, 1]))
    q8mv.Cache.of(*parts(whole))
