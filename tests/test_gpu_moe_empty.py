"""The expert layer with an empty dimension: the workspace query says 0 bytes, and a pointer that
is passed all the same is left alone."""
import numpy as np
import pytest

from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch, x_to_dev
from test_gpu_moe import _lib, bits  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,F", [(1, 0, 64), (5, 0, 64), (64, 0, 0), (3, 64, 0)])
def test_no_workspace_is_written(T, H, F):
    t = torch()
    E, k = 4, 2
    assert q4lin.moe_workspace_bytes(T, H, F, E, k) == 0
    around = t.full((1 << 16,), 0xA5, dtype=t.uint8, device="cuda")
    x, w = x_to_dev(bits((T, 64), 1, 1.0)), x_to_dev(bits((E, 64), 2, 1.0))
    bias = t.tensor([0.0, 2.0, 1.0, -1.0], device="cuda")
    ids, p = t.empty((T, k), dtype=t.int32, device="cuda"), t.empty((T, k), device="cuda")
    y = t.ones((T, 64), dtype=t.bfloat16, device="cuda")
    planes = t.zeros(4096, dtype=t.uint8, device="cuda").data_ptr()
    st = q4lin.load().q4lin_moe(x.data_ptr(), w.data_ptr(), bias.data_ptr(), planes, planes, planes, planes, ids.data_ptr(),
                                p.data_ptr(), y.data_ptr(), T, H, F, E, k, 1, around.data_ptr() + (1 << 15), None)
    t.cuda.synchronize()
    assert st == 0 and bool((around == 0xA5).all())
    if H == 0:   # logits are the bias
        assert (ids.cpu().numpy() == np.array([1, 2])).all() and bool((y == 1).all())
    else:
        assert bool((y == 0).all())
