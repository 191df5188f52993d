"""Top tokens among logits that are zeros of both signs: they are equal, so the lowest token comes first, whichever threads, warps
and CTAs of a row's cluster hold them."""
import numpy as np
import pytest

from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch
from test_gpu_logprobs import check, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    yield
    assert q4lin.device_status() == 0


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,V,k", [(6, 700, 12), (6, 9001, 5), (6, 40000, 32), (320, 3001, 4)])
def test_zeros_of_both_signs_stand_in_the_order_of_their_tokens(T, V, k, fp32):
    t = torch()
    rng = np.random.default_rng(V + k)
    x = -rng.integers(1, 9, (T, V)).astype(np.float64)
    x[0] = 0.0
    x[0, ::2] = -0.0                                          # a whole row of them
    x[1] = -0.0
    x[1, V // 2:] = 0.0                                       # the first half is all -0
    x[2, rng.choice(V, 3, replace=False)] = -0.0              # fewer than there are places
    x[2, rng.choice(V, 2, replace=False)] = 0.0
    x[3, rng.choice(V, 60, replace=False)] = np.where(rng.random(60) < 0.5, 0.0, -0.0)
    x[4, 8 * rng.choice(V // 8, 40, replace=False)] = np.where(rng.random(40) < 0.5, 0.0, -0.0)
    x[4, rng.choice(V, 2, replace=False)] = 1.0               # something above them
    for r in range(5, T):
        x[r, rng.choice(V, 50, replace=False)] = np.where(rng.random(50) < 0.5, 0.0, -0.0)
    xd, f = to_dev(x, fp32)
    assert (np.signbit(f) & (f == 0)).any()
    tok = np.zeros((T, 1), dtype=np.int32)
    check(q4lin.token_logprobs(xd, t.from_numpy(tok).cuda(), k), f, tok, k)
