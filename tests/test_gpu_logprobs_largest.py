"""Logits of +inf beside FP32's largest finite number: the infinite ones share the row, the finite ones have nothing,
wherever they stand (before an infinite one of the same thread, behind it, in other threads and CTAs)."""
import math

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


@pytest.mark.parametrize("T,V", [(8, 5003), (8, 40000), (320, 2100)])
def test_the_largest_finite_logit_beside_infinite_ones(T, V):
    t = torch()
    top = float(np.finfo(np.float32).max)
    x = np.random.default_rng(V).normal(size=(T, V))
    x[0, [0, 1, 2, 3]] = math.inf, top, top, 1.0             # one chunk
    x[1, [0, V - 1]] = top, math.inf
    x[2] = top
    x[2, V // 2] = math.inf
    x[3, :V // 2] = math.inf
    x[3, V // 2:] = top
    x[4, [7, 900]] = top, top                                # no infinite one
    x[5] = top
    x[6, 2::3] = math.inf
    x[6, ::3] = top
    x[6, 1::3] = -top
    x[7, 5], x[7, 6], x[7, 2000] = math.inf, math.nan, top
    xd, f = to_dev(x, True)
    tok = np.tile(np.array([0, 1, V // 2, V - 1], dtype=np.int32), (T, 1))
    check(q4lin.token_logprobs(xd, t.from_numpy(tok).cuda(), 6), f, tok, 6)
