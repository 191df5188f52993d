"""Entropies of rows that are nearly certain of one token: never below zero, and as small as they are.

Bound where the other tokens' sum d = V e^-margin is below 2^-25: S is exactly 1 in FP32 whatever the order, so ln S,
which is d, comes out as 0 (off by d), and the other term is a sum of products of one sign: V / 128 + 64 roundings,
the exponential's 2^-22 and its argument's (2^-23 of up to 60 / ln 2: 2^-16) together below 2^-15 of it.  The
entropy there is taken from its closed form, ln(1 + d) + margin d / (1 + d) with d = (V - 1) e^-margin: the oracle's S
is a sum next to 1 in FP64, a multiple of 2^-52, which is 6e-3 of a d of 4e-14."""
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


def rows(V, margins):
    """A row per margin: zeros and one larger logit, now in a thread's first chunk, mostly far behind it."""
    x = np.zeros((len(margins), V))
    for r, m in enumerate(margins):
        x[r, (r * 7919 + V // 3) % V] = m
    return x


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("copies,V", [(1, 5003), (1, 40000), (20, 40000)])
def test_nearly_certain_rows(copies, V, fp32):
    t = torch()
    margins = [30.0, 32.5, 35.0, 38.0, 39.5, 39.875, 40.0, 40.25, 44.0, 50.0, 60.0, 34.0, 36.0, 37.0, 39.0, 39.25]
    one = rows(V, margins)
    x, f = to_dev(np.tile(one, (copies, 1)), fp32)
    tok = t.zeros((len(x), 1), dtype=t.int32, device="cuda")
    got = q4lin.token_logprobs(x, tok, 0)[1].cpu().numpy().astype(np.float64)
    margin = f[:len(margins)].max(axis=1)      # (as rounded to the logits' type)
    d = (V - 1) * np.exp(-margin)
    want = np.log1p(d) + margin * d / (1 + d)
    assert (d < 2.0 ** -25).all()
    for c in range(copies):
        e = got[c * len(margins):(c + 1) * len(margins)]
        assert (e >= 0).all(), e.min()
        assert (np.abs(e - want) <= d + 2.0 ** -15 * want).all(), np.max(np.abs(e - want) / want)


@pytest.mark.parametrize("fp32", [False, True])
def test_margins_of_every_size(fp32):
    t = torch()
    margins = np.arange(0, 64, 0.5)
    for V in (3, 64, 1000, 30011):
        x, f = to_dev(rows(V, margins), fp32)
        tok = np.zeros((len(margins), 1), dtype=np.int32)
        got = q4lin.token_logprobs(x, t.from_numpy(tok).cuda(), 1)
        assert (got[1] >= 0).all(), float(got[1].min())
        check(got, f, tok, 1)
