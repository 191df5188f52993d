"""Prompts with scores of -inf: a key whose weight is exactly 0 leaves finite values alone, and 0 times a value that is not
finite is NaN, as the definition has it; a row of which every score is -inf is NaN.  Blocks on the diagonal, where such values
are put in by the rows themselves, and blocks before it."""
import numpy as np
import pytest

from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch, x_to_dev, y_bits
from test_gpu_prompt_attention import bits, check

pytestmark = pytest.mark.gpu

INF, NINF, NAN = 0x7F80, 0xFF80, 0x7FC0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def run(q, k, v, cu):
    out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), torch().tensor(cu, dtype=torch().int32, device="cuda"))
    with np.errstate(invalid="ignore"):
        check(y_bits(out), q, k, v, cu)


@pytest.mark.parametrize("Hq,Hk,D", [(2, 1, 64), (3, 1, 128), (4, 4, 40)])
@pytest.mark.parametrize("lens", [[1], [1, 1, 2], [200, 130], [300]])
@pytest.mark.parametrize("value", [INF, NINF, NAN])
def test_weights_of_zero_meet_values_that_are_not_finite(lens, Hq, Hk, D, value):
    """q's first values are positive, so k's -inf there makes the score -inf."""
    T, cu = sum(lens), np.cumsum([0] + lens)
    q, k, v = bits((T, Hq, D), 1), bits((T, Hk, D), 2), bits((T, Hk, D), 3)
    q[..., 0] &= 0x7FFF
    q[..., 0] |= 0x0080                  # (not zero)
    for a, n in zip(cu, lens):
        for t in {0, n // 3, n // 2, n - 1}:
            k[a + t, :, 0] = NINF
            v[a + t, 0, 3], v[a + t, -1, D - 1] = value, value
        if n > 6:
            v[a + n // 5, 0, 7] = value      # one with a weight
    run(q, k, v, cu)


@pytest.mark.parametrize("lens", [[1], [3, 140], [260]])
def test_rows_without_any_weight_are_nan(lens):
    """Every key's score is -inf; some values are infinite."""
    T, cu = sum(lens), np.cumsum([0] + lens)
    q, k, v = bits((T, 2, 64), 1), bits((T, 1, 64), 2), bits((T, 1, 64), 3)
    q[..., 0] = 0x3F80
    k[..., 0] = NINF
    v[::3, 0, 5] = INF
    v[1::4, 0, 9] = NINF
    out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), torch().tensor(cu, dtype=torch().int32, device="cuda"))
    assert out.isnan().all()
    run(q, k, v, cu)
