"""Queries near the ends of bf16's range with scales that bring the scores back: powers of two on the way in and out."""
import numpy as np
import pytest

from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin, synth

import oracle
from gpu_util import x_to_dev, y_bits
from test_gpu_kv4 import bits, check, dev, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


@pytest.mark.parametrize("n,Hq,Hk,D", [(1, 4, 2, 64), (1, 4, 1, 96), (2, 8, 1, 128)])
@pytest.mark.parametrize("size,same_sign", [(100, False), (118, False), (122, True), (124, False), (125, True), (-100, False), (-124, True)])
def test_large_and_small_queries(n, Hq, Hk, D, size, same_sign):
    """q of about 2^size (all of one sign: their sum leaves FP32's range), the scale 2^-size D^-1/2."""
    lengths = [300, 64, 1]
    cache, table = filled(3, lengths, 6, Hk, D, n + D)
    f = oracle.bf16_bits_to_f64(bits((3 * n, Hq, D), D + n, 0.5))
    q = synth.to_bf16_bits(np.ldexp(np.abs(f) if same_sign else f, size))
    assert np.isfinite(oracle.bf16_bits_to_f64(q)).all()
    scale = float(np.float32(2.0 ** -size * D ** -0.5))
    got = q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32)), scale=scale)
    check(y_bits(got), q, cache, table, lengths, D, scale)
