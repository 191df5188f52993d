"""What the expert layer loses between its two products.  The intermediate h holds 32 bits in the
definition's plain form; the products' operands must not take it to fewer than FP32 sums lose anyway.

y is rounded to bf16, so the loss is looked for where that rounding is small: outputs of at most
1/256 of their token's rms(y), whose half step is at most 2^-8 2^-9 = 8e-6 rms.  An h rounded once to
11 bits puts errors of 2^-11 / sqrt(12) = 1.4e-4 (at the low end of a binade; 1e-4 over it) of rms(y)
into y; two terms put 2^-22 there, and FP32 sums of a few thousand terms of random sign some 2^-24
sqrt(n) = 2e-6 to 6e-6.  Bound on the root mean square over those outputs: 2.5e-5 rms(y)."""
import numpy as np
import pytest

from oracle import decoder_ops as do, q4_oracle
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch, x_to_dev, y_bits
from test_gpu_moe import _lib, dev, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# latency form with and without tiles of more than four slots; joined and throughput, whole and
# narrow tiles, one and two column tiles; long F, where the down product runs in chunks
SHAPES = [(1, 4096, 768, 8, 8), (16, 4096, 776, 2, 1), (4, 4096, 1408, 8, 4), (64, 2048, 768, 20, 4), (64, 2560, 1280, 8, 2),
          (19, 4096, 1016, 20, 3), (19, 2048, 1944, 9, 6), (48, 1024, 4096, 2, 1), (4, 4096, 6008, 4, 2)]


@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
def test_h_keeps_its_bits(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    rng = np.random.default_rng(F)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    y = q4lin.moe_experts(x_to_dev(x), t.from_numpy(ids).cuda(), t.from_numpy(p).cuda(), dev(gu), dev(gus), dev(dn), dev(dns))
    t.cuda.synchronize()
    want = do.moe_experts(x, ids, p, gu, gus, dn, dns)
    got = q4_oracle.bf16_bits_to_f64(y_bits(y))
    rms = np.sqrt((want * want).mean(axis=1, keepdims=True)) * np.ones_like(want)
    small = np.abs(want) <= rms / 256
    assert small.sum() >= 8
    off = (got - want)[small] / rms[small]
    assert np.sqrt((off * off).mean()) <= 2.5e-5
