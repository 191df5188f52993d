"""The expert layer on activations far from 1: the intermediate h goes with the square of x, up to
2^120 and down to 2^-122 here, and y is finite and normal.  Bound as for the layer everywhere
(8e-3 |y| + 1e-3 rms(y)): a power of two changes nothing but exponents."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import assert_close, torch, x_to_dev, y_bits
from test_gpu_moe import _lib, dev, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def scaled(x, e):
    """bf16 bits times 2^e (zeros stay)."""
    return np.where((x & 0x7FFF) == 0, x, (x.astype(np.int32) + e * 128)).astype(np.uint16)


@pytest.mark.parametrize("T,H,F,E,k", [(2, 264, 136, 4, 2), (6, 512, 520, 2, 1), (40, 264, 136, 6, 3), (64, 4096, 264, 20, 2)])
@pytest.mark.parametrize("big", [True, False])
def test_powers_of_two(T, H, F, E, k, big):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    # the largest |h| to about 2^120, or the typical one to about 2^-122 (where silu(g) is g / 2)
    g = do.q4_oracle.linear(gu[0], gus[0], x)
    e = (60 if big else -61) - int(np.log2(np.abs(g).max() if big else np.sqrt((g * g).mean())))
    x = scaled(x, e)
    want = do.moe_experts(x, ids, p, gu, gus, dn, dns)
    assert np.isfinite(want).all() and np.abs(want).max() < 3e38 and np.sqrt((want * want).mean()) > 2e-38
    y = q4lin.moe_experts(x_to_dev(x), t.from_numpy(ids).cuda(), t.from_numpy(p).cuda(), dev(gu), dev(gus), dev(dn), dev(dns))
    t.cuda.synchronize()
    assert_close(y_bits(y), want, f"T={T} H={H} F={F} e={e}")
