"""The expert layer on long columns: F beyond what a tile of whole columns holds (the down product
runs in chunks of F, a last one of any length), H at which the tiles of the first product narrow,
many experts.  Bound as for the layer everywhere (8e-3 |y| + 1e-3 rms(y)); the same bits again."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import assert_close, torch, x_to_dev, y_bits
from test_gpu_moe import _lib, dev, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

SHAPES = [(64, 64, 14336, 4, 2), (4, 40, 14336, 8, 2), (20, 24, 6000, 3, 2), (17, 264, 4808, 5, 3), (1, 64, 40960, 2, 1),
          (33, 72, 32768, 2, 1), (5, 136, 20488, 3, 2), (64, 3584, 488, 20, 2), (40, 16384, 24, 4, 2), (2, 30000, 16, 2, 2),
          (64, 64, 40, 1000, 8), (30, 264, 136, 300, 16)]


@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
def test_experts_match_oracle(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[T // 2, 0] = -1 if T > 1 else ids[0, 0]
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    args = (x_to_dev(x), t.from_numpy(ids).cuda(), t.from_numpy(p).cuda(), dev(gu), dev(gus), dev(dn), dev(dns))
    ws = t.empty(q4lin.moe_workspace_bytes(T, H, F, E, k), dtype=t.uint8, device="cuda")
    ys = [q4lin.moe_experts(*args, workspace=ws) for _ in range(8)]
    t.cuda.synchronize()
    assert_close(y_bits(ys[0]), do.moe_experts(x, ids, p, gu, gus, dn, dns), f"T={T} H={H} F={F} E={E} k={k}")
    assert all(t.equal(y.view(t.int16), ys[0].view(t.int16)) for y in ys)
