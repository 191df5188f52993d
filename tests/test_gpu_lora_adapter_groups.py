"""LinearLora beyond 32 tokens with few adapters of low rank, where the second product runs as
further K groups of the tile kernel, and what Inf and NaN in an adapter may reach on every route.
Bound as for LinearLora everywhere: 8e-3 |y| + 1e-3 rms(y)."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from oracle import q4_oracle
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import assert_close, y_bits
from test_gpu_lora import _lib, call, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# all adapters' ranks within 64, within 128 (K on both sides of 4096), just past it; K and N that
# end inside a group or a tile, fewer K groups than a tile's split, several token tiles
SHAPES = [(300, 640, 33, 2, 8), (129, 4104, 40, 3, 40), (1000, 1160, 75, 2, 24), (640, 5120, 257, 7, 16), (2000, 4096, 600, 1, 64),
          (77, 72, 65, 4, 16), (5120, 1024, 300, 2, 32), (260, 4096, 48, 16, 8), (260, 4088, 48, 16, 8), (200, 4160, 50, 17, 8),
          (33, 8, 34, 1, 8), (6144, 5120, 1024, 4, 16), (500, 17408, 70, 5, 24)]


@pytest.mark.parametrize("N,K,T,L,R", SHAPES)
def test_matches_oracle(N, K, T, L, R):
    p = problem(N, K, T, L, R, N + T)
    y = call(p)
    assert_close(y_bits(y), do.linear_lora(*p), f"lora {N}x{K} T={T} L={L} R={R}")
    assert np.array_equal(y_bits(call(p)), y_bits(y))   # deterministic


@pytest.mark.parametrize("T", [40, 130, 300])
@pytest.mark.parametrize("K", [520, 4168])
def test_ranks_and_unused_garbage(T, K):
    N, L, R = 200, 4, 16
    ranks = [0, 5, 16, 99]
    p = problem(N, K, T, L, R, 5 + T, ids=np.arange(T) % (L + 1))
    a, b = p[3].copy(), p[4].copy()
    for i, r in enumerate(ranks):
        r = min(max(r, 0), R)
        a[i, r:], b[i, :, r:] = 0x7FC0, 0x7FC0
    q = p[:3] + (a, b) + p[5:]
    assert_close(y_bits(call(q, ranks)), do.linear_lora(*p, ranks), f"ranks T={T}")


@pytest.mark.parametrize("T,L,R", [(1, 3, 16), (8, 3, 16), (30, 3, 16), (40, 3, 16), (40, 12, 64), (75, 2, 64), (300, 4, 16), (300, 9, 32)])
def test_inf_and_nan_stay_with_their_adapter(T, L, R):
    N, K = 400, 4168
    p = problem(N, K, T, L, R, 77 + T, ids=np.arange(T) % (L + 1))
    ids = p[5]
    b = p[4].copy()
    hurt = 0 if T == 1 else 1
    b[hurt, 7, 3], b[hurt, 130, R - 1], b[hurt, N - 1, 0] = 0x7F80, 0x7FC0, 0xFF80   # Inf, NaN, -Inf
    clean = p[4].copy()
    for n, r in ((7, 3), (130, R - 1), (N - 1, 0)):
        clean[hurt, n, r] = 0
    y = y_bits(call(p[:4] + (b,) + p[5:]))
    want = do.linear_lora(*p[:4], clean, *p[5:])
    v = q4_oracle.bf16_bits_to_f64(y)
    own = ids == hurt
    assert own.any()
    bad = np.zeros_like(want, dtype=bool)
    for n in (7, 130, N - 1):
        bad[own, n] = True
    assert not np.isfinite(v[bad]).any()
    assert np.isnan(v[own, 130]).all()
    y, want = y.copy(), want.copy()
    y[bad], want[bad] = 0, 0.0
    assert_close(y, want, f"T={T} L={L} R={R}")
