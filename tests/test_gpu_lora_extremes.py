"""LinearLora where an adapter holds infinities, or A x comes close to the largest FP32 value, on
every route: the definition's infinities with their signs, its NaN, and finite values where it has
them.  Tokens of other adapters, and other rows, within the layer's bound (8e-3 |y| + 1e-3 rms(y))."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from oracle import q4_oracle

from gpu_util import assert_close, y_bits
from test_gpu_lora import _lib, call, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# the GEMV, the streaming route, few adapters of low rank (further K groups), many (the FP32 term;
# ranks within one step of 16, and beyond)
ROUTES = [(1, 3, 16), (8, 3, 16), (30, 3, 16), (40, 3, 16), (300, 4, 16), (40, 12, 64), (75, 20, 16), (130, 9, 72)]


@pytest.mark.parametrize("T,L,R", ROUTES)
def test_infinities_in_b(T, L, R):
    N, K = 400, 4168
    p = problem(N, K, T, L, R, 177 + T, ids=np.arange(T) % L)
    hurt = 0
    x = q4_oracle.bf16_bits_to_f64(p[2])
    u = x @ q4_oracle.bf16_bits_to_f64(p[3])[hurt].T        # [T, R]
    own = p[5] == hurt
    assert (np.abs(u[own][:, [0, 3, R - 1]]) > 1e-5).all()   # (signs are beyond doubt)
    b, clean = p[4].copy(), p[4].copy()
    inf, minus, nan = 0x7F80, 0xFF80, 0x7FC0
    for n, r, v in ((7, 3, inf), (9, 3, minus), (130, R - 1, inf), (131, 0, nan), (N - 1, 0, minus), (N - 1, R - 1, minus)):
        b[hurt, n, r], clean[hurt, n, r] = v, 0
    with np.errstate(invalid="ignore"):
        want = do.linear_lora(*p[:4], b, *p[5:])
    bad = ~np.isfinite(want)
    assert bad[own].sum() == 5 * own.sum() and not bad[~own].any()
    y = y_bits(call(p[:4] + (b,) + p[5:]))
    got = q4_oracle.bf16_bits_to_f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    plain = do.linear_lora(*p[:4], clean, *p[5:])
    y, plain = y.copy(), plain.copy()
    y[bad], plain[bad] = 0, 0.0
    assert_close(y, plain, f"T={T} L={L} R={R}")


@pytest.mark.parametrize("T,L,R", ROUTES)
def test_a_x_between_the_largest_bf16_and_the_largest_fp32(T, L, R):
    """u = 3.4e38 rounds to an infinite bf16; times B = 2^-120 it adds 256 to y."""
    N, K = 200, 520
    p = list(problem(N, K, T, L, R, 9 + T, ids=np.arange(T) % L))
    bf = lambda e: (127 + e) << 7                            # 2^e   # noqa: E731
    x, a, b, sc = p[2].copy(), p[3].copy(), p[4].copy(), p[6].copy()
    x[:, 64] = bf(0)
    a[0], b[0] = 0, 0
    a[0, 2, 64] = bf(100)
    b[0, :, 2] = bf(-120)
    b[0, 5, 2] = bf(-120) | 0x8000
    sc[0] = np.float32(3.4e38) / np.float32(2.0**100)
    p[2], p[3], p[4], p[6] = x, a, b, sc
    want = do.linear_lora(*p)
    assert np.isfinite(want).all() and np.abs(want[p[5] == 0]).min() > 50
    assert_close(y_bits(call(tuple(p))), want, f"T={T} L={L} R={R}")
