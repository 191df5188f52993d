"""V scales of tokens that only some of a sequence's new tokens see, and scales that are not finite: neither costs other columns
or other groups of values their bits.

Bound: that of test_gpu_kv4.py for each row by itself, over the tokens that the row sees."""
import numpy as np
import pytest

import oracle
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin

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


def v_scales(cache, Hk, D):
    """The fp16 bits of V's scales, a view [pages, Hk, 64 tokens, groups]."""
    g = -(-D // 64)
    return cache[:, :, 64 * D:].view(np.uint16).reshape(len(cache), Hk, 2, 64, g)[:, :, 1]


@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 4), (96, 9)])
@pytest.mark.parametrize("L,n", [(70, 4), (64, 3), (200, 2), (130, 8), (66, 5)])
@pytest.mark.parametrize("bits16", [0x7C00, 0xFC00, 0x7E00, 0x7BFF])      # +-inf, NaN, 65504
def test_a_new_tokens_scale_reaches_the_rows_that_see_it_alone(L, n, D, Hq, bits16):
    """The other tokens' scales are 2^-14 and less; the last new token's is not finite, or the largest there is."""
    cache, table = filled(1, [L], 4, 1, D, L + n, std=2.0 ** -12)
    q = bits((n, Hq, D), L, 1.5)
    page, o = table[0, (L - 1) // 64], (L - 1) % 64
    v_scales(cache, 1, D)[page, 0, o] = bits16
    got = y_bits(q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array([L], dtype=np.int32))))
    seen = cache.copy()
    v_scales(seen, 1, D)[page, 0, o] = 0       # (the rows below do not see that token)
    for i in range(n - 1):
        m = L - (n - 1 - i)
        if m > 0:
            only = np.zeros_like(seen)
            only[table[0]] = seen[table[0]]
            v_scales(only, 1, D)[table[0, (m - 1) // 64], 0, (m - 1) % 64 + 1:] = 0
            if (m - 1) // 64 < 3:
                v_scales(only, 1, D)[table[0, (m - 1) // 64 + 1:], 0] = 0
            check(got[i:i + 1], q[i:i + 1], only, table, [m], D)
    last = oracle.bf16_bits_to_f64(got[n - 1])
    if bits16 == 0x7BFF:
        only = np.zeros_like(cache)
        only[table[0]] = cache[table[0]]
        check(got[n - 1:], q[n - 1:], only, table, [L], D)
    else:
        assert not np.isfinite(last).all()


@pytest.mark.parametrize("L,n,Hq", [(64, 1, 4), (300, 1, 4), (300, 3, 8)])
def test_an_infinite_scale_stays_with_its_group_of_values(L, n, Hq):
    """Heads of 128 values: the second group of the columns that see the token is as it would be without it."""
    D = 128
    cache, table = filled(1, [L], 5, 1, D, L)
    q = bits((n, Hq, D), L, 1.5)
    clean = cache.copy()
    v_scales(cache, 1, D)[table[0, 0], 0, 20, 0] = 0x7C00
    v_scales(clean, 1, D)[table[0, 0], 0, 20, 0] = 0
    got = y_bits(q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array([L], dtype=np.int32))))
    y, _ = ao.kv4_attention(q, clean, table, [L], D)
    f = oracle.bf16_bits_to_f64(got)
    assert np.isfinite(f[..., 64:]).all() and not np.isfinite(f[..., :64]).any()
    # the first group's place is taken by the clean result: check() then holds the second to its bound
    mixed = got.copy()
    from weight_only_bit_q4_gb300 import synth
    mixed[..., :64] = synth.to_bf16_bits(y)[..., :64]
    check(mixed, q, clean, table, [L], D)
