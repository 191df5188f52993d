"""The oracle of the attention operators and the logits' answers against plain Python loops on tiny
shapes, its cache layout as a bijection, and its quantiser on values worked out by hand."""
import math

import numpy as np
import pytest

import oracle
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import synth


def bits(shape, seed, std=1.0):
    n = int(np.prod(shape))
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x4154), n) * std).reshape(shape)


def test_prompt_attention_against_loops():
    T, Hq, Hk, D = 7, 4, 2, 8
    q, k, v = bits((T, Hq, D), 1), bits((T, Hk, D), 2), bits((T, Hk, D), 3)
    y, _ = ao.prompt_attention(q, k, v, [1, 4, 4, 6])
    f = oracle.bf16_bits_to_f64
    assert np.isnan(y[[0, 6]]).all()
    for a, t in ((1, 1), (1, 3), (4, 4), (4, 5)):
        for h in range(Hq):
            w = [math.exp(sum(f(q)[t, h, d] * f(k)[j, h // 2, d] for d in range(D)) / math.sqrt(D)) for j in range(a, t + 1)]
            for d in range(D):
                want = sum(x * f(v)[a + i, h // 2, d] for i, x in enumerate(w)) / sum(w)
                assert math.isclose(y[t, h, d], want, rel_tol=1e-12, abs_tol=1e-12)
    assert np.allclose(y[1], np.repeat(f(v)[1], 2, axis=0))     # a sequence's first row sees itself alone


def test_quantiser_by_hand():
    x = np.zeros(70)
    x[:6] = [7.0, -7.0, 3.5, 0.5, 1.5, -8.0 / 7]                # scale 1: halves go to even
    x[64:] = [-14.0, 1.0, 2.9, 3.0, 0.0, 13.0]                  # scale 2 (a short last group)
    codes, s = ao.kv4_quantise(synth.to_bf16_bits(x))
    assert oracle.fp16_bits_to_f64(s).tolist() == [1.0, 2.0]
    assert codes[:7].tolist() == [15, 1, 12, 8, 10, 7, 8]
    assert codes[64:].tolist() == [1, 8, 9, 10, 8, 14]          # 1.5 to 2, 6.5 to 6
    x[3] = np.inf
    codes, s = ao.kv4_quantise(synth.to_bf16_bits(x))
    assert np.isnan(oracle.fp16_bits_to_f64(s)[0]) and oracle.fp16_bits_to_f64(s)[1] == 2.0
    assert np.isnan(ao.kv4_values(codes, s)[:64]).all()
    codes, s = ao.kv4_quantise(synth.to_bf16_bits(np.full(64, 1e30)))
    assert oracle.fp16_bits_to_f64(s) == 65504.0 and (codes == 15).all()
    codes, s = ao.kv4_quantise(synth.to_bf16_bits(np.full(64, 1e-30)))
    assert oracle.fp16_bits_to_f64(s) == 0.0 and (codes == 8).all()


@pytest.mark.parametrize("D", [64, 96, 128])
def test_layout_uses_every_nibble_once(D):
    used = np.zeros((2, ao.page_bytes(D)), dtype=int)
    for o in range(ao.PAGE):
        kb, vb, sh, ks, vs = ao.places(D, o)
        for b, n in zip(kb + vb, sh + sh):
            used[n // 4, b] += 1
        for b in ks + vs:
            used[:, b:b + 2] += 1
    assert (used == 1).all()
    cache = np.zeros((2, 3, ao.page_bytes(D)), dtype=np.uint8)
    codes, s = ao.kv4_quantise(bits((2, D), D))
    for side in range(2):
        ao.kv4_store(cache, 1, 2, 37, side, codes[side], s[side])
    for side in range(2):
        c, t = ao.kv4_load(cache, 1, 2, 37, side, D)
        assert np.array_equal(c, codes[side]) and np.array_equal(t, s[side])


def test_cache_attention_is_prompt_attention_of_its_values():
    D, n = 64, 70
    kq, ks = ao.kv4_quantise(bits((n, 2, D), 5))
    vq, vs = ao.kv4_quantise(bits((n, 2, D), 6))
    table = np.array([[2, 0]])
    cache = np.zeros((3, 2, ao.page_bytes(D)), dtype=np.uint8)
    for t in range(n):
        for h in range(2):
            ao.kv4_store(cache, table[0, t // 64], h, t % 64, 0, kq[t, h], ks[t, h])
            ao.kv4_store(cache, table[0, t // 64], h, t % 64, 1, vq[t, h], vs[t, h])
    q = bits((3, 4, D), 7)
    y, _ = ao.kv4_attention(q, cache, table, [n], D)
    k, v = ao.kv4_values(kq, ks), ao.kv4_values(vq, vs)
    for i in range(3):
        for h in range(4):
            m = n - 2 + i
            p = np.exp(k[:m, h // 2] @ oracle.bf16_bits_to_f64(q)[i, h] / 8.0)
            assert np.allclose(y[i, h], p @ v[:m, h // 2] / p.sum(), rtol=1e-12)
    y, _ = ao.kv4_attention(q, cache, table, [1], D)             # the first two see nothing
    assert (y[:2] == 0).all() and np.allclose(y[2], np.repeat(v[0], 2, axis=0))
    y, _ = ao.kv4_attention(q, cache, np.array([[2, 9]]), [n], D)  # the second page is not there
    for i in range(3):
        p = np.exp(k[:64, 0] @ oracle.bf16_bits_to_f64(q)[i, 0] / 8.0)
        assert np.allclose(y[i, 0], p @ v[:64, 0] / p.sum(), rtol=1e-12)


def test_logprobs_by_hand():
    inf, nan = math.inf, math.nan
    x = np.array([[0.0, math.log(2), 0.0, -inf], [-inf] * 4, [1.0, inf, 3.0, inf], [0.0, nan, 5.0, 1.0]])
    logp, h, ids, top = ao.token_logprobs(x, [[1, 3], [0, -1], [1, 0], [2, 4]], 3)
    assert np.allclose(logp[0], [math.log(0.5), -inf]) and np.isclose(h[0], 1.5 * math.log(2))
    assert ids[0].tolist() == [1, 0, 2] and np.allclose(top[0], np.log([0.5, 0.25, 0.25]))
    assert logp[1].tolist() == [-inf, 0.0] and h[1] == 0 and (ids[1] == -1).all() and (top[1] == -inf).all()
    assert np.allclose(logp[2], [math.log(0.5), -inf]) and ids[2].tolist() == [1, 3, 2]
    assert np.allclose(top[2], [math.log(0.5)] * 2 + [-inf]) and np.isclose(h[2], math.log(2))
    assert np.isnan(logp[3, 0]) and logp[3, 1] == 0 and np.isnan(h[3]) and ids[3].tolist() == [2, 3, 0]
