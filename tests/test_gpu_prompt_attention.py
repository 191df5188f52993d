"""Attention over packed prompts on the GPU against the FP64 oracle.

Bound per value y = sum p v / sum p, W = sum p |v| / sum p: the output's rounding, 2^-8 |y|; the weights'
in the second product, 2^-8 W; scores in FP32, D products and their sums in any order, scale and
log2 e: an exponent off by (D + 8) 2^-24 of the largest sum of magnitudes scale * sum |q k|, which
enters a weight and the sum of weights: twice that of W; the exponential's own 2^-22, likewise twice;
FP32 sums of len terms: (len / 8 + 16) 2^-24 W for numerator and denominator each."""
import numpy as np
import pytest

import oracle
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import torch, x_to_dev, y_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def bits(shape, seed, std=1.0):
    n = int(np.prod(shape))
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x5041), n) * std).reshape(shape)


def check(got, q, k, v, cu, scale=None):
    T, Hq, D = q.shape
    y, w = ao.prompt_attention(q, k, v, cu, scale)
    f = oracle.bf16_bits_to_f64
    scale = D ** -0.5 if scale is None else scale
    with np.errstate(all="ignore"):
        off = 2.0 ** -8 + 2 * (abs(scale) * mags(q, k) * (D + 8) * 2.0 ** -24 + 2.0 ** -22 + (T / 8 + 16) * 2.0 ** -24)
        tol = 2.0 ** -8 * np.abs(y) + off * w + 1e-38
    rows = ~np.isnan(y).all(axis=(1, 2)) if np.isfinite(f(v)).all() and np.isfinite(f(q)).all() else slice(cu[0], cu[-1])
    g, y, tol = oracle.bf16_bits_to_f64(got)[rows], y[rows], tol[rows]
    fin = np.isfinite(y)
    assert (np.abs(g - y)[fin] <= tol[fin]).all(), np.nanmax(np.abs(g - y)[fin] / tol[fin])
    assert np.array_equal(np.isnan(g), np.isnan(y)) and np.array_equal(g[np.isinf(y)], y[np.isinf(y)])


def mags(*both):
    """A bound of sum |q_d k_d| over all pairs of rows (Cauchy-Schwarz)."""
    return np.prod([np.sqrt((np.where(np.isfinite(x), x, 0) ** 2).sum(-1)).max()
                    for x in map(oracle.bf16_bits_to_f64, both)])


@pytest.mark.parametrize("lens,pad,Hq,Hk,D", [
    ([1], 0, 1, 1, 8), ([1, 1, 1], 2, 2, 1, 128), ([2], 0, 4, 4, 64), ([127], 0, 4, 1, 128), ([128], 1, 2, 2, 128),
    ([129], 0, 6, 2, 96), ([64, 0, 65, 1, 0, 200], 7, 5, 1, 80), ([300], 0, 7, 7, 40), ([255, 257], 0, 8, 1, 64),
    ([31, 33, 17, 400, 5], 3, 4, 2, 112), ([513], 0, 3, 1, 128), ([700, 3], 0, 2, 1, 120), ([0, 0], 5, 2, 1, 64),
    ([383, 385], 0, 10, 2, 16)])
def test_matches_oracle(lens, pad, Hq, Hk, D):
    t = torch()
    T = sum(lens) + pad + 2                                   # two rows before the first sequence
    cu = np.cumsum([2] + lens)
    row = bits((T, (Hq + 2 * Hk) * D + 8), T + D)             # packed rows
    q, k, v = (np.ascontiguousarray(row[:, a * D:b * D].reshape(T, -1, D))
               for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    r = x_to_dev(row)
    cud = t.tensor(cu, dtype=t.int32, device="cuda")
    views = [r[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))]
    out = t.full((T, Hq + 1, D), 7.0, dtype=t.bfloat16, device="cuda")   # rows with a gap behind them
    q4lin.prompt_attention(*views, cud, out=out[:, :Hq])
    t.cuda.synchronize()
    assert (out[:, Hq] == 7.0).all() and (out[:2] == 7.0).all() and (out[cu[-1]:] == 7.0).all()
    check(y_bits(out[:, :Hq].contiguous()), q, k, v, cu)
    again = q4lin.prompt_attention(*views, cud)               # the same bits, other rows
    t.cuda.synchronize()
    assert t.equal(again[2:cu[-1]].view(t.int16), out[2:cu[-1], :Hq].contiguous().view(t.int16))
    assert t.equal(r.view(t.int16), x_to_dev(row).view(t.int16))


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-0.3, 1.0), (5.0, 2.0), (0.125, 30.0), (1e-30, 1.0)])
def test_scales_and_large_scores(scale, std):
    t = torch()
    q, k, v = bits((150, 2, 64), 1, std), bits((150, 1, 64), 2, std), bits((150, 1, 64), 3, 1e3)
    cu = [0, 90, 150]
    out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), t.tensor(cu, dtype=t.int32, device="cuda"), scale)
    check(y_bits(out), q, k, v, cu, scale)


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(D):
    """NaN and infinities in later tokens, other sequences and rows of no sequence; rows that see one get the
    definition's value."""
    t = torch()
    T, cu = 420, [3, 200, 400]
    q, k, v = bits((T, 2, D), 11), bits((T, 1, D), 12), bits((T, 1, D), 13)
    inf, ninf, nan = 0x7F80, 0xFF80, 0x7FC0
    v[:3], v[400:], k[:3], k[400:], q[400:] = nan, inf, nan, nan, inf
    v[150, 0, 5] = inf
    v[180, 0, 5] = ninf          # rows from here on: inf - inf
    v[100, 0, 7] = nan
    v[199, 0, D - 1] = ninf      # the last row of its sequence
    v[330, 0, 0] = inf
    v[260, 0, 9] = ninf
    k[390, 0, 3] = nan           # (rows 390 .. 399 see it)
    out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), t.tensor(cu, dtype=t.int32, device="cuda"))
    check(y_bits(out), q, k, v, cu)


def test_cu_seqlens_outside_the_tensors():
    """Bounds beyond T or below 0 are taken into [0, T]; a sequence that would run backwards is empty."""
    t = torch()
    q, k, v = bits((100, 2, 64), 1), bits((100, 1, 64), 2), bits((100, 1, 64), 3)
    args = [x_to_dev(x) for x in (q, k, v)]
    out = q4lin.prompt_attention(*args, t.tensor([-5, 40, 1 << 30], dtype=t.int32, device="cuda"))
    check(y_bits(out), q, k, v, [0, 40, 100])
    out = t.full((100, 2, 64), 7.0, dtype=t.bfloat16, device="cuda")
    q4lin.prompt_attention(*args, t.tensor([90, 20, -1], dtype=t.int32, device="cuda"), out=out)
    t.cuda.synchronize()
    assert (out == 7.0).all()


def test_many_sequences():
    t = torch()
    lens = [(i * 7) % 5 for i in range(700)]
    T = sum(lens)
    q, k, v = bits((T, 2, 64), 1), bits((T, 1, 64), 2), bits((T, 1, 64), 3)
    cu = np.cumsum([0] + lens)
    out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), t.tensor(cu, dtype=t.int32, device="cuda"))
    check(y_bits(out), q, k, v, cu)


def test_long_prompt_sampled_rows():
    """A prompt of many tiles: sampled rows against FP64 on the GPU."""
    t = torch()
    T, Hq, Hk, D = 9000, 4, 2, 128
    q, k, v = (x_to_dev(bits((T, h, D), i, 2.0)) for i, h in ((1, Hq), (2, Hk), (3, Hk)))
    out = q4lin.prompt_attention(q, k, v, t.tensor([0, T], dtype=t.int32, device="cuda"))
    for r in [0, 1, 127, 128, 129, 4095, 4096, 5000, 8191, 8192, 8960, 8998, 8999]:
        for h in range(Hq):
            s = k[:r + 1, h // 2].double() @ q[r, h].double() * D ** -0.5
            p = t.softmax(s, 0)
            y, w = p @ v[:r + 1, h // 2].double(), p @ v[:r + 1, h // 2].double().abs()
            size = float((k[:r + 1, h // 2].double().abs() @ q[r, h].double().abs()).max()) * D ** -0.5
            off = 2.0 ** -8 + 2 * (size * (D + 8) * 2.0 ** -24 + 2.0 ** -22 + (T / 8 + 16) * 2.0 ** -24)
            assert ((out[r, h].double() - y).abs() <= 2.0 ** -8 * y.abs() + off * w).all(), (r, h)


def test_streams_graph_and_refusals():
    t = torch()
    q, k, v = (x_to_dev(bits((130, h, 64), i)) for i, h in ((1, 4), (2, 2), (3, 2)))
    cu = t.tensor([0, 50, 130], dtype=t.int32, device="cuda")
    want = q4lin.prompt_attention(q, k, v, cu)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = q4lin.prompt_attention(q, k, v, cu, stream=s)
    s.synchronize()
    assert t.equal(got, want)
    out, g = t.zeros_like(want), t.cuda.CUDAGraph()
    qs = q.clone()
    with t.cuda.graph(g):
        q4lin.prompt_attention(qs, k, v, cu, out=out)
    qs.copy_(q * 2)
    cu.copy_(t.tensor([0, 120, 130]))
    g.replay()
    t.cuda.synchronize()
    assert t.equal(out, q4lin.prompt_attention(q * 2, k, v, cu))
    for bad in (dict(q=q.float()), dict(q=q.flatten(1)), dict(k=k[:100]), dict(v=v[:, :1]), dict(cu_seqlens=cu.long()),
                dict(out=out[:, :2]), dict(cu_seqlens=cu.cpu()), dict(k=k.transpose(1, 2))):
        kw = dict(q=q, k=k, v=v, cu_seqlens=cu)
        kw.update(bad)
        with pytest.raises(ValueError):
            q4lin.prompt_attention(**kw)
    for bad in (dict(q=q[:, :3], out=out[:, :3]), dict(scale=float("nan")), dict(q=t.zeros((130, 4, 136), dtype=t.bfloat16, device="cuda"),
                k=t.zeros((130, 2, 136), dtype=t.bfloat16, device="cuda"), v=t.zeros((130, 2, 136), dtype=t.bfloat16, device="cuda"))):
        kw = dict(q=q, k=k, v=v, cu_seqlens=cu)
        kw.update(bad)
        with pytest.raises(q4lin.Q4LinError):
            q4lin.prompt_attention(**kw)
