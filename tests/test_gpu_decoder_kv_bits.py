"""The decoder-block example with its cache in bf16: a step's attention on unrounded bf16 keys and values, prompts and steps
agree, head sizes that the 4-bit cache does not take, captured steps.

Bound of the plain FP32 attention against FP64: the output's rounding, 2^-8 |y|, and FP32's own errors in the scores (sums of
D products, below (D + 8) 2^-24 sum |q k| D^-1/2), twice, of sum p |v|."""
import numpy as np
import pytest

import oracle
from examples.decoder_block import DecoderBlock
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch
from test_gpu_decoder_answer import packed
from test_gpu_decoder_block import SIZES, host, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def attention64(q, keys, values):
    """(y, sum p |v|, bound of the scores) of heads [Hq, D] over one request's keys and values [L, Hk, D], FP64."""
    G = q.shape[0] // keys.shape[1]
    y, w, e = [], [], []
    for h in range(q.shape[0]):
        k, v = keys[:, h // G], values[:, h // G]
        s = k @ q[h] * q.shape[1] ** -0.5
        p = np.exp(s - s.max())
        p /= p.sum()
        y.append(p @ v)
        w.append(p @ np.abs(v))
        e.append((np.abs(k) @ np.abs(q[h])).max() * q.shape[1] ** -0.5)
    return np.array(y), np.array(w), np.array(e)[:, None]


@pytest.mark.parametrize("D", [64, 48, 128])      # (the rotation takes multiples of 16)
def test_prompts_then_a_step_over_a_bf16_cache(D):
    t = torch()
    lengths = [70, 1, 33]
    block = DecoderBlock(3, 72, seed=3, V=300, kv_bits=16, **{**SIZES, "D": D})
    cu, rows, at = packed(lengths)
    gen = t.Generator(device="cuda").manual_seed(1)
    x = t.randn((len(rows), SIZES["H"]), device="cuda", generator=gen).to(t.bfloat16)
    adapters = (t.arange(3, device="cuda") % 4 - 1).int()
    out = block.prefill(x, adapters[rows.long()], cu, rows, at)
    assert t.isfinite(out).all()
    positions = t.tensor(lengths, dtype=t.int32, device="cuda")
    _, got = block.step(out[cu[1:].long() - 1].clone(), adapters, positions)
    f = oracle.bf16_bits_to_f64
    qkv = host(got["qkv"])
    nq, nk = block.Hq * D, block.Hk * D
    # the step's own key and value stand in the cache bit for bit
    cache = host(block.cache)
    for r, n in enumerate(lengths):
        assert np.array_equal(cache[0, r, n].reshape(-1), qkv[r, nq:nq + nk])
        assert np.array_equal(cache[1, r, n].reshape(-1), qkv[r, nq + nk:])
        y, w, e = attention64(f(qkv[r, :nq]).reshape(-1, D), f(cache[0, r, :n + 1]), f(cache[1, r, :n + 1]))
        a = f(host(got["a"])[r]).reshape(-1, D)
        assert (np.abs(a - y) <= 2.0 ** -8 * np.abs(y) + 2 * (D + 8) * 2.0 ** -24 * (e + 8) * w + 1e-6).all()


def test_a_prompt_at_once_and_token_by_token_agree():
    """A prompt of one token leaves the same keys and values as a step, whose attention is that token's value itself."""
    t = torch()
    block = DecoderBlock(2, 8, seed=5, kv_bits=16, **SIZES)
    x = t.randn((2, SIZES["H"]), device="cuda").to(t.bfloat16)
    adapters = t.full((2,), -1, dtype=t.int32, device="cuda")
    cu, rows, at = packed([1, 1])
    block.prefill(x, adapters, cu, rows, at)
    held = block.cache.clone()
    _, got = block.step(x, adapters, at)
    assert t.equal(held.view(t.int16), block.cache.view(t.int16))
    want = block.cache[1, :, 0].repeat_interleave(block.Hq // block.Hk, dim=1).flatten(1)
    assert t.equal(got["a"].view(t.int16), want.view(t.int16))     # the first token sees only itself: its own value


def test_captured_steps_over_a_bf16_cache():
    t = torch()
    x, adapters, positions = inputs(5, 11)
    plain, captured = (DecoderBlock(5, 8, seed=1, kv_bits=16, **SIZES) for _ in range(2))
    xs, ps = x.clone(), positions.clone()
    captured.step(xs, adapters, ps)
    captured.cache.zero_()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        out, _ = captured.step(xs, adapters, ps)
    captured.cache.zero_()
    for _ in range(3):
        x, _ = plain.step(x, adapters, positions)
        positions += 1
        graph.replay()
        xs.copy_(out)
        ps += 1
    t.cuda.synchronize()
    assert t.isfinite(x.float()).all() and t.equal(x.view(t.int16), xs.view(t.int16))


def test_other_widths_are_refused():
    with pytest.raises(ValueError):
        DecoderBlock(1, 8, kv_bits=8, **SIZES)
