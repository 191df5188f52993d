"""Prompts, decode steps and answers of the decoder-block example together: the cache holds what the prompts left, a
decode step attends to it as the oracle says, and decoding a prompt token by token agrees with the prompt at once."""
import numpy as np
import pytest

import oracle
from examples.decoder_block import DecoderBlock
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch
from test_gpu_decoder_block import SIZES, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def packed(lengths):
    t = torch()
    n = t.tensor(lengths, device="cuda")
    cu = t.nn.functional.pad(n.cumsum(0), (1, 0)).int()
    rows = t.arange(len(lengths), dtype=t.int32, device="cuda").repeat_interleave(n)
    return cu, rows, t.arange(len(rows), dtype=t.int32, device="cuda") - cu[rows.long()]


def test_prompt_then_steps_then_answers():
    t = torch()
    lengths = [70, 1, 130, 9]
    block = DecoderBlock(4, 140, seed=3, V=1000, **SIZES)
    D, Hk = block.D, block.Hk
    cu, rows, at = packed(lengths)
    gen = t.Generator(device="cuda").manual_seed(1)
    x = t.randn((len(rows), SIZES["H"]), device="cuda", generator=gen).to(t.bfloat16)
    adapters = (t.arange(4, device="cuda") % 4 - 1).int()
    out = block.prefill(x, adapters[rows.long()], cu, rows, at)
    assert t.isfinite(out).all()
    # a step: its attention over the cache that the prompts (and the step itself) left
    xs = out[cu[1:].long() - 1].clone()
    positions = t.tensor(lengths, dtype=t.int32, device="cuda")
    y, got = block.step(xs, adapters, positions)
    q = host(got["qkv"])[:, :block.Hq * D].reshape(4, block.Hq, D)
    want, w = ao.kv4_attention(q, host(block.cache), host(block.table), [n + 1 for n in lengths], D)
    a = oracle.bf16_bits_to_f64(host(got["a"])).reshape(want.shape)
    # (the attention's own test has the bound's parts; scores here are below 40: 2^-14 covers theirs)
    assert (np.abs(a - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * w + 1e-6).all()
    # the step's token is in the cache: what is read back is the quantised key and value
    k = host(got["qkv"])[:, block.Hq * D:(block.Hq + Hk) * D].reshape(4, Hk, D)
    kr, _ = q4lin.kv4_read(block.cache, block.table, positions, D)
    values = ao.kv4_values(*ao.kv4_quantise(k))
    assert (np.abs(oracle.bf16_bits_to_f64(host(kr)) - values) <= 2.0 ** -8 * np.abs(values)).all()
    tok = t.tensor([[5, 999]] * 4, dtype=t.int32, device="cuda")
    logp, entropy, ids, top = block.answer(y, tok)
    logits = oracle.linear(host(block.head[0]), host(block.head[1]), host(block.norm(y, 1)))
    assert logp.shape == (4, 2) and top.shape == ids.shape == (4, 5)
    for r in range(4):
        m = logits[r].max()
        logs = logits[r] - m - np.log(np.exp(logits[r] - m).sum())
        # logits are bf16: 2^-8 of each, and the sum of exponentials by as much of the largest
        tol = 2.0 ** -8 * (np.abs(logits[r]) + np.abs(logits[r]).max()) + 8e-3 * np.abs(logits[r]) + 1e-3 * np.sqrt((logits ** 2).mean()) * 2
        assert (np.abs(host(logp)[r] - logs[[5, 999]]) <= tol[[5, 999]] + tol.max()).all()
        assert (np.abs(host(top)[r] - logs[host(ids)[r]]) <= tol[host(ids)[r]] + tol.max()).all()


def test_a_prompt_at_once_and_token_by_token():
    """The same tokens through prompt_attention on bf16 keys and values and through decode steps over 4-bit ones: the first
    token sees only itself, so its attention differs by its value's quantisation alone."""
    t = torch()
    block = DecoderBlock(1, 70, seed=5, **SIZES)
    x = t.randn((1, SIZES["H"]), device="cuda").to(t.bfloat16)
    adapters = t.full((1,), -1, dtype=t.int32, device="cuda")
    cu, rows, at = packed([1])
    block.prefill(x, adapters, cu, rows, at)
    _, v = q4lin.kv4_read(block.cache, block.table, at, block.D, rows=rows)
    _, got = block.step(x, adapters, at)
    want = v.repeat_interleave(block.Hq // block.Hk, dim=1).flatten(1)
    # p = 1 exactly; the value passes as fp16 weight (2^-11) times an exact code, and is rounded to bf16 once here, once there
    assert ((got["a"].double() - want.double()).abs() <= (2 * 2.0 ** -8 + 2.0 ** -11) * want.double().abs()).all()
