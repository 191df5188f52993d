"""The operators together, as the decoder-block example runs them: every operator's output
against the FP64 oracle on the inputs it got, at the bounds of its own tests, and the captured
step against the plain one bit for bit."""
import numpy as np
import pytest

from examples.decoder_block import DecoderBlock
from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import assert_close, torch

pytestmark = pytest.mark.gpu

SIZES = dict(H=264, Hq=6, Hk=2, D=64, F=136, E=12, top_k=3, L=3, R=8)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def host(t):
    """numpy copy: the bits of 16-bit floats, other types as they are."""
    if t.dtype in (torch().bfloat16, torch().float16):
        return t.contiguous().view(torch().int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


def inputs(T, seed):
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(seed)
    x = t.randn((T, SIZES["H"]), device="cuda", generator=gen).to(t.bfloat16)
    adapters = (t.arange(T, device="cuda") % 4 - 1).to(t.int32)
    positions = (t.arange(T, device="cuda") % 5).to(t.int32)
    return x, adapters, positions


@pytest.mark.parametrize("T", [1, 5, 33])
def test_every_operator_of_a_step_matches_the_oracle(T):
    block = DecoderBlock(T, 8, seed=T, **SIZES)
    x, adapters, positions = inputs(T, T)
    _, got = block.step(x, adapters, positions)
    h = {k: host(v) for k, v in got.items()}
    ids, sc = host(adapters), host(block.adapter_scales)
    want = do.linear_lora(host(block.qkv[0]), host(block.qkv[1]), h["xn"], host(block.qkv_a), host(block.qkv_b), ids, sc)
    assert_close(h["raw"], want)
    want = do.linear_lora(host(block.o[0]), host(block.o[1]), h["a"], host(block.o_a), host(block.o_b), ids, sc)
    assert_close(h["o"], want)
    D, nq, nk = block.D, block.Hq * block.D, block.Hk * block.D
    for at, n, w in ((0, nq, block.q_weight), (nq, nk, block.k_weight)):
        want = do.qk_norm_rope(h["raw"][:, at:at + n].reshape(T, -1, D), host(w), host(block.cos_sin), host(positions))
        assert_close(np.ascontiguousarray(h["qkv"][:, at:at + n]), want.reshape(T, -1))
    assert np.array_equal(h["qkv"][:, nq + nk:], h["raw"][:, nq + nk:])   # values are left alone
    _, _, logits = do.moe_router(h["hn"], host(block.router), block.top_k)
    for t in range(T):   # largest first; FP32 sums may swap logits closer than 1e-4
        best = np.sort(logits[t])[::-1][:block.top_k]
        assert np.abs(logits[t, h["ids"][t]] - best).max() < 1e-4
    want = do.moe_experts(h["hn"], h["ids"], h["weights"], host(block.gate_up[0]), host(block.gate_up[1]),
                          host(block.down[0]), host(block.down[1]))
    assert_close(h["y"], want)


def test_captured_steps_repeat_the_plain_ones():
    t = torch()
    x, adapters, positions = inputs(5, 11)
    plain, captured = DecoderBlock(5, 8, seed=1, **SIZES), DecoderBlock(5, 8, seed=1, **SIZES)
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
    assert t.isfinite(x.float()).all()
    assert t.equal(x.view(t.int16), xs.view(t.int16))
