"""Log probabilities, entropy and top tokens on the GPU against the FP64 oracle.

Bound of a log probability x - M - ln S: FP32's roundings of the two differences, 2^-23 (|x - M| + ln S); S itself, with the
exponential's 2^-22 and that of its argument (2^-24 of up to 40 / ln 2: 2^-18 only for terms e^-40 and less of the
largest, else 2^-24 |x - M| and so within 2^-23 of a term's share), and sums of V / 128 + 24 terms a thread and
through the trees: (V / 128 + 32) 2^-24.  The entropy adds the same relative error of its second term."""
import math

import numpy as np
import pytest

import oracle
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import torch, x_to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    yield
    assert q4lin.device_status() == 0


def logits(T, V, seed, std=3.0):
    x = synth.normal(synth.stream_state(seed, 0x4C50), T * V).reshape(T, V) * std
    return x


def to_dev(x, fp32):
    """(tensor, its values in FP64)."""
    if fp32:
        f = x.astype(np.float32)
        return torch().from_numpy(f).cuda(), f.astype(np.float64)
    b = synth.to_bf16_bits(x)
    return x_to_dev(b), oracle.bf16_bits_to_f64(b)


def check(got, x, targets, k):
    logp, ent, ids, top = (g.cpu().numpy().astype(np.float64) for g in got)
    wl, we, wi, wt = ao.token_logprobs(x, targets, k)
    V = x.shape[1]
    rel = 2.0 ** -22 + 2.0 ** -23 + (V / 128 + 32) * 2.0 ** -24
    assert np.array_equal(ids, wi)
    for g, w in ((logp.reshape(wl.shape), wl), (top, wt)):
        assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(np.isinf(g), np.isinf(w))
        f = np.isfinite(w)
        with np.errstate(invalid="ignore"):
            assert (np.abs(g - w)[f] <= 2.0 ** -23 * (np.abs(w[f]) + 2 * math.log(V)) + rel).all(), np.max(np.abs(g - w)[f])
    assert np.array_equal(np.isnan(ent), np.isnan(we))
    f = np.isfinite(we)
    assert (np.abs(ent - we)[f] <= (rel + 2.0 ** -21) * (1 + we[f])).all(), np.max(np.abs(ent - we)[f])


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,V,n,k", [(1, 1, 1, 1), (3, 2, 2, 2), (2, 7, 1, 5), (5, 33, 3, 8), (4, 1000, 1, 0), (7, 4099, 4, 32),
                                     (1, 50001, 2, 8), (2, 131072, 1, 16), (330, 777, 1, 3), (40, 20000, 0, 5), (1, 262144, 1, 8)])
def test_matches_oracle(T, V, n, k, fp32):
    t = torch()
    x, f = to_dev(logits(T, V, T + V), fp32)
    tok = np.random.default_rng(V).integers(-1, V + 1, (T, n)).astype(np.int32)   # some are padding
    td = t.from_numpy(tok).cuda()
    check(q4lin.token_logprobs(x, td, k), f, tok, k)
    # rows of a longer stride, starting anywhere
    wide = t.full((T, V + 5), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 3:3 + V] = x
    a, b = q4lin.token_logprobs(wide[:, 3:3 + V], td, k), q4lin.token_logprobs(x, td, k)
    check(a, f, tok, k)
    for u, v in zip(q4lin.token_logprobs(x, td, k), b):
        assert t.equal(u, v)


@pytest.mark.parametrize("fp32", [False, True])
def test_ties_masks_and_values_that_are_not_finite(fp32):
    t = torch()
    V = 5003
    x = logits(14, V, 3)
    inf, nan = math.inf, math.nan
    x[0] = 1.5                                             # all equal: the first tokens
    x[1] = -inf                                            # nothing
    x[2], x[2, 77], x[2, 4000] = -inf, 2.0, -3.0           # two tokens
    x[3, 4001], x[3, 9] = inf, inf
    x[4, 1234] = nan
    x[5, ::2] = -inf
    x[6] = np.round(x[6])                                  # many ties
    x[7] = -1e30
    x[8, 100] = 1e30
    x[9] = np.linspace(-50, 50, V)                         # every chunk beats the one before
    x[10] = np.linspace(50, -50, V)
    x[11], x[11, 5] = 0.0, 40.0                            # nearly certain
    x[12, :4000] = -inf
    x[13] = -3.3e38
    x[13, 17] = -3.2e38
    xd, f = to_dev(x, fp32)
    tok = np.tile(np.array([0, 77, 4001, 1234, -1, V], dtype=np.int32), (14, 1))
    check(q4lin.token_logprobs(xd, t.from_numpy(tok).cuda(), 12), f, tok, 12)
    got = q4lin.token_logprobs(xd, t.from_numpy(tok[:, 0].copy()).cuda(), 0)
    assert got[0].shape == (14,) and got[2].shape == (14, 0)


def test_large_rows_in_order():
    """A row whose logits rise all the way on one CTA per row: every insertion there can be."""
    t = torch()
    V = 40000
    x, f = to_dev(np.tile(np.arange(V) * 1e-3, (320, 1)), True)
    tok = np.zeros((320, 1), dtype=np.int32)
    got = q4lin.token_logprobs(x, t.from_numpy(tok).cuda(), 32)
    assert (got[2].cpu().numpy() == np.arange(V - 1, V - 33, -1)).all()
    check(tuple(g[:2] for g in got), f[:2], tok[:2], 32)


def test_streams_graph_and_refusals():
    t = torch()
    x, f = to_dev(logits(3, 999, 1), False)
    tok = t.tensor([[1], [2], [3]], dtype=t.int32, device="cuda")
    want = q4lin.token_logprobs(x, tok, 4)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = q4lin.token_logprobs(x, tok, 4, stream=s)
    s.synchronize()
    outs = [t.zeros_like(w) for w in want]
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        q4lin.token_logprobs(x, tok, 4, *outs)
    g.replay()
    t.cuda.synchronize()
    for a, b, c in zip(want, got, outs):
        assert t.equal(a, b) and t.equal(a, c)
    for bad in (dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x.T), dict(targets=tok.long()), dict(targets=tok[:2]),
                dict(entropy=outs[1][:2]), dict(top_ids=outs[2][:, :3])):
        kw = dict(logits=x, targets=tok, top_k=4)
        kw.update(bad)
        with pytest.raises(ValueError):
            q4lin.token_logprobs(**kw)
    with pytest.raises(q4lin.Q4LinError):
        q4lin.token_logprobs(x, tok, 33)
