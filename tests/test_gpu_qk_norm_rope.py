"""Head norms with the position rotation on the GPU against the FP64 oracle.

Bound per value: one bf16 rounding (2^-8 relative) plus FP32 arithmetic on the norm and the
two rotated terms (about ten roundings of 2^-24, 2e-6 of the head's largest |z|)."""
import numpy as np
import pytest

import oracle
from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import torch, x_to_dev, y_bits

pytestmark = pytest.mark.gpu
P = 3000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    yield
    assert q4lin.device_status() == 0


def bits(shape, seed, std):
    n = int(np.prod(shape))
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x516B), n) * std).reshape(shape)


def table(rot):
    ang = np.arange(P)[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def close(got_bits, want, what):
    got = oracle.bf16_bits_to_f64(got_bits).reshape(want.shape)
    tol = 2.0 ** -8 * np.abs(want) + 2e-6 * np.abs(want).max(axis=-1, keepdims=True) + 1e-37
    assert (np.abs(got - want) <= tol).all(), (what, np.max(np.abs(got - want) / tol))


def weights(D, seed):
    return synth.to_bf16_bits(1.0 + 0.2 * synth.normal(synth.stream_state(seed, 0x5157), D))


@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", [
    (1, 32, 8, 128, 128, False), (1, 1, 1, 8, 0, False), (3, 5, 1, 64, 64, True), (133, 28, 4, 96, 64, True),
    (17, 3, 3, 80, 48, False), (9, 2, 0, 256, 256, False), (9, 0, 2, 256, 32, True), (7, 7, 1, 192, 96, False),
    (50, 40, 8, 128, 64, False), (600, 32, 8, 128, 128, False), (900, 33, 2, 40, 32, True), (2, 300, 1, 16, 16, False)])
def test_matches_oracle_from_packed_rows(T, Hq, Hk, D, rot, inter):
    t = torch()
    ld = (Hq + 2 * Hk) * D + 8                       # packed rows, not a multiple of anything large
    rows = bits((T, ld), T + D, 3.0)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, P, T).astype(np.int32)
    qw, kw, cs = weights(D, 1), weights(D, 2), table(rot)
    r = x_to_dev(rows)
    q, k = q4lin.qk_norm_rope(r[:, :Hq * D], r[:, Hq * D:(Hq + Hk) * D], x_to_dev(qw), x_to_dev(kw),
                              t.from_numpy(cs).cuda(), t.from_numpy(pos).cuda(), interleaved=inter)
    t.cuda.synchronize()
    qr = rows[:, :Hq * D].reshape(T, Hq, D)
    kr = rows[:, Hq * D:(Hq + Hk) * D].reshape(T, Hk, D)
    if Hq:
        close(y_bits(q), do.qk_norm_rope(qr, qw, cs, pos, interleaved=inter), "q")
    if Hk:
        close(y_bits(k), do.qk_norm_rope(kr, kw, cs, pos, interleaved=inter), "k")
    # in place, three-dimensional views: the same bits, and nothing else in the rows changes
    q4lin.qk_norm_rope(r[:, :Hq * D].unflatten(1, (Hq, D)), r[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)), x_to_dev(qw),
                       x_to_dev(kw), t.from_numpy(cs).cuda(), t.from_numpy(pos).cuda(), interleaved=inter,
                       q_out=r[:, :Hq * D].unflatten(1, (Hq, D)), k_out=r[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)))
    t.cuda.synchronize()
    rb = y_bits(r)
    assert np.array_equal(rb[:, :Hq * D], y_bits(q).reshape(T, -1))
    assert np.array_equal(rb[:, Hq * D:(Hq + Hk) * D], y_bits(k).reshape(T, -1))
    assert np.array_equal(rb[:, (Hq + Hk) * D:], rows[:, (Hq + Hk) * D:])


def test_positions_outside_the_table_zero_heads_and_large_values():
    t = torch()
    T, H, D, rot = 6, 2, 64, 32
    rows = bits((T, 2 * H * D), 8, 1.0)
    rows[2] = 0                                        # a head of zeros: eps decides, 0 comes out
    rows[3] = synth.to_bf16_bits(np.full(2 * H * D, 1e18))   # squares near the top of FP32
    rows[4] = synth.to_bf16_bits(np.full(2 * H * D, 1e-20))  # squares below its smallest normal
    pos = np.array([-1, P, 0, 5, P - 1, 1 << 30], dtype=np.int32)
    w, cs = weights(D, 3), table(rot)
    r = x_to_dev(rows)
    out = t.full((T, 2 * H * D), 7.0, dtype=t.bfloat16, device="cuda")
    q4lin.qk_norm_rope(r[:, :H * D], r[:, H * D:], x_to_dev(w), x_to_dev(w), t.from_numpy(cs).cuda(),
                       t.from_numpy(pos).cuda(), q_out=out[:, :H * D], k_out=out[:, H * D:])
    t.cuda.synchronize()
    got = y_bits(out)
    for i in (0, 1, 5):
        assert (out[i] == 7.0).all()
    want = do.qk_norm_rope(rows.reshape(T, 2 * H, D), w, cs, pos)
    for i in (2, 3, 4):
        close(got[i], want[i], f"row {i}")


def test_stream_graph_and_refusals():
    t = torch()
    T, H, D = 4, 2, 64
    r, w = x_to_dev(bits((T, 2 * H * D), 8, 1.0)), x_to_dev(weights(D, 3))
    cs, pos = t.from_numpy(table(64)).cuda(), t.arange(T, dtype=t.int32, device="cuda")
    q, k = r[:, :H * D], r[:, H * D:]
    a = q4lin.qk_norm_rope(q, k, w, w, cs, pos)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    b = q4lin.qk_norm_rope(q, k, w, w, cs, pos, stream=s)
    s.synchronize()
    assert t.equal(a[0], b[0]) and t.equal(a[1], b[1])
    qo, ko = t.zeros_like(a[0]), t.zeros_like(a[1])
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        q4lin.qk_norm_rope(q, k, w, w, cs, pos, q_out=qo, k_out=ko)
    g.replay()
    t.cuda.synchronize()
    assert t.equal(a[0], qo) and t.equal(a[1], ko)
    for bad in (dict(positions=pos.long()), dict(q_weight=w.float()), dict(cos_sin=cs[:, :48]), dict(q=q.float()),
                dict(k_out=qo[:, :D])):
        kw = dict(q=q, k=k, q_weight=w, k_weight=w, cos_sin=cs, positions=pos)
        kw.update(bad)
        with pytest.raises(ValueError):
            q4lin.qk_norm_rope(**kw)
    with pytest.raises(q4lin.Q4LinError):
        q4lin.qk_norm_rope(q, k, w, w, cs[:, :8].contiguous(), pos)
