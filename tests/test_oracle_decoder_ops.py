"""The oracle of the decoder-block operators against plain Python loops on tiny shapes."""
import math

import numpy as np

import oracle
from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import synth


def _b(shape, seed, std=1.0):
    n = int(np.prod(shape))
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x4F70), n) * std).reshape(shape)


def _f(bits):
    return oracle.bf16_bits_to_f64(np.asarray(bits))


def test_lora_against_loops():
    N, K, T, L, R = 5, 72, 4, 3, 8
    wq, s, x = synth.make_problem(N, K, T, w_seed=1, x_seed=2)
    a, b = _b((L, R, K), 3, 0.1), _b((L, N, R), 4)
    ids, sc, ranks = np.array([2, -1, 0, 7]), np.array([0.5, 1.0, 2.0]), np.array([5, 8, 0])
    got = do.linear_lora(wq, s, x, a, b, ids, sc, ranks)
    base = oracle.linear_loops(wq, s, x)
    for t in range(T):
        for n in range(N):
            v = base[t][n]
            i = ids[t]
            if 0 <= i < L:
                for r in range(ranks[i]):
                    u = sum(_f(a)[i, r, k] * _f(x)[t, k] for k in range(K))
                    v += sc[i] * _f(b)[i, n, r] * u
            assert math.isclose(got[t, n], v, rel_tol=1e-11, abs_tol=1e-11)


def test_router_order_ties_and_masks():
    x = _b((2, 8), 5)
    w = np.repeat(_b((1, 8), 6), 5, axis=0)          # five equal experts: ties by index
    ids, p, _ = do.moe_router(x, w, 3)
    assert (ids == [[0, 1, 2], [0, 1, 2]]).all() and np.allclose(p, 1 / 3)
    ids, p, _ = do.moe_router(x, w, 3, bias=[-np.inf, 0, np.nan, 0, -np.inf])
    assert (ids == [[1, 3, -1], [1, 3, -1]]).all() and np.allclose(p, [0.5, 0.5, 0])
    ids, p, _ = do.moe_router(x, w, 2, bias=[-np.inf] * 5)
    assert (ids == -1).all() and (p == 0).all()
    _, p, _ = do.moe_router(x, w, 2, renormalize=False)
    assert np.allclose(p, 0.2)
    ids, p, _ = do.moe_router(x, w, 2, bias=[0, np.inf, 0, 0, 0])
    assert (ids == [[1, 0], [1, 0]]).all() and np.allclose(p, [1, 0])


def test_experts_against_loops():
    T, H, F, E, k = 2, 24, 16, 3, 2
    gu = [synth.make_problem(2 * F, H, T, w_seed=10 + e, x_seed=1) for e in range(E)]
    dn = [synth.make_problem(H, F, T, w_seed=20 + e, x_seed=1) for e in range(E)]
    x = gu[0][2]
    ids, p = np.array([[2, 0], [-1, 1]]), np.array([[0.75, 0.25], [0.5, 0.5]])
    got = do.moe_experts(x, ids, p, np.stack([g[0] for g in gu]), np.stack([g[1] for g in gu]),
                         np.stack([d[0] for d in dn]), np.stack([d[1] for d in dn]))
    for t in range(T):
        want = [0.0] * H
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            y = oracle.linear_loops(gu[e][0], gu[e][1], x)[t]
            h = [y[f] / (1 + math.exp(-y[f])) * y[F + f] for f in range(F)]
            wd = oracle.dequantize(dn[e][0], dn[e][1])
            for n in range(H):
                want[n] += p[t, j] * sum(wd[n, f] * h[f] for f in range(F))
        assert np.allclose(got[t], want, rtol=1e-11, atol=1e-11)


def test_rotation_keeps_norms_and_relative_angles():
    T, heads, D, rot = 3, 2, 32, 16
    v = _b((T, heads, D), 7)
    w = synth.to_bf16_bits(np.ones(D))
    ang = np.arange(40)[:, None] * 10.0 ** (-np.arange(rot // 2) / 4)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], axis=1)
    for inter in (False, True):
        z0 = do.qk_norm_rope(v, w, cs, [0, 0, 0], interleaved=inter)       # angle 0: the norm alone
        assert np.allclose((z0 ** 2).mean(axis=-1), 1.0, atol=1e-4)
        z = do.qk_norm_rope(v, w, cs, [5, 9, 99], interleaved=inter)
        assert np.isnan(z[2]).all() and np.allclose(z[:2, :, rot:], z0[:2, :, rot:])
        assert np.allclose((z[:2] ** 2).sum(-1), (z0[:2] ** 2).sum(-1))
        # a product of two rotated heads depends on the difference of their positions
        same = np.repeat(v[:1], 3, axis=0)
        r = do.qk_norm_rope(same, w, cs, [3, 10, 17], interleaved=inter)
        assert np.allclose((r[0] * r[1]).sum(-1), (r[1] * r[2]).sum(-1))
