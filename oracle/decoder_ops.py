"""CPU FP64 oracle for the operators around the projections of a decoder block:
low-rank adapters beside a shared Q4 projection, the mixture-of-experts layer with Q4
experts and its router, and the head norms with the position rotation.

TEST INFRASTRUCTURE ONLY, like the rest of this package; no code shared with the CUDA
library.  Everything is FP64 on the decoded operands.
"""
from __future__ import annotations

import numpy as np

from . import fused_ops, q4_oracle


def linear_lora(wq, scale_bits, x_bits, a_bits, b_bits, ids, adapter_scales=None, ranks=None):
    """y_ref [T, N] = W x + sc_a B_a (A_a x); ids outside [0, L): the projection alone."""
    y = q4_oracle.linear(wq, scale_bits, x_bits).copy()
    x = q4_oracle.bf16_bits_to_f64(np.asarray(x_bits))
    L, R = np.asarray(a_bits).shape[:2]
    for t, i in enumerate(np.asarray(ids)):
        if not 0 <= i < L:
            continue
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        A = q4_oracle.bf16_bits_to_f64(np.asarray(a_bits)[i, :r])
        B = q4_oracle.bf16_bits_to_f64(np.asarray(b_bits)[i, :, :r])
        sc = 1.0 if adapter_scales is None else float(adapter_scales[i])
        y[t] += sc * (B @ (A @ x[t]))
    return y


def moe_router(x_bits, w_bits, top_k, bias=None, renormalize=True):
    """(ids [T, k], weights [T, k], logits [T, E]): the experts with the largest logits, largest
    first, ties by the lowest expert; -inf and NaN are never chosen (id -1, weight 0)."""
    x = q4_oracle.bf16_bits_to_f64(np.asarray(x_bits))
    w = q4_oracle.bf16_bits_to_f64(np.asarray(w_bits))
    logits = x @ w.T
    if bias is not None:
        logits = logits + np.asarray(bias, dtype=np.float64)
    T, E = logits.shape
    ids = np.full((T, top_k), -1, dtype=np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        can = [e for e in range(E) if logits[t, e] > -np.inf]
        if not can:
            continue
        m = max(logits[t, e] for e in can)
        ex = {e: 1.0 if logits[t, e] == m else float(np.exp(logits[t, e] - m)) for e in can}
        pick = sorted(can, key=lambda e: (-logits[t, e], e))[:top_k]
        z = sum(ex[e] for e in pick) if renormalize else sum(ex.values())
        for j, e in enumerate(pick):
            ids[t, j] = e
            weights[t, j] = ex[e] / z
    return ids, weights, logits


def moe_experts(x_bits, ids, weights, wq_gu, s_gu, wq_dn, s_dn):
    """y_ref [T, H] = sum_j weights[t, j] W_down,e (silu(gate) * up), ids outside [0, E) left out."""
    x_bits, ids = np.asarray(x_bits), np.asarray(ids)
    T, H = x_bits.shape
    E, F2 = np.asarray(wq_gu).shape[:2]
    F = F2 // 2
    y = np.zeros((T, H))
    for e in range(E):
        hit = [(t, j) for t in range(T) for j in range(ids.shape[1]) if ids[t, j] == e]
        if not hit:
            continue
        rows = sorted({t for t, _ in hit})
        gu = q4_oracle.linear(wq_gu[e], s_gu[e], x_bits[rows])
        h = fused_ops.silu(gu[:, :F]) * gu[:, F:]
        o = h @ q4_oracle.dequantize(*q4_oracle.logical_planes(wq_dn[e], s_dn[e], F)).T
        for t, j in hit:
            y[t] += float(weights[t, j]) * o[rows.index(t)]
    return y


def qk_norm_rope(v_bits, w_bits, cos_sin, positions, eps=1e-6, interleaved=False):
    """One side: v [T, heads, D] bf16 bits -> FP64 [T, heads, D]; tokens outside the table are NaN."""
    v = q4_oracle.bf16_bits_to_f64(np.asarray(v_bits))
    w = q4_oracle.bf16_bits_to_f64(np.asarray(w_bits))
    T, heads, D = v.shape
    P, rot = np.asarray(cos_sin).shape
    half = rot // 2
    z = v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps) * w
    out = z.copy()
    for t, p in enumerate(np.asarray(positions)):
        if not 0 <= p < P:
            out[t] = np.nan
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(cos_sin[p, i]), float(cos_sin[p, half + i])
            out[t, :, a] = z[t, :, a] * c - z[t, :, b] * s
            out[t, :, b] = z[t, :, b] * c + z[t, :, a] * s
    return out
