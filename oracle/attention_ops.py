"""CPU FP64 oracle for a decoder's attention and its logits: attention over packed prompts, the
paged 4-bit cache (its quantiser, its layout and the attention over it) and log probabilities.

TEST INFRASTRUCTURE ONLY, like the rest of this package; no code shared with the CUDA
library.  bf16 and fp16 operands come as bit patterns; everything is FP64 on the decoded values.
"""
from __future__ import annotations

import math

import numpy as np

from . import q4_oracle

PAGE = 64


def softmax_rows(scores, values):
    """(softmax(scores) values, softmax(scores) |values|) over the last axis; scores [n], values [n, D]."""
    with np.errstate(all="ignore"):
        p = np.exp(scores - scores.max())
        z = p.sum()
        return p @ values / z, p @ np.abs(values) / z


def prompt_attention(q_bits, k_bits, v_bits, cu, scale=None):
    """(y, spread) FP64 [T, Hq, D]: causal attention within sequences cu[s] .. cu[s + 1]; spread is the same sum over
    |v|.  Rows of no sequence are NaN.  Only the tokens that a row sees enter its sums."""
    q, k, v = (q4_oracle.bf16_bits_to_f64(np.asarray(x)) for x in (q_bits, k_bits, v_bits))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    y, w = np.full((2, T, Hq, D), np.nan)
    for a, b in zip(cu[:-1], cu[1:]):
        for t in range(a, b):
            for h in range(Hq):
                with np.errstate(all="ignore"):
                    s = scale * (k[a:t + 1, h // G] @ q[t, h])
                    y[t, h], w[t, h] = softmax_rows(s, v[a:t + 1, h // G])
    return y, w


def kv4_quantise(x_bits):
    """Codes [..., D] (0..15) and fp16 scale bits [..., ceil(D / 64)] of bf16 values [..., D]."""
    x = q4_oracle.bf16_bits_to_f64(np.asarray(x_bits))
    D = x.shape[-1]
    codes = np.full(x.shape, 8, dtype=np.uint8)
    scales = np.zeros(x.shape[:-1] + (-(-D // 64),), dtype=np.float16)
    for i in range(scales.shape[-1]):
        part = x[..., 64 * i:64 * i + 64]
        with np.errstate(all="ignore"):
            top = np.abs(part).max(axis=-1)
            bad = ~np.isfinite(part).all(axis=-1)
            s = np.where(bad, np.nan, np.minimum(top / 7.0, 65504.0)).astype(np.float16)
            d = s.astype(np.float64)[..., None]
            # (np.rint rounds halves to even)
            q = np.where(d > 0, np.clip(np.rint(np.where(d > 0, part / np.where(d > 0, d, 1.0), 0.0)), -8, 7) + 8, 8)
        codes[..., 64 * i:64 * i + 64] = q
        scales[..., i] = s
    return codes, scales.view(np.uint16)


def kv4_values(codes, scale_bits):
    """FP64 values [..., D] of codes and scales."""
    s = q4_oracle.fp16_bits_to_f64(np.asarray(scale_bits))
    return (codes.astype(np.float64) - 8.0) * np.repeat(s, 64, axis=-1)[..., :codes.shape[-1]]


def page_bytes(D):
    return 64 * D + 256 * -(-D // 64)


def places(D, o):
    """Where token o of a page stands in its record: for every value i of K and of V the byte and the shift of its
    code, and the byte of every group's K and V scale."""
    kb, vb, sh = [], [], []
    for i in range(D):
        block, n = divmod(i, 8)
        j, c = divmod(block, 4)
        kb.append(o * (D // 2) + 4 * (c * (D // 32) + j) + n // 2)
        vb.append(32 * D + (i // 2) * 64 + 16 * (o % 8 // 2) + 4 * (o // 16) + 2 * (o % 2) + o % 16 // 8)
        sh.append(4 * (i % 2))
    g = -(-D // 64)
    ks = [64 * D + 2 * (o * g + i) for i in range(g)]
    vs = [64 * D + 128 * g + 2 * (o * g + i) for i in range(g)]
    return kb, vb, sh, ks, vs


def kv4_store(cache, page, h, o, side, codes, scale_bits):
    """One token's codes [D] and scales of a head into the cache (uint8 [pages, Hk, page_bytes]); side 0 K, 1 V."""
    kb, vb, sh, ks, vs = places(len(codes), o)
    rec = cache[page, h]
    for b, n, q in zip((kb, vb)[side], sh, codes):
        rec[b] = (rec[b] & (0xF0 >> n)) | (int(q) << n)
    for b, s in zip((ks, vs)[side], scale_bits):
        rec[b], rec[b + 1] = int(s) & 0xFF, int(s) >> 8


def kv4_load(cache, page, h, o, side, D):
    """Codes [D] and scale bits of one token and head."""
    kb, vb, sh, ks, vs = places(D, o)
    rec = cache[page, h].astype(int)
    codes = np.array([rec[b] >> n & 15 for b, n in zip((kb, vb)[side], sh)], dtype=np.uint8)
    return codes, np.array([rec[b] | rec[b + 1] << 8 for b in (ks, vs)[side]], dtype=np.uint16)


def kv4_tokens(cache, table_row, n, h, D):
    """(K, V, known) of the first n tokens of a sequence: FP64 [n, D] twice; known: the token's page is there."""
    k, v = np.zeros((2, n, D))
    known = np.zeros(n, dtype=bool)
    for i in range(-(-n // PAGE)):
        page, m = int(table_row[i]), min(PAGE, n - i * PAGE)
        if not 0 <= page < cache.shape[0]:
            continue
        known[i * PAGE:i * PAGE + m] = True
        for side, out in ((0, k), (1, v)):
            got = [kv4_load(cache, page, h, o, side, D) for o in range(m)]
            out[i * PAGE:i * PAGE + m] = kv4_values(np.array([c for c, _ in got]), np.array([s for _, s in got]))
    return k, v, known


def kv4_attention(q_bits, cache, table, lengths, D, scale=None):
    """(y, spread) FP64 [S * n, Hq, D] over the paged cache; a token that sees nothing gives zeros."""
    q = q4_oracle.bf16_bits_to_f64(np.asarray(q_bits))
    T, Hq, _ = q.shape
    S, M = table.shape
    n, Hk = T // S, cache.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    y, w = np.zeros((2, T, Hq, D))
    for s in range(S):
        L = min(max(int(lengths[s]), 0), M * PAGE)
        for h in range(Hk):
            k, v, known = kv4_tokens(cache, table[s], L, h, D)
            for i in range(n):
                seen = known & (np.arange(L) < L - n + 1 + i)
                if not seen.any():
                    continue
                for hq in range(h * G, (h + 1) * G):
                    with np.errstate(all="ignore"):
                        y[s * n + i, hq], w[s * n + i, hq] = softmax_rows(scale * (k[seen] @ q[s * n + i, hq]), v[seen])
    return y, w


def token_logprobs(x, targets, top_k):
    """(logprobs [T, n], entropy [T], ids [T, k], top logprobs [T, k]) of FP64 logits [T, V]."""
    T, V = x.shape
    targets = np.asarray(targets).reshape(T, -1)
    logp, entropy = np.zeros(targets.shape), np.zeros(T)
    ids, top = np.full((T, top_k), -1), np.full((T, top_k), -np.inf)
    for t in range(T):
        row = x[t]
        can = [v for v in range(V) if row[v] > -np.inf]      # (NaN is not)
        order = sorted(can, key=lambda v: (-row[v], v))[:top_k]
        if np.isnan(row).any():
            logs = np.full(V, np.nan)
            entropy[t] = np.nan
        elif not can:
            logs = np.full(V, -np.inf)
        else:
            m = row.max()
            with np.errstate(all="ignore"):
                d = np.where(row == m, 0.0, row - m)
                logs = d - math.log(np.exp(d).sum())
                p = np.exp(logs)
                entropy[t] = -np.where(p > 0, p * logs, 0.0).sum()
        for j, v in enumerate(targets[t]):
            logp[t, j] = logs[v] if 0 <= v < V else 0.0
        for j, v in enumerate(order):
            ids[t, j], top[t, j] = v, logs[v]
    return logp, entropy, ids, top
