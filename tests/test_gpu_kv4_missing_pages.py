"""Cache attention over long sequences with runs of pages that are not there (freed leading pages, holes longer than a
warp group's ring), at every width of the query: against FP64 over the pages that are there.

Bound: that of test_gpu_kv4.py, over the tokens that are there, taken as they stand in the pages."""
import numpy as np
import pytest

import oracle
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch, x_to_dev, y_bits
from test_gpu_kv4 import bits, dev, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def holes(rng, M, at_start, at_end):
    """A row of M pages: runs of 12 to 40 missing ones (ids below 0 and beyond the pool) between 1 to 4 present ones."""
    row = [-1] * at_start
    while len(row) < M - at_end:
        row += list(rng.integers(0, 12, rng.integers(1, 5))) + [int(rng.choice([-1, 12, -(1 << 31), (1 << 31) - 1]))] * rng.integers(12, 41)
    return row[:M - at_end] + [12] * at_end


def reference(q, cache, table, lengths, Hk, D):
    """(y, sum p |v| / sum p) FP64 [S * n, Hq, D]; every page is decoded once."""
    t = torch()
    P, (S, M) = len(cache), table.shape
    n, Hq = q.shape[0] // S, q.shape[1]
    kv = np.stack([ao.kv4_tokens(cache, np.array([p]), 64, h, D)[:2] for p in range(P) for h in range(Hk)])
    kv = t.from_numpy(kv).cuda().view(P, Hk, 2, 64, D)
    f = t.from_numpy(oracle.bf16_bits_to_f64(q)).cuda().view(S, n, Hk, Hq // Hk, D)
    y, w = t.zeros((2, S, n, Hk, Hq // Hk, D), dtype=t.float64, device="cuda")
    most = 1
    for s in range(S):
        pages = np.flatnonzero((table[s] >= 0) & (table[s] < P))
        at = (pages[:, None] * 64 + np.arange(64)).reshape(-1)
        k, v = kv[t.from_numpy(table[s][pages].astype(np.int64)).cuda()].permute(2, 1, 0, 3, 4).reshape(2, Hk, len(at), D)
        for i in range(n):
            m = int((at < lengths[s] - (n - 1 - i)).sum())
            if m == 0:
                continue
            most = max(most, m)
            p = (t.einsum("hgd,hmd->hgm", f[s, i], k[:, :m]) * D ** -0.5).softmax(-1)
            y[s, i] = t.einsum("hgm,hmd->hgd", p, v[:, :m])
            w[s, i] = t.einsum("hgm,hmd->hgd", p, v[:, :m].abs())
    return y.view(S * n, Hq, D).cpu().numpy(), w.view(S * n, Hq, D).cpu().numpy(), most


@pytest.mark.parametrize("n,Hq,Hk,D", [(4, 7, 1, 64), (17, 1, 1, 64), (3, 9, 1, 96), (1, 64, 2, 128), (9, 8, 1, 64), (2, 8, 1, 128), (1, 4, 1, 64)])
def test_runs_of_missing_pages(n, Hq, Hk, D):
    """Eight sequences of 3200 pages of the table: more than 40 for every group of warps."""
    t = torch()
    S, M = 8, 3200
    rng = np.random.default_rng(n + Hq)
    cache, _ = filled(1, [64], 12, Hk, D, n, extra=0)
    table = np.array([holes(rng, M, *ends) for ends in ((0, 0), (1000, 0), (0, 40), (13, 13), (3199, 0), (3200, 0), (2000, 900), (6, 0))])
    table[4, -1] = 5
    table[7, 6:] = rng.integers(0, 12, M - 6)      # nothing missing behind the sixth page
    table = table.astype(np.int32)
    lengths = np.array([M * 64 - i for i in (0, 1, 63, 64, 5, 0, 700, 9)], dtype=np.int32)
    q = bits((S * n, Hq, D), D, 1.5)
    args = x_to_dev(q), dev(cache), dev(table), dev(lengths)
    got = q4lin.kv4_attention(*args)
    assert q4lin.device_status() == 0
    y, w, most = reference(q, cache, table, lengths, Hk, D)
    f = oracle.bf16_bits_to_f64
    sc = oracle.fp16_bits_to_f64(cache[:, :, 64 * D:].copy().view(np.uint16)).reshape(12 * Hk, 2, -1)
    size = D ** -0.5 * np.abs(f(q)).sum(-1).max() * 15 * sc[:, 0].max()
    off = 2.0 ** -11 + 2 * (size * (D + 8) * 2.0 ** -24 + 2.0 ** -22)
    tol = 2.0 ** -8 * np.abs(y) + off * w + ((most / 8 + 32) * 2.0 ** -24 * 16 + most * 2.0 ** -35) * sc[:, 1].max() + 1e-38
    err = np.abs(f(y_bits(got)) - y)
    assert (err <= tol).all(), np.max(err / tol)
    assert (got[5 * n:6 * n] == 0).all()
    for _ in range(3):
        assert t.equal(q4lin.kv4_attention(*args).view(t.int16), got.view(t.int16))
    assert q4lin.device_status() == 0
