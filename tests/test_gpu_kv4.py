"""The paged 4-bit cache on the GPU: written bytes against the FP64 oracle's exactly, read-back values, and the
attention over it.

Bound of the attention per value y = sum p v / sum p, with W = sum p |v| / sum p: the output's rounding, 2^-8 |y|; each
weight times its token's scale as fp16, 2^-11 W; an exponent off by (D + 8) 2^-24 of the largest scale * sum |q| 15 s
(codes up to 15 before the zero point is taken off), twice; the exponential's 2^-22, twice; FP32 sums of
the products before the zero point is taken off, (len / 8 + 32) 2^-24 of sum p 16 s / sum p; weights 2^-28 below
the largest possible of their page, off by at most 2^-38 of it: len 2^-35 of the largest scale."""
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
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x4B56), n) * std).reshape(shape)


def dev(x):
    return torch().from_numpy(np.ascontiguousarray(x)).cuda()


def noise(shape, seed):
    return np.random.default_rng(seed).integers(0, 256, shape, dtype=np.uint8)


def extremes(x):
    """Rows with values that are not finite, too large or too small for a scale, zeros and exact halves."""
    T = x.shape[0]
    rows = [np.full(x.shape[1:], 0x7F7F, np.uint16), np.zeros(x.shape[1:], np.uint16), np.full(x.shape[1:], 1, np.uint16),
            synth.to_bf16_bits(np.arange(x[0].size).reshape(x.shape[1:]) % 15 * 0.5 - 3.5)]
    for t, r in zip(range(T), rows):
        x[t] = r
    if T > 4:
        x[4, :, 3], x[4, :, -1] = 0x7FC0, 0xFF80
    return x


@pytest.mark.parametrize("T,Hk,D,named", [(1, 1, 64, False), (1, 8, 128, False), (5, 2, 96, False), (70, 1, 128, True),
                                          (200, 2, 64, True), (333, 3, 96, True), (130, 8, 128, True)])
def test_append_writes_the_oracles_bytes_and_reads_them_back(T, Hk, D, named):
    t = torch()
    rng = np.random.default_rng(T + D)
    S, M = (3, 7) if named else (T + 1, 3)
    P = S * M + 2
    table = rng.permutation(P)[:S * M].reshape(S, M).astype(np.int32)
    if named:    # runs of tokens of each sequence, one of them across pages; some are padding
        rows = np.sort(rng.integers(0, S, T)).astype(np.int32)
        pos = np.concatenate([np.arange((rows == s).sum()) + 50 * s for s in range(S)]).astype(np.int32)
        rows[T // 2], pos[T // 3] = -1, -7
        pos[T // 4], rows[T // 5] = M * 64, S
        table[1, 1] = P
    else:
        rows = None
        pos = rng.integers(0, M * 64, T).astype(np.int32)
    ld = 2 * Hk * D + 16
    kv = bits((T, ld), T)
    k, v = kv[:, :Hk * D].reshape(T, Hk, D).copy(), kv[:, Hk * D:2 * Hk * D].reshape(T, Hk, D).copy()
    k, v = extremes(k), extremes(v)[::-1].copy()
    kv[:, :Hk * D], kv[:, Hk * D:2 * Hk * D] = k.reshape(T, -1), v.reshape(T, -1)
    cache = noise((P, Hk, ao.page_bytes(D)), T)
    r = x_to_dev(kv)
    c = dev(cache)
    args = (c, dev(table), dev(pos))
    q4lin.kv4_append(r[:, :Hk * D].unflatten(1, (Hk, D)), r[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D)), *args,
                     rows=None if rows is None else dev(rows))
    ko, vo = t.full((2, T, Hk, D), 7.0, dtype=t.bfloat16, device="cuda")
    q4lin.kv4_read(*args, D, rows=None if rows is None else dev(rows), k=ko, v=vo)
    t.cuda.synchronize()
    out = [y_bits(ko), y_bits(vo)]
    for i in range(T):
        s = i if rows is None else rows[i]
        page = table[s, pos[i] // 64] if 0 <= s < S and 0 <= pos[i] < M * 64 else -1
        for side, x in ((0, k), (1, v)):
            codes, sc = ao.kv4_quantise(x[i])
            if not 0 <= page < P:
                assert (out[side][i] == 0x40E0).all()
                continue
            for h in range(Hk):
                ao.kv4_store(cache, page, h, pos[i] % 64, side, codes[h], sc[h])
            with np.errstate(all="ignore"):
                want = ao.kv4_values(codes, sc)
                nan = np.isnan(want)
                got = oracle.bf16_bits_to_f64(out[side][i])
                assert np.array_equal(np.isnan(got), nan)
                assert (np.abs(got - want)[~nan] <= 2.0 ** -8 * np.abs(want)[~nan]).all()
    got = c.cpu().numpy()
    same = got == cache
    assert same.all(), np.argwhere(~same)[:10]
    a, b = q4lin.kv4_read(*args, D, rows=None if rows is None else dev(rows))
    ok = ko != 7.0
    assert t.equal(a.view(t.int16)[ok], ko.view(t.int16)[ok])


def filled(S, lengths, M, Hk, D, seed, extra=2, std=1.0):
    """A cache whose sequences hold random tokens (whole pages, noise behind their ends), its table and the codes."""
    rng = np.random.default_rng(seed)
    P = S * M + extra
    cache = noise((P, Hk, ao.page_bytes(D)), seed)
    g = -(-D // 64)
    sc = (rng.random((P, Hk, 128 * g)) * 0.3 + 0.02) * std
    cache[:, :, 64 * D:] = sc.astype(np.float16).view(np.uint8).reshape(P, Hk, -1)
    table = rng.permutation(P)[:S * M].reshape(S, M).astype(np.int32)
    return cache, table


def check(got, q, cache, table, lengths, D, scale=None):
    y, w = ao.kv4_attention(q, cache, table, lengths, D, scale)
    f = oracle.bf16_bits_to_f64
    scale = D ** -0.5 if scale is None else scale
    g = -(-D // 64)
    sc = np.abs(oracle.fp16_bits_to_f64(cache[:, :, 64 * D:].copy().view(np.uint16)).reshape(cache.shape[0], -1))
    sc = np.where(np.isfinite(sc), sc, 0)
    k_top, v_top = sc.reshape(len(sc), -1, 2, 64 * g)[:, :, 0].max(), sc.reshape(len(sc), -1, 2, 64 * g)[:, :, 1].max()
    L = max(1, min(int(np.max(lengths)), table.shape[1] * 64))
    with np.errstate(all="ignore"):
        size = abs(scale) * np.where(np.isfinite(f(q)), np.abs(f(q)), 0).sum(-1).max() * 15 * k_top
        off = 2.0 ** -11 + 2 * (size * (D + 8) * 2.0 ** -24 + 2.0 ** -22)
        tol = 2.0 ** -8 * np.abs(y) + off * w + ((L / 8 + 32) * 2.0 ** -24 * 16 + L * 2.0 ** -35) * v_top + 1e-38
    g = f(got)
    fin = np.isfinite(y)
    assert (np.abs(g - y)[fin] <= tol[fin]).all(), np.nanmax(np.abs(g - y)[fin] / tol[fin])
    assert np.array_equal(np.isnan(g), np.isnan(y))


@pytest.mark.parametrize("lengths,n,Hq,Hk,D", [
    ([1], 1, 1, 1, 64), ([64], 1, 8, 1, 128), ([65], 1, 4, 4, 96), ([63, 0, 200], 1, 8, 2, 128), ([130, 7], 1, 5, 1, 64),
    ([1000], 1, 32, 8, 128), ([700, 64, 1, 129, 0, 448, 513], 1, 14, 2, 96), ([300, 3], 4, 28, 4, 96),
    ([200], 8, 8, 8, 64), ([2, 0, 5, 64, 66], 4, 7, 1, 128), ([257, 90], 3, 8, 1, 128), ([150], 16, 9, 3, 64),
    ([1500, 20], 2, 16, 2, 128), ([40] * 30, 1, 4, 2, 64), ([520] * 40, 1, 2, 2, 64), ([64] * 170, 1, 3, 1, 64)])
def test_attention_matches_oracle(lengths, n, Hq, Hk, D):
    t = torch()
    S = len(lengths)
    M = max(1, -(-max(lengths) // 64)) + 1
    cache, table = filled(S, lengths, M, Hk, D, S + n + D)
    q = bits((S * n, (Hq + 1) * D), S + D, 1.5)
    qd = x_to_dev(q)[:, D:].unflatten(1, (Hq, D))
    out = t.full((S * n, Hq + 1, D), 7.0, dtype=t.bfloat16, device="cuda")
    args = dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32))
    q4lin.kv4_attention(qd, *args, out=out[:, :Hq])
    t.cuda.synchronize()
    assert (out[:, Hq] == 7.0).all()
    check(y_bits(out[:, :Hq].contiguous()), q[:, D:].reshape(S * n, Hq, D), cache, table, lengths, D)
    again = q4lin.kv4_attention(qd, *args)
    t.cuda.synchronize()
    assert t.equal(again.view(t.int16), out[:, :Hq].contiguous().view(t.int16))


def test_bad_pages_lengths_and_what_lies_behind_a_sequence():
    """Page ids out of range, lengths beyond the table and below zero; NaN scales behind the ends reach nobody."""
    D, Hk, Hq = 128, 2, 4
    lengths = [200, 1 << 30, -3, 64, 130]
    cache, table = filled(5, lengths, 4, Hk, D, 5)
    table[0, 1], table[1, 3], table[1, 0], table[3, 0], table[4, 2] = -1, 22, 1 << 30, -5, table[4, 2]
    raw = cache[:, :, 64 * D:].view(np.uint16).reshape(len(cache), Hk, 2, 64, 2)
    raw[table[0, 3], :, :, 8:] = 0x7E00       # sequence 0 ends at its fourth page's token 8
    raw[table[4, 2], :, :, 2:] = 0xFC00       # sequence 4 at token 2 of its third
    q = bits((5, Hq, D), 3)
    got = q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32)))
    check(y_bits(got), q, cache, table, lengths, D)
    assert (got[2] == 0).all() and (got[3] == 0).all()


def test_scales_of_every_size_and_values_that_are_not_finite():
    """V scales from fp16's smallest to its largest, in tokens of very different weight; a token of NaN; a zero scale; q from
    1e-30 to 1e4; q with an infinity."""
    D, Hk, Hq, S = 64, 1, 8, 6
    lengths = [300, 300, 70, 300, 128, 90]
    cache, table = filled(S, lengths, 5, Hk, D, 9)
    raw = cache[:, :, 64 * D:].view(np.uint16).reshape(len(cache), Hk, 2, 64)
    tiny = np.array([1, 0, 0x0400, 0x3C00], dtype=np.uint16)
    raw[table[0, :3], 0, 1] = np.tile(tiny, 16)
    raw[table[0, 3:], 0, 1] = 1
    raw[table[1, 1], 0, 1] = 0x7BFF           # 65504 in one page
    raw[table[3, 2], 0, 1, 20] = 0x7FFF       # NaN values, seen by row 3
    raw[table[4, 1], 0, 0, 63] = 0x7FFF       # a NaN key: the last token
    raw[table[2], 0, 1] = 0                   # values of zero
    q = bits((S, Hq, D), 4)
    q[5] = synth.to_bf16_bits(oracle.bf16_bits_to_f64(q[5]) * np.logspace(-30, 3, Hq)[:, None])
    q[5, 0, 1:] = 0
    q[2, 3, 5] = 0x7F80
    got = q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32)))
    y = y_bits(got)
    for s in range(S):      # one by one: the bound goes by the scales of the cache
        only = np.zeros_like(cache)
        only[table[s]] = cache[table[s]]
        check(y[s:s + 1], q[s:s + 1], only, table[s:s + 1], lengths[s:s + 1], D)


def test_a_cache_beyond_32_bits():
    """Records behind the 4 GiB mark are written, read and attended to."""
    t = torch()
    D, Hk = 128, 8
    P = (5 << 30) // (Hk * ao.page_bytes(D))
    cache = t.zeros((P, Hk, ao.page_bytes(D)), dtype=t.uint8, device="cuda")
    table = dev(np.array([[P - 1, 0], [P - 2, P - 3]], dtype=np.int32))
    k, v = bits((140, Hk, D), 1), bits((140, Hk, D), 2)
    rows = dev(np.repeat(np.array([0, 1], dtype=np.int32), 70))
    pos = dev(np.tile(np.arange(70, dtype=np.int32), 2))
    q4lin.kv4_append(x_to_dev(k), x_to_dev(v), cache, table, pos, rows=rows)
    a, b = q4lin.kv4_read(cache, table, pos, D, rows=rows)
    for got, x in ((a, k), (b, v)):
        want = ao.kv4_values(*ao.kv4_quantise(x))
        assert (np.abs(oracle.bf16_bits_to_f64(y_bits(got)) - want) <= 2.0 ** -8 * np.abs(want)).all()
    q = bits((2, 16, D), 3)
    got = q4lin.kv4_attention(x_to_dev(q), cache, table, dev(np.array([70, 70], dtype=np.int32)))
    pages = [P - 1, 0, P - 2, P - 3]
    small = cache[pages].cpu().numpy()
    del cache
    check(y_bits(got), q, small, np.array([[0, 1], [2, 3]]), [70, 70], D)


def test_streams_graph_workspace_and_refusals():
    t = torch()
    D, Hk, Hq, lengths = 64, 2, 6, [900, 30]
    cache, table = filled(2, lengths, 15, Hk, D, 3)
    q, c, tb = x_to_dev(bits((2, Hq, D), 1)), dev(cache), dev(table)
    ln = dev(np.array(lengths, dtype=np.int32))
    want = q4lin.kv4_attention(q, c, tb, ln)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = q4lin.kv4_attention(q, c, tb, ln, stream=s)
    s.synchronize()
    assert t.equal(got, want)
    need = q4lin.kv4_workspace_bytes(2, 1, Hq, Hk, D, 15)
    ws = t.full((need + 256,), 0xFF, dtype=t.uint8, device="cuda")     # (its contents do not matter)
    out, g = t.zeros_like(want), t.cuda.CUDAGraph()
    k, v = x_to_dev(bits((2, Hk, D), 5)), x_to_dev(bits((2, Hk, D), 6))
    pos = dev(np.array([900, 30], dtype=np.int32))
    with t.cuda.graph(g):      # a decode step: append, then attend
        q4lin.kv4_append(k, v, c, tb, pos)
        q4lin.kv4_attention(q, c, tb, ln, out=out, workspace=ws)
    for step in range(70):     # over a page's end
        ln += 1
        g.replay()
        pos += 1
    t.cuda.synchronize()
    assert (ws[need:] == 0xFF).all()
    host = c.cpu().numpy()
    check(y_bits(out), y_bits(q), host, table, [970, 100], D)
    for h in range(Hk):
        kt, _, _ = ao.kv4_tokens(host, table[1], 100, h, D)
        want_k = ao.kv4_values(*ao.kv4_quantise(y_bits(k)[1, h]))
        assert np.array_equal(kt[30:], np.repeat(want_k[None], 70, axis=0))
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(cache=c[:, :, :-16].contiguous()), dict(page_table=tb.long()),
                dict(lengths=ln[:1]), dict(out=out[:1]), dict(workspace=ws[:256]), dict(page_table=tb.cpu())):
        kw = dict(q=q, cache=c, page_table=tb, lengths=ln)
        kw.update(bad)
        with pytest.raises(ValueError):
            q4lin.kv4_attention(**kw)
    with pytest.raises(q4lin.Q4LinError):
        q4lin.kv4_attention(q[:, :5], c, tb, ln)
    for bad in (dict(k=k.float()), dict(v=v[:1]), dict(positions=pos.long()), dict(rows=pos[:1]), dict(cache=c[:, :1].contiguous())):
        kw = dict(k=k, v=v, cache=c, page_table=tb, positions=pos)
        kw.update(bad)
        with pytest.raises(ValueError):
            q4lin.kv4_append(**kw)
    with pytest.raises(ValueError):
        q4lin.kv4_append(*[x_to_dev(bits((3, Hk, D), 1))] * 2, c, tb, dev(np.zeros(3, dtype=np.int32)))
