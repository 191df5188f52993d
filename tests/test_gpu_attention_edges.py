"""Calls of the attention operators at their ends: empty tables and caches, many sequences, several passes over cut
sequences, rows of any alignment, calls that overlap on two streams and graphs that share a workspace."""
import numpy as np
import pytest

import oracle
from oracle import attention_ops as ao
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import to_dev, torch, x_to_dev, y_bits
from test_gpu_kv4 import bits, dev, filled
from test_gpu_kv4 import check as check_cache
from test_gpu_prompt_attention import check as check_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def test_empty_tables_caches_and_batches():
    t = torch()
    q = x_to_dev(bits((3, 4, 64), 1))
    lens = dev(np.array([5, 0, 700], dtype=np.int32))
    cache = t.zeros((2, 2, ao.page_bytes(64)), dtype=t.uint8, device="cuda")
    none = t.empty((3, 0), dtype=t.int32, device="cuda")
    assert (q4lin.kv4_attention(q, cache, none, lens) == 0).all()                      # no pages in the table
    assert (q4lin.kv4_attention(q, cache[:0], none, lens) == 0).all()                  # nor in the cache
    table = t.zeros((3, 11), dtype=t.int32, device="cuda")
    assert (q4lin.kv4_attention(q, cache[:0], table, lens) == 0).all()                 # every page is out of range
    assert q4lin.kv4_attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 4, 64)
    k, v = x_to_dev(bits((3, 2, 64), 2)), x_to_dev(bits((3, 2, 64), 3))
    pos = dev(np.zeros(3, dtype=np.int32))
    q4lin.kv4_append(k, v, cache, none, pos)
    assert (cache == 0).all()
    a, b = q4lin.kv4_read(cache, none, pos, 64)
    assert (a == 0).all() and (b == 0).all()
    q4lin.kv4_append(k[:0], v[:0], cache, table, pos[:0])
    cu = dev(np.array([0], dtype=np.int32))
    out = t.full((3, 4, 64), 7.0, dtype=t.bfloat16, device="cuda")
    q4lin.prompt_attention(q, k, v, cu, out=out)                                        # no sequence
    assert (out == 7.0).all()
    assert q4lin.prompt_attention(q[:0], k[:0], v[:0], cu).shape == (0, 4, 64)
    got = q4lin.token_logprobs(t.empty((0, 9), dtype=t.bfloat16, device="cuda"), t.empty((0, 2), dtype=t.int32, device="cuda"), 3)
    assert got[0].shape == (0, 2) and got[2].shape == (0, 3)


@pytest.mark.parametrize("S", [400, 1000])
def test_cache_of_more_sequences_than_threads(S):
    rng = np.random.default_rng(S)
    lengths = [int(x) for x in rng.integers(0, 90, S)]
    cache, table = filled(S, lengths, 2, 1, 64, S)
    q = bits((S, 2, 64), S, 1.5)
    got = q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32)))
    check_cache(y_bits(got), q, cache, table, lengths, 64)


@pytest.mark.parametrize("lengths,n,Hq,Hk,D", [([1300, 5, 640], 8, 8, 1, 128), ([900, 1200], 5, 12, 2, 96), ([2000], 3, 6, 1, 64)])
def test_cut_sequences_in_several_passes(lengths, n, Hq, Hk, D):
    """More than 32 columns, and sequences longer than a share: partial sums of every pass."""
    cache, table = filled(len(lengths), lengths, -(-max(lengths) // 64), Hk, D, n)
    q = bits((len(lengths) * n, Hq, D), n, 1.5)
    got = q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32)))
    check_cache(y_bits(got), q, cache, table, lengths, D)


def test_sequences_that_share_pages():
    """A common prefix stands in one set of pages."""
    lengths = [150, 130, 128]
    cache, table = filled(3, lengths, 3, 2, 64, 4)
    table[1:, :2] = table[0, :2]
    q = bits((3, 4, 64), 4)
    got = q4lin.kv4_attention(x_to_dev(q), dev(cache), dev(table), dev(np.array(lengths, dtype=np.int32)))
    check_cache(y_bits(got), q, cache, table, lengths, 64)


@pytest.mark.parametrize("S,Hq,Hk,D", [(33, 2, 1, 64), (100, 3, 1, 128), (256, 2, 2, 40), (257, 2, 1, 64)])
def test_prompts_of_many_sequences(S, Hq, Hk, D):
    t = torch()
    rng = np.random.default_rng(S)
    lens = [int(x) for x in rng.choice([0, 1, 3, 17, 40, 150], S, p=[0.2, 0.2, 0.3, 0.2, 0.08, 0.02])]
    T = sum(lens)
    q, k, v = bits((T, Hq, D), 1), bits((T, Hk, D), 2), bits((T, Hk, D), 3)
    cu = np.cumsum([0] + lens)
    out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), t.tensor(cu, dtype=t.int32, device="cuda"))
    check_prompt(y_bits(out), q, k, v, cu)


@pytest.mark.parametrize("skip", [0, 8])
def test_prompt_rows_of_any_16_byte_alignment(skip):
    """Outputs whose rows start 16 bytes off a 32-byte boundary, and such as do not."""
    t = torch()
    q, k, v = bits((200, 2, 64), 1), bits((200, 2, 64), 2), bits((200, 2, 64), 3)
    wide = t.full((200, 3 * 64), 7.0, dtype=t.bfloat16, device="cuda")
    out = wide[:, skip:skip + 128].unflatten(1, (2, 64))
    cu = t.tensor([0, 200], dtype=t.int32, device="cuda")
    q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), cu, out=out)
    check_prompt(y_bits(out.contiguous()), q, k, v, [0, 200])
    assert (wide[:, :skip] == 7.0).all() and (wide[:, skip + 128:] == 7.0).all()


def test_values_that_are_not_finite_in_a_long_prompt():
    """A CTA that has met one keeps looking in its later units: every tile's diagonal, with heads in pairs and alone."""
    t = torch()
    for Hq, Hk in ((2, 1), (3, 1)):
        T = 1500
        q, k, v = bits((T, Hq, 64), 1), bits((T, Hk, 64), 2), bits((T, Hk, 64), 3)
        for i in range(60, T, 127):
            v[i, 0, i % 64] = 0x7F80 if i % 2 else 0xFF80
        v[T - 1] = 0x7FC0
        out = q4lin.prompt_attention(x_to_dev(q), x_to_dev(k), x_to_dev(v), t.tensor([0, T], dtype=t.int32, device="cuda"))
        check_prompt(y_bits(out), q, k, v, [0, T])


def test_calls_that_overlap_on_two_streams():
    """Prompts beside the tile route of the layer (both hold tensor memory), cache attention beside itself."""
    t = torch()
    q, k, v = (x_to_dev(bits((1500, h, 128), i)) for i, h in ((1, 4), (2, 2), (3, 2)))
    cu = t.tensor([0, 700, 1500], dtype=t.int32, device="cuda")
    rng = np.random.default_rng(1)
    w, s, x = to_dev(rng.integers(0, 256, (512, 512), dtype=np.uint8),
                     (rng.random((512, 16)) * 0.02).astype(np.float16).view(np.uint16), bits((200, 1024), 5))
    cache, table = filled(4, [900] * 4, 15, 2, 64, 3)
    c, tb, ln = dev(cache), dev(table), dev(np.array([900, 20, 300, 640], dtype=np.int32))
    qd = x_to_dev(bits((4, 4, 64), 1))
    want = q4lin.prompt_attention(q, k, v, cu), q4lin.linear(w, s, x), q4lin.kv4_attention(qd, c, tb, ln)
    t.cuda.synchronize()
    a, b = t.cuda.Stream(), t.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((q4lin.prompt_attention(q, k, v, cu, stream=a), q4lin.linear(w, s, x, stream=b),
                    q4lin.kv4_attention(qd, c, tb, ln, stream=a)))
        got.append((q4lin.prompt_attention(q, k, v, cu, stream=b), q4lin.linear(w, s, x, stream=a),
                    q4lin.kv4_attention(qd, c, tb, ln, stream=b)))
    t.cuda.synchronize()
    for outs in got:
        for o, x in zip(outs, want):
            assert t.equal(o.view(t.int16), x.view(t.int16))


def test_two_graphs_share_a_workspace():
    t = torch()
    cache, table = filled(2, [1200, 700], 19, 2, 64, 3)
    c, tb, ln = dev(cache), dev(table), dev(np.array([1200, 700], dtype=np.int32))
    qs = [x_to_dev(bits((2, 4, 64), 1)), x_to_dev(bits((6, 4, 64), 2))]
    want = [q4lin.kv4_attention(x, c, tb, ln) for x in qs]
    ws = t.empty(max(q4lin.kv4_workspace_bytes(2, n, 4, 2, 64, 19) for n in (1, 3)), dtype=t.uint8, device="cuda")
    outs, graphs = [t.zeros_like(w) for w in want], []
    for x, o in zip(qs, outs):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            q4lin.kv4_attention(x, c, tb, ln, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        ws.fill_(0xFF)
        for g in graphs + graphs[::-1]:
            g.replay()
        t.cuda.synchronize()
        for o, w in zip(outs, want):
            assert t.equal(o.view(t.int16), w.view(t.int16))


@pytest.mark.parametrize("lens,Hq,Hk,D", [([391, 346], 21, 7, 128), ([700, 3, 300], 4, 4, 64), ([600, 401], 6, 3, 96),
                                          ([1100], 3, 1, 40)])
def test_prompts_from_a_cold_cache(lens, Hq, Hk, D):
    """Blocks that arrive late: another buffer, larger than the L2 cache, is written ahead of every call."""
    t = torch()
    T = sum(lens)
    q, k, v = (bits((T, h, D), i, s) for i, h, s in ((1, Hq, 1.5), (2, Hk, 1.0), (3, Hk, 1.0)))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    qd, kd, vd, cd = x_to_dev(q), x_to_dev(k), x_to_dev(v), dev(cu)
    want = q4lin.prompt_attention(qd, kd, vd, cd)
    want = q4lin.prompt_attention(qd, kd, vd, cd)
    check_prompt(y_bits(want), q, k, v, cu)
    other = t.empty(1 << 28, dtype=t.uint8, device="cuda")
    for i in range(20):
        other.fill_(i)
        t.cuda.synchronize()
        assert t.equal(q4lin.prompt_attention(qd, kd, vd, cd).view(t.int16), want.view(t.int16))


def test_cache_and_logits_from_a_cold_cache():
    t = torch()
    cache, table = filled(3, [3000, 40, 1900], 47, 2, 96, 3)
    c, tb, ln = dev(cache), dev(table), dev(np.array([3000, 40, 1900], dtype=np.int32))
    qs = [x_to_dev(bits((3 * n, 6, 96), n)) for n in (1, 4, 9)]
    x = x_to_dev(bits((40, 30011), 5, 3.0))
    tok = t.arange(40, dtype=t.int32, device="cuda")[:, None]
    run = lambda: [q4lin.kv4_attention(q, c, tb, ln) for q in qs] + list(q4lin.token_logprobs(x, tok, 5))
    want = run()
    other = t.empty(1 << 28, dtype=t.uint8, device="cuda")
    for i in range(10):
        other.fill_(i)
        t.cuda.synchronize()
        for a, b in zip(run(), want):
            assert t.equal(a.view(t.int16 if a.dtype == t.bfloat16 else t.int32), b.view(t.int16 if a.dtype == t.bfloat16 else t.int32))


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 1)])
def test_rows_of_prompts_behind_the_4_gib_mark(Hq, Hk):
    """Heads as columns of very wide rows, with values that are not finite (which are fetched again by their addresses)."""
    t = torch()
    T, D, wide = 310, 64, 1 << 23
    cu = np.array([0, 30, 310], dtype=np.int32)
    wq, wk, wv = bits((T, Hq, D), 1), bits((T, Hk, D), 2), bits((T, Hk, D), 3)
    wv[300, 0, 5], wv[40, -1, 60] = 0x7F80, 0x7FC0
    rows = t.empty((T, wide), dtype=t.bfloat16, device="cuda")
    parts, at = [], 8
    for x in (wq, wk, wv, np.zeros_like(wq)):
        part = rows[:, at:at + x.shape[1] * D].unflatten(1, (x.shape[1], D))
        part.copy_(x_to_dev(x))
        parts.append(part)
        at = wide - 40 * D if at == 8 else at + x.shape[1] * D
    q, k, v, out = parts
    assert 256 * wide * 2 == 4 << 30   # rows 256 and on
    got = q4lin.prompt_attention(q, k, v, dev(cu), out=out)
    check_prompt(y_bits(got.contiguous()), wq, wk, wv, cu)
    assert t.equal(q.contiguous().view(t.int16), x_to_dev(wq).view(t.int16))


def test_rows_of_logits_behind_the_4_gib_mark():
    t = torch()
    x = bits((3, 5000), 4, 3.0)
    rows = t.empty((2 * ((1 << 31) + 8) + 5000,), dtype=t.bfloat16, device="cuda").as_strided((3, 5000), ((1 << 31) + 8, 1))
    rows.copy_(x_to_dev(x))
    tok = dev(np.array([[7], [4999], [0]], dtype=np.int32))
    for a, b in zip(q4lin.token_logprobs(rows, tok, 4), q4lin.token_logprobs(x_to_dev(x), tok, 4)):
        assert t.equal(a, b)
