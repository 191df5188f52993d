"""The mixture-of-experts layer on the GPU against the FP64 oracle.

y within the layer's bound (8e-3 |y| + 1e-3 rms(y)).  Router weights: FP32 sums of H exact
products (each partial sum within 2^-24 relative of the running magnitude, at most about
sqrt(H) 2^-24 |x||w| = 1e-5 on logits of a few units) through exp: 1e-4 relative.
"""
import numpy as np
import pytest

from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import assert_close, torch, x_to_dev, y_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def bits(shape, seed, std):
    n = int(np.prod(shape))
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x4D6F), n) * std).reshape(shape)


def planes(E, rows, K, seed):
    Kp = (K + 127) // 128 * 128
    wq = synth.packed_codes(E * rows, Kp, seed).reshape(E, rows, Kp // 2)
    s = synth.group_scales(E * rows, Kp, seed).reshape(E, rows, Kp // 64)
    return wq, s


def poison_padding(s, K):
    """NaN scale bits in the groups that hold no column < K."""
    s = s.copy()
    s[..., (K + 63) // 64:] = 0x7E00
    return s


def dev(a):
    t = torch()
    a = np.ascontiguousarray(a)
    return t.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def problem(T, H, F, E, seed):
    gu, gus = planes(E, 2 * F, H, seed)
    dn, dns = planes(E, H, F, seed + 1)
    return bits((T, H), seed + 2, 1.0), gu, poison_padding(gus, H), dn, poison_padding(dns, F)


SHAPES = [(1, 2048, 768, 16, 8), (1, 8, 8, 1, 1), (3, 264, 136, 5, 2), (8, 512, 256, 8, 2), (9, 1992, 1016, 6, 3),
          (16, 256, 72, 4, 4), (19, 648, 520, 20, 3), (33, 512, 128, 3, 2), (64, 1024, 256, 40, 8), (65, 136, 64, 4, 8),
          (130, 64, 40, 2, 1), (40, 80, 24, 100, 16), (2, 5120, 1408, 4, 2)]


@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
def test_experts_match_oracle(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    args = (x_to_dev(x), dev(ids), dev(p), dev(gu), dev(gus), dev(dn), dev(dns))
    y = q4lin.moe_experts(*args)
    t.cuda.synchronize()
    want = do.moe_experts(x, ids, p, gu, gus, dn, dns)
    assert_close(y_bits(y), want, f"moe T={T} H={H} F={F} E={E} k={k}")
    assert np.array_equal(y_bits(q4lin.moe_experts(*args)), y_bits(y))   # deterministic


def test_choices_that_add_nothing_and_duplicates():
    t = torch()
    T, H, F, E, k = 12, 264, 136, 4, 3
    x, gu, gus, dn, dns = problem(T, H, F, E, 77)
    rng = np.random.default_rng(1)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)       # duplicates among a token's choices
    ids[3] = -1                                             # a token without any: +0
    ids[4] = [E, 1 << 30, -(1 << 31)]
    ids[5, 1] = -7
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    p[3:5] = np.nan                                         # their weights are not used
    p[5, 1] = np.inf
    y = q4lin.moe_experts(x_to_dev(x), dev(ids), dev(p), dev(gu), dev(gus), dev(dn), dev(dns))
    t.cuda.synchronize()
    assert (y_bits(y)[3:5] == 0).all()
    assert_close(y_bits(y), do.moe_experts(x, ids, p, gu, gus, dn, dns), "partial choices")


def test_all_tokens_on_one_expert():
    t = torch()
    T, H, F, E, k = 64, 256, 128, 32, 2
    x, gu, gus, dn, dns = problem(T, H, F, E, 5)
    ids = np.full((T, k), 7, dtype=np.int32)                # both choices too
    p = np.full((T, k), 0.5, dtype=np.float32)
    y = q4lin.moe_experts(x_to_dev(x), dev(ids), dev(p), dev(gu), dev(gus), dev(dn), dev(dns))
    t.cuda.synchronize()
    assert_close(y_bits(y), do.moe_experts(x, ids, p, gu, gus, dn, dns), "one expert")


def near_ties(logits, k):
    top = -np.sort(-logits, axis=1)[:, :k + 1]
    return (np.diff(-top, axis=1) < 1e-4).any(axis=1)


@pytest.mark.parametrize("T,H,E,k,renorm", [(1, 2048, 128, 8, True), (2, 72, 3, 3, False), (5, 520, 64, 1, True),
                                            (37, 1024, 40, 5, False), (64, 2048, 128, 8, True), (4, 8, 1, 1, True),
                                            (9, 264, 1000, 16, False), (300, 64, 33, 4, True)])
def test_router_matches_oracle(T, H, E, k, renorm):
    t = torch()
    x, w = bits((T, H), T + E, 1.0), bits((E, H), T + E + 1, 2.0 * H ** -0.5)
    ids, p = q4lin.moe_router(x_to_dev(x), x_to_dev(w), k, renormalize=renorm)
    t.cuda.synchronize()
    want, wp, logits = do.moe_router(x, w, k, renormalize=renorm)
    clear = ~near_ties(logits, k)
    assert clear.sum() >= T // 2
    assert np.array_equal(ids.cpu().numpy()[clear], want[clear])
    assert np.allclose(p.cpu().numpy()[clear], wp[clear], rtol=1e-4, atol=1e-7)


def test_router_ties_masks_and_infinities():
    t = torch()
    x = bits((3, 64), 3, 1.0)
    w = np.repeat(bits((1, 64), 4, 0.2), 70, axis=0)         # equal experts: the lowest first
    xd, wd = x_to_dev(x), x_to_dev(w)
    ids, p = q4lin.moe_router(xd, wd, 4)
    assert (ids.cpu().numpy() == [0, 1, 2, 3]).all() and np.allclose(p.cpu().numpy(), 0.25)
    inf = float("inf")
    for bias, renorm in (([-inf] * 70, True), ([-inf] * 68 + [0.0, float("nan")], False),
                         ([0.0] * 35 + [inf] + [0.0] * 34, True), ([0.0] * 69 + [inf], False),
                         ([-inf] * 60 + [1.0, 2.0, 3.0] + [-inf] * 7, True)):
        b = t.tensor(bias, dtype=t.float32, device="cuda")
        ids, p = q4lin.moe_router(xd, wd, 4, bias=b, renormalize=renorm)
        want, wp, _ = do.moe_router(x, w, 4, bias=bias, renormalize=renorm)
        assert np.array_equal(ids.cpu().numpy(), want)
        assert np.allclose(p.cpu().numpy(), wp, rtol=1e-4, atol=1e-7)


@pytest.mark.parametrize("T,H,F,E,k", [(1, 512, 256, 16, 4), (21, 264, 136, 12, 3)])
def test_whole_layer_stream_window_and_graph(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, 50 + T)
    w = bits((E, H), 9, 2.0 * H ** -0.5)
    ids_ref, p_ref, logits = do.moe_router(x, w, k)
    assert not near_ties(logits, k).any()
    xd, wd = x_to_dev(x), x_to_dev(w)
    pl = (dev(gu), dev(gus), dev(dn), dev(dns))
    buf = t.full((512 + T * H + 512,), -3.0, dtype=t.bfloat16, device="cuda")
    y = buf[512:512 + T * H].view(T, H)
    ws = t.empty(q4lin.moe_workspace_bytes(T, H, F, E, k), dtype=t.uint8, device="cuda")
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    ids, p = t.empty((T, k), dtype=t.int32, device="cuda"), t.empty((T, k), device="cuda")
    for _ in range(10):   # calls chained on one workspace
        q4lin.moe(xd, wd, *pl, k, y=y, ids=ids, weights=p, workspace=ws, stream=stream)
    stream.synchronize()
    want = do.moe_experts(x, ids_ref, p_ref, gu, gus, dn, dns)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert_close(y_bits(y), want, "whole layer")
    assert bool((buf[:512] == -3.0).all()) and bool((buf[512 + T * H:] == -3.0).all())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        q4lin.moe(xd, wd, *pl, k, y=y, ids=ids, weights=p, workspace=ws)
    x2 = bits((T, H), 4242, 1.0)
    xd.copy_(x_to_dev(x2))
    g.replay()
    t.cuda.synchronize()
    i2, p2, l2 = do.moe_router(x2, w, k)
    if not near_ties(l2, k).any():
        assert_close(y_bits(y), do.moe_experts(x2, i2, p2, gu, gus, dn, dns), "replay")


def test_empty_intermediate_and_wrapper_refusals():
    t = torch()
    x, gu, gus, dn, dns = problem(2, 64, 128, 4, 1)
    ids, p = t.zeros((2, 2), dtype=t.int32, device="cuda"), t.ones((2, 2), device="cuda")
    y = t.ones((2, 64), dtype=t.bfloat16, device="cuda")
    st = q4lin.load().q4lin_moe_experts(None, None, None, None, None, None, None, y.data_ptr(), 2, 64, 0, 4, 2, None, None)
    t.cuda.synchronize()
    assert st == 0 and (y_bits(y) == 0).all()
    args = [x_to_dev(x), ids, p, dev(gu), dev(gus), dev(dn), dev(dns)]
    for i, bad in ((1, ids.long()), (2, p.half()), (3, dev(gu[:, :-1])), (5, dev(dn[:, :32])), (0, x_to_dev(x).float())):
        q = list(args)
        q[i] = bad
        with pytest.raises(ValueError):
            q4lin.moe_experts(*q)
