"""The expert kernels' forms on both sides of the rules that choose them: more than 16 choices
with few and with many items per CTA in either product (K shared by warps, or not), one and two
token tiles together, K ranges of a single copy, odd sizes.  Bound as for the layer everywhere
(8e-3 |y| + 1e-3 rms(y)); the same bits call after call."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import assert_close, torch, x_to_dev, y_bits
from test_gpu_moe import _lib, dev, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

SHAPES = [(64, 2560, 1280, 8, 2), (40, 2440, 1224, 8, 3), (19, 584, 1944, 9, 6), (64, 520, 2008, 10, 4), (20, 4096, 40, 16, 2),
          (16, 4104, 264, 8, 2), (17, 2048, 768, 20, 1), (24, 240, 1016, 60, 2), (40, 64, 2048, 33, 3)]


@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
def test_experts_match_oracle(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[T // 2, 0] = -1
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    args = (x_to_dev(x), t.from_numpy(ids).cuda(), t.from_numpy(p).cuda(), dev(gu), dev(gus), dev(dn), dev(dns))
    y = q4lin.moe_experts(*args)
    t.cuda.synchronize()
    assert_close(y_bits(y), do.moe_experts(x, ids, p, gu, gus, dn, dns), f"T={T} H={H} F={F} E={E} k={k}")
    again = [q4lin.moe_experts(*args) for _ in range(10)]
    t.cuda.synchronize()
    assert all(t.equal(a.view(t.int16), y.view(t.int16)) for a in again)


@pytest.mark.parametrize("T,E,H,k", [(4, 5, 40, 2), (5, 20, 264, 3), (8, 128, 2048, 8), (9, 17, 1992, 4), (33, 300, 512, 16), (64, 1024, 104, 5)])
def test_router_of_four_tokens_and_more(T, E, H, k):
    t = torch()
    rng = np.random.default_rng(E)
    x = rng.standard_normal((T, H)).astype(np.float32)
    w = (rng.standard_normal((E, H)) * H ** -0.5).astype(np.float32)
    xb, wb = t.from_numpy(x).bfloat16(), t.from_numpy(w).bfloat16()
    bias = rng.standard_normal(E).astype(np.float32)
    bias[E // 2] = -np.inf
    ids, p = q4lin.moe_router(xb.cuda(), wb.cuda(), k, bias=t.from_numpy(bias).cuda())
    t.cuda.synchronize()
    bits = lambda b: b.view(t.int16).numpy().view(np.uint16)   # noqa: E731
    want_ids, want_p, logits = do.moe_router(bits(xb), bits(wb), k, bias)
    ids, p = ids.cpu().numpy(), p.cpu().numpy()
    best = np.take_along_axis(logits, want_ids, axis=1)
    got = np.take_along_axis(logits, ids, axis=1)
    assert (ids >= 0).all() and np.abs(got - best).max() < 1e-4   # FP32 sums may swap closer logits
    same = ids == want_ids
    assert np.allclose(p[same], want_p[same], rtol=3e-4)
    assert all(len(set(r)) == k for r in ids.tolist()) and (ids != E // 2).all()
