"""The expert layer at long H (the first product's columns near what shared memory holds, in the
form that the many choices would not take otherwise), and the whole layer over several passes with a
short last one.  Bound as for the layer everywhere (8e-3 |y| + 1e-3 rms(y)); router weights 1e-4."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin

from gpu_util import assert_close, torch, x_to_dev, y_bits
from test_gpu_moe import _lib, bits, dev, near_ties, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,F,E,k", [(64, 38912, 8, 8, 2), (3, 48000, 16, 2, 2), (1, 28672, 24, 3, 1)])
def test_long_hidden_sizes(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    p = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    y = q4lin.moe_experts(x_to_dev(x), t.from_numpy(ids).cuda(), t.from_numpy(p).cuda(), dev(gu), dev(gus), dev(dn), dev(dns))
    t.cuda.synchronize()
    assert_close(y_bits(y), do.moe_experts(x, ids, p, gu, gus, dn, dns), f"T={T} H={H} F={F} E={E} k={k}")


# passes of 512 / k tokens: 64 + 6, 4 x 32 + 2, 512 + 8, 170 + 170 + 1 (a latency-form last one among them)
@pytest.mark.parametrize("T,H,F,E,k", [(70, 136, 72, 12, 8), (130, 264, 136, 40, 16), (520, 64, 40, 5, 1), (341, 72, 520, 6, 3)])
def test_whole_layer_over_several_passes(T, H, F, E, k):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T + H)
    w = bits((E, H), T, 2.0 * H ** -0.5)
    args = (x_to_dev(x), x_to_dev(w), dev(gu), dev(gus), dev(dn), dev(dns), k)
    ws = t.empty(q4lin.moe_workspace_bytes(T, H, F, E, k), dtype=t.uint8, device="cuda")
    outs = [q4lin.moe(*args, workspace=ws) for _ in range(5)]
    t.cuda.synchronize()
    y, ids, p = outs[0]
    want_ids, want_p, logits = do.moe_router(x, w, k)
    clear = ~near_ties(logits, k)
    ids_h, p_h = ids.cpu().numpy(), p.cpu().numpy()
    assert clear.sum() > T // 2 and np.array_equal(ids_h[clear], want_ids[clear])
    assert np.allclose(p_h[clear], want_p[clear], rtol=1e-4, atol=1e-7)
    assert_close(y_bits(y), do.moe_experts(x, ids_h, p_h, gu, gus, dn, dns), f"passes T={T} k={k}")
    for o in outs[1:]:
        assert all(t.equal(a.view(t.int16) if a.dtype == t.bfloat16 else a, b.view(t.int16) if b.dtype == t.bfloat16 else b)
                   for a, b in zip(o, outs[0]))
