"""The router on weights that the call before it in the stream has just written, a projection of
this library among the writers (its kernels let the next one start early): every call must see the
weights of its own turn.  Compared bit by bit with calls whose weights lay there long before."""
import pytest

from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import to_dev, torch, x_to_dev
from test_gpu_moe import _lib, bits  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

ROUNDS = 60


@pytest.mark.parametrize("T,E,H", [(1, 64, 2048), (2, 24, 512), (5, 128, 2048), (64, 100, 1032)])
def test_weights_written_by_the_call_before(T, E, H):
    t = torch()
    k = 4
    wq, s, xa = synth.make_problem(H, 512, E, w_seed=5, x_seed=6)
    wq, s, xa = to_dev(wq, s, xa)
    sources = [xa, x_to_dev(bits((E, 512), 7, 1.0))]   # w_router = this library's projection of one of them
    x = x_to_dev(bits((T, H), 8, 1.0))
    ws = t.empty(max(q4lin.workspace_bytes(H, 512, E), 256), dtype=t.uint8, device="cuda")
    want = []
    for src in sources:
        w = q4lin.linear(wq, s, src, workspace=ws)
        t.cuda.synchronize()
        want.append(q4lin.moe_router(x, w, k))
        t.cuda.synchronize()
    assert not t.equal(want[0][0], want[1][0])
    w = t.empty((E, H), dtype=t.bfloat16, device="cuda")
    got = []
    for r in range(ROUNDS):
        q4lin.linear(wq, s, sources[r % 2], y=w, workspace=ws)
        got.append(q4lin.moe_router(x, w, k))
    for r in range(ROUNDS):   # and by a kernel that knows nothing of early starts
        w.copy_(q4lin.linear(wq, s, sources[r % 2], workspace=ws))
        got.append(q4lin.moe_router(x, w, k))
    t.cuda.synchronize()
    for r, (ids, p) in enumerate(got):
        assert t.equal(ids, want[r % 2][0]) and t.equal(p, want[r % 2][1]), r
