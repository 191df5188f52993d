"""The streaming routes (1 to 32 tokens) give the same bits call after call, every format and
LinearLora, with calls back to back: a ring stage refilled before a warp has read it would show
as rows that differ now and then.  T = 1, 4: the GEMV; 8, 13, 32: warp-MMA."""
import pytest

from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import to_dev, torch, x_to_dev
from test_gpu_formats import _dev
from test_gpu_lora import _lib, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

CALLS = 100


def repeat(call):
    t = torch()
    ys = [call().view(t.int16) for _ in range(CALLS)]
    t.cuda.synchronize()
    differing = [i for i, y in enumerate(ys) if not t.equal(y, ys[0])]
    assert not differing, f"calls {differing[:8]} differ from the first"


@pytest.mark.parametrize("T", [1, 4, 8, 13, 32])
@pytest.mark.parametrize("qtype", ["q4g64", "q5g64", "q6g64", "w8g32"])
def test_formats(qtype, T):
    t = torch()
    N, K = 6144, 5120
    if qtype == "q4g64":
        d = to_dev(*synth.make_problem(N, K, T, w_seed=1, x_seed=2))
        repeat(lambda: q4lin.linear(*d))
        return
    planes, s, x = synth.make_problem_fmt(qtype, N, K, T, w_seed=1, x_seed=2)
    planes, s, x = tuple(_dev(p) for p in planes), _dev(s), _dev(x).view(t.bfloat16)
    repeat(lambda: q4lin.linear_qtype(qtype, planes, s, x))


@pytest.mark.parametrize("T", [1, 8])
def test_fused_forms(T):
    N, K = 5120, 4104
    d = to_dev(*synth.make_problem(N, K, T, w_seed=3, x_seed=4))
    r = q4lin.linear(*d)
    repeat(lambda: q4lin.linear_add(*d, r))
    repeat(lambda: q4lin.linear_swiglu(*d))


@pytest.mark.parametrize("T,L,R", [(1, 4, 16), (1, 2, 256), (4, 3, 16), (8, 9, 32), (13, 24, 32), (32, 4, 64)])
def test_linear_lora(T, L, R):
    t = torch()
    p = problem(6000, 4104, T, L, R, 3)
    args = to_dev(*p[:3]) + (x_to_dev(p[3]), x_to_dev(p[4]), t.from_numpy(p[5]).cuda(), t.from_numpy(p[6]).cuda())
    ws = t.empty(q4lin.lora_workspace_bytes(6000, 4104, T, L, R), dtype=t.uint8, device="cuda")
    repeat(lambda: q4lin.linear_lora(*args, workspace=ws))
