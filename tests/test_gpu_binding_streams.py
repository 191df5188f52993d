"""Calls on another stream that allocate their own scratch and outputs, while the current stream
takes and fills blocks of the same sizes: the results are those of the same calls alone."""
import pytest

from weight_only_bit_q4_gb300 import q4lin

from gpu_util import to_dev, torch, x_to_dev
from test_gpu_lora import _lib  # noqa: F401  (the fixture)
from test_gpu_lora import problem as lora_problem
from test_gpu_moe import bits, dev
from test_gpu_moe import problem as moe_problem

pytestmark = pytest.mark.gpu


def lora_call(T):
    t = torch()
    p = lora_problem(1000, 2048, T, 6, 32, T)
    args = to_dev(*p[:3]) + (x_to_dev(p[3]), x_to_dev(p[4]), t.from_numpy(p[5]).cuda(), t.from_numpy(p[6]).cuda())
    return lambda stream=None: (q4lin.linear_lora(*args, stream=stream),), q4lin.lora_workspace_bytes(1000, 2048, T, 6, 32)


def linear_call(T):
    p = lora_problem(1000, 2048, T, 1, 8, T)
    args = to_dev(*p[:3])
    return lambda stream=None: (q4lin.linear(*args, stream=stream),), q4lin.workspace_bytes(1000, 2048, T)


def moe_call(T):
    x, gu, gus, dn, dns = moe_problem(T, 512, 256, 16, T)
    args = (x_to_dev(x), x_to_dev(bits((16, 512), 9, 0.1)), dev(gu), dev(gus), dev(dn), dev(dns), 4)
    return lambda stream=None: q4lin.moe(*args, stream=stream), q4lin.moe_workspace_bytes(T, 512, 256, 16, 4)


@pytest.mark.parametrize("make,T", [(lora_call, 1), (lora_call, 9), (lora_call, 100), (linear_call, 8), (moe_call, 2),
                                    (moe_call, 60)])
def test_scratch_and_outputs_of_a_side_stream(make, T):
    t = torch()
    call, need = make(T)
    want = call()
    t.cuda.synchronize()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    got, other = [], []
    for _ in range(40):
        outs = call(side)
        got.append(outs)
        # what the allocator would hand out next on the current stream, were it freed there
        other.append(t.full((need,), 0xFF, dtype=t.uint8, device="cuda"))
        other.append([t.full_like(o, 7) for o in want])
        if len(other) > 8:
            del other[:4]
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    for outs in got:
        for o, w in zip(outs, want):
            assert t.equal(o, w)
