"""The choices of a token are added in order, in FP32, in every form.  Four choices of one expert
with weights 2^30, 1, -2^30, 1 give its output once in that order (2^30 o + o is 2^30 o), twice where
the even and the odd ones are added apart."""
import pytest

from weight_only_bit_q4_gb300 import q4lin

from gpu_util import torch, x_to_dev
from test_gpu_moe import _lib, dev, problem  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,F,E", [(1, 264, 136, 3), (4, 512, 256, 2), (5, 264, 136, 3), (70, 4096, 264, 20), (6, 40, 14336, 2)])
def test_choices_are_added_in_order(T, H, F, E):
    t = torch()
    x, gu, gus, dn, dns = problem(T, H, F, E, T)
    args = (dev(gu), dev(gus), dev(dn), dev(dns))
    ids = (t.arange(T, device="cuda", dtype=t.int32) % E)[:, None].repeat(1, 4)

    def run(*p):
        return q4lin.moe_experts(x_to_dev(x), ids, t.tensor([p] * T, device="cuda"), *args).view(t.int16)
    once = run(1.0, 0.0, 0.0, 0.0)
    assert not t.equal(once, run(2.0, 0.0, 0.0, 0.0))
    assert t.equal(run(2.0**30, 1.0, -2.0**30, 1.0), once)
    assert bool((run(1.0, 2.0**30, -2.0**30, 0.0) == 0).all())   # (the first is lost in the second)
