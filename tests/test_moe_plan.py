"""What the expert layer plans before it launches anything: columns too long for shared memory are
refused by every entry in the same way, whatever T, and by nothing that the header does not name."""
import pytest

from weight_only_bit_q4_gb300 import build as q4build
from weight_only_bit_q4_gb300 import q4lin

from test_operator_args import P

LIMIT = 48000   # include/q4lin.h


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4lin.load()


def moe(lib, T, H, F, E, k):
    return lib.q4lin_moe(P, P, None, P, P, P, P, P, P, P, T, H, F, E, k, 1, P, None)


def experts(lib, T, H, F, E, k):
    return lib.q4lin_moe_experts(P, P, P, P, P, P, P, P, T, H, F, E, k, P, None)


@pytest.mark.parametrize("T", [1, 4, 64, 70, 1000])
@pytest.mark.parametrize("E,k", [(2, 1), (8, 2), (1024, 8), (1024, 16)])
def test_columns_beyond_shared_memory_are_refused_before_any_launch(lib, T, E, k):
    H = 1 << 17
    for call in (moe, experts):
        assert call(lib, T, H, 8, E, k) == 2
        assert "shared memory" in q4lin.last_error_detail()
    assert q4lin.moe_workspace_bytes(T, H, 8, E, k) == 0


@pytest.mark.parametrize("T", [1, 2, 4, 16, 17, 64, 70, 1000])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (8, 2), (64, 8), (128, 8), (1000, 5), (1024, 16)])
def test_sizes_up_to_the_limit_are_planned(lib, T, E, k):
    for H in (8, 2048, 28672, 38912, LIMIT):
        for F in (8, 768, 14336, 32768, 65536):
            if E * max(2 * F, H) < 1 << 31:
                assert q4lin.moe_workspace_bytes(T, H, F, E, k) > 0, (T, H, F, E, k)
