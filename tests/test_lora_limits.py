"""Sizes at the end of LinearLora's range, on the host: what the launches cannot express is refused
by the route query, the workspace query and the entry alike."""
import pytest

from weight_only_bit_q4_gb300 import build as q4build
from weight_only_bit_q4_gb300 import q4lin

from test_operator_args import lora

ROWS = 65535 * 1024   # rows that a grid of 1024-row CTAs reaches


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4lin.load()


@pytest.mark.parametrize("N,ok", [(ROWS, True), (ROWS + 1, False), ((1 << 26) - 1, False), (1 << 26, False)])
@pytest.mark.parametrize("L,R", [(4, 16), (16, 64)])
def test_rows_beyond_the_grid(lib, N, ok, L, R):
    assert q4lin.lora_route(N, 128, 40, R) == (q4lin.ROUTE_TC_SPLITK if ok else -1)
    assert (q4lin.lora_workspace_bytes(N, 128, 40, L, R) > 0) == ok
    if not ok:
        assert lora(lib, N=N, K=128, T=40, L=L, R=R) == 2
