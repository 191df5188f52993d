"""Host-side refusals and size queries of the operators around the projections: no GPU, the
fake pointers are never dereferenced."""
import ctypes

import pytest

from weight_only_bit_q4_gb300 import build as q4build
from weight_only_bit_q4_gb300 import q4lin

P = 256   # an aligned, non-null address


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4lin.load()


def lora(lib, N=64, K=128, T=2, L=3, R=8, wq=P, s=P, x=P, a=P, b=P, ids=P, sc=P, ranks=P, y=P, ws=P):
    return lib.q4lin_linear_lora(wq, s, x, a, b, ids, sc, ranks, y, N, K, T, L, R, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(K=-8), 1), (dict(L=-1), 1), (dict(R=-8), 1),
    (dict(K=100), 2), (dict(R=12), 2), (dict(R=264), 2),
    (dict(wq=None), 1), (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(ids=None), 1), (dict(y=None), 1),
    (dict(a=P + 8), 3), (dict(b=P + 8), 3), (dict(ids=P + 2), 3), (dict(sc=P + 1), 3), (dict(ranks=P + 2), 3),
    (dict(y=P + 8), 3), (dict(ws=None), 4), (dict(ws=P + 16), 3), (dict(L=1 << 40), 1),
    (dict(N=0), 0), (dict(T=0), 0)])
def test_lora_refusals(lib, kw, status):
    assert lora(lib, **kw) == status
    assert (q4lin.last_error_detail() == "") == (status == 0)


def test_lora_queries(lib):
    assert q4lin.lora_route(6144, 5120, 1, 16) == q4lin.ROUTE_GEMV
    assert q4lin.lora_route(6144, 5120, 2, 16) == q4lin.ROUTE_STREAM_MMA
    assert q4lin.lora_route(6144, 5120, 32, 256) == q4lin.ROUTE_STREAM_MMA
    assert q4lin.lora_route(6144, 5120, 33, 16) == q4lin.ROUTE_TC_SPLITK
    assert q4lin.lora_route(6144, 5120, 1, 12) == -1 and q4lin.lora_route(6144, 100, 1, 16) == -1
    for T in (1, 8, 33, 1024):
        ws = q4lin.lora_workspace_bytes(6144, 5120, T, 4, 16)
        assert ws > 0 and ws % 256 == 0
    # no adapters: the projection alone, with its own workspace
    assert q4lin.lora_workspace_bytes(6144, 5120, 8, 0, 16) == q4lin.workspace_bytes(6144, 5120, 8)
    assert q4lin.lora_workspace_bytes(6144, 100, 8, 4, 16) == 0


def router(lib, T=2, H=64, E=8, k=2, x=P, w=P, bias=None, ids=P, p=P):
    return lib.q4lin_moe_router(x, w, bias, ids, p, T, H, E, k, 1, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(H=-8), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 2), (dict(E=1025), 2),
    (dict(E=64, k=17), 2), (dict(H=60), 2), (dict(x=None), 1), (dict(w=None), 1), (dict(ids=None), 1), (dict(p=None), 1),
    (dict(x=P + 8), 3), (dict(w=P + 4), 3), (dict(bias=P + 2), 3), (dict(ids=P + 1), 3), (dict(T=0), 0)])
def test_router_refusals(lib, kw, status):
    assert router(lib, **kw) == status


def experts(lib, T=2, H=64, F=128, E=8, k=2, x=P, ids=P, p=P, gu=P, gus=P, dn=P, dns=P, y=P, ws=P):
    return lib.q4lin_moe_experts(x, ids, p, gu, gus, dn, dns, y, T, H, F, E, k, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(F=-8), 1), (dict(E=0), 1), (dict(E=2000), 2), (dict(k=17), 2), (dict(k=0), 1),
    (dict(H=60), 2), (dict(F=100), 2), (dict(x=None), 1), (dict(ids=None), 1), (dict(gu=None), 1), (dict(dns=None), 1),
    (dict(y=None), 1), (dict(x=P + 8), 3), (dict(gus=P + 2), 3), (dict(ids=P + 2), 3), (dict(y=P + 2), 3),
    (dict(ws=None), 4), (dict(ws=P + 32), 3), (dict(E=1024, F=1 << 22), 2), (dict(T=0), 0), (dict(H=0), 0)])
def test_experts_refusals(lib, kw, status):
    assert experts(lib, **kw) == status


def test_moe_refuses_before_any_launch(lib):
    f = lib.q4lin_moe
    ok = [P, P, None, P, P, P, P, P, P, P, 2, 64, 128, 8, 2, 1, P, None]
    for i, v, status in [(1, None, 1), (3, None, 1), (5, P + 8, 3), (9, None, 1), (14, 9, 2), (16, None, 4), (16, P + 1, 3)]:
        args = list(ok)
        args[i] = v
        assert f(*args) == status, i
    assert q4lin.moe_workspace_bytes(4, 64, 128, 8, 2) % 256 == 0 and q4lin.moe_workspace_bytes(4, 64, 128, 8, 2) > 0
    assert q4lin.moe_workspace_bytes(4, 64, 128, 8, 17) == 0


def qk(lib, q=P, ldq=64, k=P, ldk=32, qw=P, kw=P, cs=P, pos=P, qo=P, ldqo=64, ko=P, ldko=32, T=3, Hq=2, Hk=1, D=32, rot=32,
       n=16, eps=1e-6):
    return lib.q4lin_qk_norm_rope(q, ldq, k, ldk, qw, kw, cs, pos, qo, ldqo, ko, ldko, T, Hq, Hk, D, rot, n,
                                  ctypes.c_float(eps), 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(D=-8), 1), (dict(rot=-16), 1), (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1),
    (dict(D=36), 2), (dict(D=264, ldq=1024, ldk=1024, ldqo=1024, ldko=1024), 2), (dict(rot=8), 2), (dict(rot=48), 2),
    (dict(q=None), 1), (dict(ko=None), 1), (dict(kw=None), 1), (dict(cs=None), 1), (dict(pos=None), 1),
    (dict(ldq=56), 1), (dict(ldko=24), 1), (dict(ldq=68), 3), (dict(ldqo=66), 3), (dict(q=P + 8), 3), (dict(pos=P + 2), 3),
    (dict(cs=P + 8), 3), (dict(T=0), 0), (dict(Hq=0, Hk=0), 0), (dict(D=0, rot=0), 0)])
def test_qk_refusals(lib, kw, status):
    assert qk(lib, **kw) == status
