"""Host-side refusals and size queries of the attention operators and the logits' answers: no GPU, the fake
pointers are never dereferenced."""
import ctypes

import pytest

from weight_only_bit_q4_gb300 import build as q4build
from weight_only_bit_q4_gb300 import q4lin

P = 256   # an aligned, non-null address
BIG = 1 << 41


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4lin.load()


def prompt(lib, q=P, ldq=128, k=P, ldk=64, v=P, ldv=64, cu=P, out=P, ldo=128, T=3, S=1, Hq=4, Hk=2, D=32, scale=1.0):
    return lib.q4lin_prompt_attention(q, ldq, k, ldk, v, ldv, cu, out, ldo, T, S, Hq, Hk, D, ctypes.c_float(scale), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(S=-1), 1), (dict(Hq=-4), 1), (dict(D=-8), 1), (dict(D=36), 2), (dict(D=136, ldq=1024, ldk=1024, ldv=1024, ldo=1024), 2),
    (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(Hq=65537), 1), (dict(T=1 << 31), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cu=None), 1), (dict(out=None), 1),
    (dict(ldq=120), 1), (dict(ldk=56), 1), (dict(ldo=8), 1), (dict(ldv=BIG), 1), (dict(ldq=132), 3), (dict(ldo=130), 3),
    (dict(q=P + 8), 3), (dict(v=P + 2), 3), (dict(cu=P + 2), 3), (dict(T=0), 0), (dict(S=0), 0), (dict(Hq=0), 0), (dict(D=0), 0)])
def test_prompt_refusals(lib, kw, status):
    assert prompt(lib, **kw) == status
    assert (q4lin.last_error_detail() == "") == (status == 0)


def append(lib, k=P, ldk=128, v=P, ldv=128, cache=P, table=P, rows=P, pos=P, T=2, S=2, M=4, pages=8, Hk=2, D=64):
    return lib.q4lin_kv4_append(k, ldk, v, ldv, cache, table, rows, pos, T, S, M, pages, Hk, D, None)


def read(lib, k=P, ldk=128, v=P, ldv=128, cache=P, table=P, rows=P, pos=P, T=2, S=2, M=4, pages=8, Hk=2, D=64):
    return lib.q4lin_kv4_read(cache, table, rows, pos, k, ldk, v, ldv, T, S, M, pages, Hk, D, None)


@pytest.mark.parametrize("f", [append, read])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(S=-1), 1), (dict(M=-1), 1), (dict(pages=-1), 1), (dict(Hk=-1), 1), (dict(D=80), 2), (dict(D=256), 2), (dict(D=0), 2),
    (dict(M=1 << 25), 1), (dict(pages=1 << 31), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cache=None), 1),
    (dict(table=None), 1), (dict(pos=None), 1), (dict(ldk=120), 1), (dict(ldv=132), 3), (dict(k=P + 8), 3), (dict(cache=P + 8), 3),
    (dict(table=P + 2), 3), (dict(rows=P + 1), 3), (dict(pos=P + 2), 3), (dict(T=0), 0), (dict(Hk=0), 0), (dict(pages=0), 0), (dict(S=0), 0)])
def test_token_refusals(lib, f, kw, status):
    assert f(lib, **kw) == status


def attention(lib, q=P, ldq=256, cache=P, table=P, lens=P, out=P, ldo=256, S=2, n=1, Hq=4, Hk=2, D=64, M=4, pages=8, scale=1.0, ws=P):
    return lib.q4lin_kv4_attention(q, ldq, cache, table, lens, out, ldo, S, n, Hq, Hk, D, M, pages, ctypes.c_float(scale), ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(n=-1), 1), (dict(Hq=-1), 1), (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(D=72), 2), (dict(M=-1), 1),
    (dict(n=65537), 1), (dict(S=1 << 30, n=4), 1), (dict(S=(1 << 31) - 1, Hk=4), 2), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(ldq=248), 1), (dict(ldo=260), 3),
    (dict(q=P + 8), 3), (dict(cache=P + 8), 3), (dict(lens=P + 2), 3), (dict(ws=None), 4), (dict(ws=P + 16), 3), (dict(S=0), 0),
    (dict(n=0), 0), (dict(Hq=0), 0)])
def test_cache_attention_refusals(lib, kw, status):
    assert attention(lib, **kw) == status


def logprobs(lib, x=P, fp32=0, ld=100, tok=P, lp=P, ent=P, ids=P, top=P, T=2, V=100, n=1, k=4):
    return lib.q4lin_token_logprobs(x, fp32, ld, tok, lp, ent, ids, top, T, V, n, k, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(n=-1), 1), (dict(k=-1), 1), (dict(k=33), 2), (dict(V=3, k=4), 2), (dict(V=1 << 31, ld=1 << 31), 2),
    (dict(ld=99), 1), (dict(ld=BIG), 1), (dict(x=None), 1), (dict(tok=None), 1), (dict(lp=None), 1), (dict(ids=None), 1),
    (dict(top=None), 1), (dict(x=P + 1), 3), (dict(x=P + 2, fp32=1), 3), (dict(tok=P + 2), 3), (dict(ent=P + 1), 3), (dict(T=0), 0)])
def test_logprobs_refusals(lib, kw, status):
    assert logprobs(lib, **kw) == status


def test_size_queries(lib):
    assert [q4lin.kv4_page_bytes(d) for d in (64, 96, 128, 80, 0, -64, 256)] == [4352, 6656, 8704, 0, 0, 0, 0]
    for args in ((1, 1, 32, 8, 128, 16), (64, 4, 28, 4, 96, 2000)):
        ws = q4lin.kv4_workspace_bytes(*args)
        assert ws > 0 and ws % 256 == 0
    assert q4lin.kv4_workspace_bytes(1, 1, 6, 4, 128, 16) == 0      # heads that do not divide
    assert q4lin.kv4_workspace_bytes(0, 1, 8, 4, 128, 16) == 0
