"""C entry points of include/lfm2sc_hybrid.h without a GPU: exported symbols, refusals (all before the first HIP
call; the pointers are fake) and calls with nothing to do."""
import math
import os
import re

import pytest

from gated_short_causal_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lfm2sc_hybrid.h")
OK, NULLP, SHAPE, ALIGN, UNSUP, WS, PRECOND, HIP = range(8)
P, MIS = 0x10000, 0x10002


@pytest.fixture(scope="module")
def L():
    return _lib.hybrid_lib()


def test_exports_every_declared_symbol(L):
    names = set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]+?\b(lfm2sc_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(_lib.HYBRID_SIGNATURES)
    for n in names:
        assert hasattr(L, n), n


PROMPT = dict(dtype=0, D=64, Hq=8, Hkv=2, q=P, qs=512, k=P, ks=128, v=P, vs=128, T=10, cu=P, N=1, scale=0.125, out=P, os=512,
              lse=P, stream=None)


def _prompt(L, **kw):
    return L.lfm2sc_attn_prefill(*{**PROMPT, **kw}.values())


COMMON = [
    (dict(dtype=1), UNSUP), (dict(dtype=5), UNSUP), (dict(D=96), UNSUP), (dict(D=0), UNSUP), (dict(Hkv=0), SHAPE),
    (dict(Hq=6, Hkv=4), SHAPE), (dict(Hq=1, Hkv=2), SHAPE), (dict(Hq=-2), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(T=1 << 30), SHAPE), (dict(N=-1), SHAPE), (dict(T=(1 << 31) - 1, Hq=1 << 12), SHAPE),
    (dict(qs=504), SHAPE), (dict(qs=516), ALIGN), (dict(ks=120), SHAPE), (dict(vs=130), ALIGN), (dict(os=511), SHAPE),
    (dict(ks=1 << 22), SHAPE), (dict(q=None), NULLP), (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(cu=None), NULLP),
    (dict(out=None), NULLP), (dict(q=MIS), ALIGN), (dict(k=P + 8), ALIGN), (dict(v=MIS), ALIGN), (dict(out=MIS), ALIGN),
    (dict(cu=MIS), ALIGN), (dict(lse=MIS), ALIGN),
]


@pytest.mark.parametrize("kw,code", COMMON)
def test_prefill_refuses(L, kw, code):
    assert _prompt(L, **kw) == code
    assert L.lfm2sc_last_error().decode().startswith("lfm2sc_attn_prefill")


def test_prefill_no_work(L):
    assert _prompt(L, N=0, q=None, cu=None, out=None) == OK
    assert _prompt(L, T=0, q=None, k=None, v=None, cu=None, out=None) == OK
    assert L.lfm2sc_last_error().decode() == ""


BWD = dict(dtype=0, D=64, Hq=8, Hkv=2, q=P, qs=512, k=P, ks=128, v=P, vs=128, T=10, cu=P, N=1, scale=0.125, out=P, os=512,
           lse=P, do=P, dos=512, dq=P, dqs=512, dk=P, dks=128, dv=P, dvs=128, ws=P, ws_bytes=1 << 20, stream=None)


def _bwd(L, **kw):
    return L.lfm2sc_attn_backward(*{**BWD, **kw}.values())


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(lse=None), NULLP), (dict(do=None), NULLP), (dict(dq=None), NULLP), (dict(dk=None), NULLP), (dict(dv=None), NULLP),
    (dict(do=MIS), ALIGN), (dict(dq=MIS), ALIGN), (dict(dk=P + 4), ALIGN), (dict(dv=P + 8), ALIGN),
    (dict(dos=500), SHAPE), (dict(dqs=504), SHAPE), (dict(dks=129), ALIGN), (dict(dvs=64), SHAPE),
    (dict(ws=None), WS), (dict(ws_bytes=1023), WS), (dict(ws=P + 8), ALIGN),
])
def test_backward_refuses(L, kw, code):
    assert _bwd(L, **kw) == code
    assert L.lfm2sc_last_error().decode().startswith("lfm2sc_attn_backward")


def test_backward_no_work_and_workspace(L):
    assert _bwd(L, N=0, q=None, ws=None) == OK
    assert _bwd(L, T=0, q=None, ws=None) == OK
    need = L.lfm2sc_attn_backward_workspace_bytes
    assert need(0, 64, 8, 2, 1000, 3) >= 2 * 8 * 1000 * 4
    for bad in ((1, 64, 8, 2, 10, 1), (0, 80, 8, 2, 10, 1), (0, 64, 8, 3, 10, 1), (0, 64, 8, 0, 10, 1), (0, 64, 8, 2, 0, 1),
                (0, 64, 8, 2, 10, 0), (0, 64, 8, 2, 1 << 31, 1)):
        assert need(*bad) == 0, bad


CACHED = dict(dtype=0, D=64, Hq=8, Hkv=2, q=P, qs=512, N=3, Lb=2, k=P, v=P, kvs=128, pages=10, page=16, pp=P, plen=2000, table=P,
              most=4, lens=P, scale=0.125, out=P, os=512, ws=P, ws_bytes=1 << 30, stream=None)


def _cached(L, **kw):
    return L.lfm2sc_attn_cached(*{**CACHED, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=1), UNSUP), (dict(D=32), UNSUP), (dict(Hq=7), SHAPE), (dict(Hkv=0), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(N=-1), SHAPE), (dict(Lb=-1), SHAPE), (dict(N=1 << 20, Lb=1 << 10), SHAPE), (dict(plen=-1), SHAPE), (dict(plen=1 << 30), SHAPE),
    (dict(most=1 << 26), SHAPE),
    (dict(page=0), SHAPE), (dict(page=24), SHAPE), (dict(page=-16), SHAPE), (dict(most=-1), SHAPE),
    (dict(most=1 << 27), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 27), SHAPE),
    (dict(qs=504), SHAPE), (dict(qs=516), ALIGN), (dict(kvs=64), SHAPE), (dict(kvs=132), ALIGN), (dict(os=256), SHAPE),
    (dict(q=None), NULLP), (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(pp=None), NULLP), (dict(table=None), NULLP),
    (dict(lens=None), NULLP), (dict(out=None), NULLP), (dict(q=MIS), ALIGN), (dict(k=MIS), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(pp=MIS), ALIGN), (dict(table=P + 1), ALIGN), (dict(lens=MIS), ALIGN), (dict(out=MIS), ALIGN),
    (dict(ws=None), WS), (dict(ws_bytes=100), WS), (dict(ws=P + 8), ALIGN),
])
def test_cached_refuses(L, kw, code):
    assert _cached(L, **kw) == code
    assert L.lfm2sc_last_error().decode().startswith("lfm2sc_attn_cached")


def test_cached_no_work_and_workspace(L):
    assert _cached(L, N=0, q=None, k=None, out=None, ws=None) == OK
    assert _cached(L, Lb=0, q=None, k=None, out=None, ws=None) == OK
    need = L.lfm2sc_attn_cached_workspace_bytes
    assert need(0, 64, 8, 2, 3, 2, 2000, 4, 16) > 0
    for bad in ((1, 64, 8, 2, 3, 2, 20, 4, 16), (0, 64, 8, 3, 3, 2, 20, 4, 16), (0, 64, 8, 2, 0, 2, 20, 4, 16),
                (0, 64, 8, 2, 3, 0, 20, 4, 16), (0, 64, 8, 2, 3, 2, -1, 4, 16), (0, 64, 8, 2, 3, 2, 20, 4, 17),
                (0, 64, 8, 2, 3, 2, 20, -4, 16)):
        assert need(*bad) == 0, bad


DRAFTS = dict(dtype=1, V=100, N=3, Lb=2, t=P, ts=100, d=P, ds=100, tok=P, nd=P, ua=P, us=P, al=P, kl=P, nt=P, ws=P,
              ws_bytes=1 << 20, stream=None)


def _drafts(L, **kw):
    return L.lfm2sc_accept_drafts(*{**DRAFTS, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUP), (dict(V=0), SHAPE), (dict(V=1 << 30), SHAPE), (dict(Lb=-1), SHAPE), (dict(Lb=65), SHAPE),
    (dict(N=-1), SHAPE), (dict(ts=99), SHAPE), (dict(ds=99), SHAPE), (dict(N=(1 << 31) - 1, V=1 << 20, ts=1 << 20, ds=1 << 20), SHAPE),
    (dict(t=None), NULLP), (dict(tok=None), NULLP), (dict(ua=None), NULLP), (dict(us=None), NULLP), (dict(al=None), NULLP),
    (dict(nt=None), NULLP), (dict(t=MIS), ALIGN), (dict(dtype=0, t=P + 1), ALIGN), (dict(d=MIS), ALIGN), (dict(tok=MIS), ALIGN),
    (dict(nd=MIS), ALIGN), (dict(ua=MIS), ALIGN), (dict(us=MIS), ALIGN), (dict(al=MIS), ALIGN), (dict(kl=MIS), ALIGN),
    (dict(nt=MIS), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=8), WS), (dict(ws=P + 4), ALIGN),
])
def test_drafts_refuse(L, kw, code):
    assert _drafts(L, **kw) == code
    assert L.lfm2sc_last_error().decode().startswith("lfm2sc_accept_drafts")


def test_drafts_no_work_and_workspace(L):
    assert _drafts(L, N=0, t=None, ws=None) == OK
    need = L.lfm2sc_accept_drafts_workspace_bytes
    assert need(3, 0, 1) > 0
    for bad in ((0, 2, 10), (3, -1, 10), (3, 65, 10), (3, 2, 0)):
        assert need(*bad) == 0, bad
