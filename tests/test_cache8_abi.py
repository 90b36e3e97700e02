"""C entry points of the rotary positions and the 8-bit cache without a GPU: refusals (all before the first HIP call; the
pointers are fake), calls with nothing to do, workspace sizes, and the frequencies, which are host arithmetic."""
import ctypes
import math

import numpy as np
import pytest

from gated_short_causal_amd import _lib

OK, NULLP, SHAPE, ALIGN, UNSUP, WS, PRECOND, HIP = range(8)
P, MIS = 0x10000, 0x10002


@pytest.fixture(scope="module")
def L():
    return _lib.hybrid_lib()


ROT = dict(dtype=0, D=64, R=64, inter=0, inv=0, q=P, qs=512, qo=P + 4096, qos=512, Hq=8, k=P, ks=128, ko=P + 4096, kos=128, Hkv=2, T=10,
           pos=P, cu=None, N=0, freqs=P, mag=1.0, stream=None)


def _rot(L, **kw):
    return L.lfm2sc_rotary(*{**ROT, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUP), (dict(dtype=-1), UNSUP), (dict(D=60), UNSUP), (dict(D=0), UNSUP), (dict(D=520), UNSUP), (dict(D=-64), UNSUP),
    (dict(R=0), SHAPE), (dict(R=63), SHAPE), (dict(R=66), SHAPE), (dict(R=-2), SHAPE), (dict(inter=2), UNSUP), (dict(inv=-1), UNSUP),
    (dict(Hq=0), SHAPE), (dict(Hq=1 << 15), SHAPE), (dict(Hkv=-1), SHAPE), (dict(Hkv=1 << 15), SHAPE),
    (dict(mag=math.inf), SHAPE), (dict(mag=math.nan), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(N=-1), SHAPE),
    (dict(qs=504), SHAPE), (dict(qs=516), ALIGN), (dict(qos=500), SHAPE), (dict(ks=120), SHAPE), (dict(kos=132), ALIGN), (dict(qs=1 << 22), SHAPE),
    (dict(q=None), NULLP), (dict(qo=None), NULLP), (dict(k=None), NULLP), (dict(ko=None), NULLP), (dict(pos=None), NULLP), (dict(freqs=None), NULLP),
    (dict(q=P + 8), ALIGN), (dict(qo=MIS), ALIGN), (dict(k=MIS), ALIGN), (dict(ko=MIS), ALIGN), (dict(pos=MIS), ALIGN), (dict(freqs=MIS), ALIGN),
    (dict(cu=MIS, N=1), ALIGN), (dict(qo=P, qos=520), SHAPE), (dict(ko=P, kos=136), SHAPE), (dict(T=1 << 27), SHAPE),
])
def test_rotary_refuses(L, kw, code):
    assert _rot(L, **kw) == code
    assert L.lfm2sc_last_error().decode().startswith("lfm2sc_rotary")


def test_rotary_no_work(L):
    assert _rot(L, T=0, q=None, qo=None, k=None, ko=None, pos=None, freqs=None) == OK
    assert _rot(L, cu=P, N=0, pos=None) == OK
    assert _rot(L, T=0, Hkv=0, k=None, ks=0, ko=None, kos=0) == OK


def _freqs(L, R, base=10000.0, scaling=0, factor=0.0, length=0.0, low=0.0, high=0.0):
    f = (ctypes.c_float * max(1, R // 2))()
    rc = L.lfm2sc_rotary_freqs(R, base, scaling, factor, length, low, high, ctypes.addressof(f))
    return rc, np.array(f, dtype=np.float32)


def test_freqs(L):
    i = np.arange(0, 64, 2) / 64
    plain = 10000.0 ** -i
    assert (_freqs(L, 64)[1] == plain.astype(np.float32)).all()
    assert (_freqs(L, 64, scaling=1, factor=4.0)[1] == (plain / 4).astype(np.float32)).all()
    grown = _freqs(L, 64, scaling=2, factor=8.0)[1]
    np.testing.assert_allclose(grown, (10000.0 * 8.0 ** (64 / 62)) ** -i, rtol=2.0 ** -23)
    np.testing.assert_allclose(grown[-1], plain[-1] / 8, rtol=2.0 ** -22)        # the slowest pair is slowed by the whole factor
    turns = 8192 * plain / (2 * np.pi)
    parts = _freqs(L, 64, scaling=3, factor=8.0, length=8192.0, low=1.0, high=4.0)[1]
    np.testing.assert_allclose(parts[turns > 4], plain[turns > 4], rtol=2.0 ** -23)
    np.testing.assert_allclose(parts[turns < 1], plain[turns < 1] / 8, rtol=2.0 ** -23)
    mid = (turns >= 1) & (turns <= 4)
    w = (turns[mid] - 1) / 3
    assert mid.any()
    np.testing.assert_allclose(parts[mid], plain[mid] * (w + (1 - w) / 8), rtol=2.0 ** -23)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), SHAPE), (dict(R=3), SHAPE), (dict(R=514), SHAPE), (dict(R=8, scaling=4), UNSUP), (dict(R=8, scaling=-1), UNSUP),
    (dict(R=8, base=1.0), SHAPE), (dict(R=8, base=math.inf), SHAPE), (dict(R=8, base=math.nan), SHAPE), (dict(R=8, scaling=1), SHAPE),
    (dict(R=8, scaling=1, factor=math.nan), SHAPE), (dict(R=2, scaling=2, factor=2.0), SHAPE), (dict(R=8, scaling=3, factor=2.0), SHAPE),
    (dict(R=8, scaling=3, factor=2.0, length=100.0, low=2.0, high=2.0), SHAPE),
    (dict(R=8, scaling=3, factor=2.0, length=100.0, low=-1.0, high=2.0), SHAPE),
    (dict(R=8, scaling=3, factor=2.0, length=100.0, low=1.0, high=math.inf), SHAPE),
])
def test_freqs_refuse(L, kw, code):
    assert _freqs(L, **kw)[0] == code
    assert L.lfm2sc_rotary_freqs(8, 1e4, 0, 0.0, 0.0, 0.0, 0.0, None) == NULLP


POOL = dict(kp=P, vp=P, ps=2 * 16 * 64, ksc=P, vsc=P, ss=2, pages=4, S=16, B=16)
WRITE = dict(dtype=0, fmt=0, D=64, Hkv=2, k=P, ks=128, v=P, vs=128, T=6, cu=P, N=3, **POOL, table=P, most=2, len=P, stream=None)
READ = dict(dtype=0, fmt=0, D=64, Hkv=2, **POOL, table=P, most=2, len=P, k=P, ks=128, v=P, vs=128, T=6, cu=P, N=3, stream=None)
ATT = dict(dtype=0, fmt=0, D=64, Hq=8, Hkv=2, q=P, qs=512, N=3, L=1, **POOL, prefix=P, plen=5, table=P, most=2, len=P, max=32, scale=0.125,
           out=P, os=512, ws=P, wsb=1 << 24, stream=None)
POOL_BAD = [
    (dict(fmt=2), UNSUP), (dict(fmt=-1), UNSUP), (dict(D=96), UNSUP), (dict(D=0), UNSUP), (dict(Hkv=0), SHAPE), (dict(S=8, B=1, ss=16), SHAPE),
    (dict(S=24), SHAPE), (dict(S=0), SHAPE), (dict(S=-16), SHAPE), (dict(B=0), SHAPE), (dict(B=2), SHAPE), (dict(B=32), SHAPE),
    (dict(B=48, S=256, ps=1 << 20, ss=1 << 10), SHAPE), (dict(B=256, S=256, ps=1 << 20, ss=1 << 10), SHAPE), (dict(B=-1), SHAPE),
    (dict(ps=2 * 16 * 64 - 16), SHAPE), (dict(ps=2 * 16 * 64 + 8), ALIGN), (dict(ps=1 << 31), SHAPE), (dict(ss=1), SHAPE), (dict(ss=1 << 31), SHAPE),
    (dict(S=1 << 23, ps=1 << 30, ss=1 << 22, B=16), SHAPE), (dict(most=-1), SHAPE), (dict(most=1 << 26), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 27), SHAPE), (dict(kp=None), NULLP), (dict(vp=None), NULLP), (dict(ksc=None), NULLP), (dict(vsc=None), NULLP),
    (dict(kp=P + 8), ALIGN), (dict(vp=MIS), ALIGN), (dict(ksc=MIS), ALIGN), (dict(vsc=MIS), ALIGN), (dict(table=None), NULLP),
    (dict(table=MIS), ALIGN), (dict(len=None), NULLP), (dict(len=MIS), ALIGN), (dict(N=-1), SHAPE),
]
ROWS_BAD = POOL_BAD + [
    (dict(dtype=2), UNSUP), (dict(dtype=-1), UNSUP), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(ks=120), SHAPE), (dict(vs=132), ALIGN),
    (dict(ks=1 << 22), SHAPE), (dict(k=None), NULLP), (dict(v=None), NULLP), (dict(k=MIS), ALIGN), (dict(v=P + 8), ALIGN), (dict(cu=MIS), ALIGN),
    (dict(cu=None, T=7), SHAPE), (dict(cu=None, N=0), SHAPE), (dict(N=(1 << 31) - 1), SHAPE),
]


@pytest.mark.parametrize("kw,code", ROWS_BAD)
@pytest.mark.parametrize("name,args", [("lfm2sc_cache8_write", WRITE), ("lfm2sc_cache8_read", READ)])
def test_cache_rows_refuse(L, name, args, kw, code):
    assert getattr(L, name)(*{**args, **kw}.values()) == code
    assert L.lfm2sc_last_error().decode().startswith(name)


@pytest.mark.parametrize("name,args", [("lfm2sc_cache8_write", WRITE), ("lfm2sc_cache8_read", READ)])
@pytest.mark.parametrize("kw", [dict(N=0), dict(T=0), dict(most=0), dict(cu=None, N=0, T=0)])
def test_cache_rows_no_work(L, name, args, kw):
    nothing = {x: None for x in ("k", "v", "kp", "vp", "ksc", "vsc", "table", "len")}
    assert getattr(L, name)(*{**args, **nothing, **kw}.values()) == OK


@pytest.mark.parametrize("kw,code", POOL_BAD + [
    (dict(dtype=1), UNSUP), (dict(Hq=7), SHAPE), (dict(Hq=0), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(L=-1), SHAPE),
    (dict(plen=-1), SHAPE), (dict(plen=1 << 30), SHAPE), (dict(max=33), SHAPE), (dict(max=-1), SHAPE), (dict(qs=504), SHAPE), (dict(os=516), ALIGN),
    (dict(q=None), NULLP), (dict(q=MIS), ALIGN), (dict(out=None), NULLP), (dict(out=MIS), ALIGN), (dict(prefix=None), NULLP), (dict(prefix=MIS), ALIGN),
    (dict(N=1 << 20, L=1 << 10), SHAPE), (dict(N=(1 << 31) - 1, L=(1 << 31) - 1), SHAPE),
    (dict(plen=20000, ws=None), WS), (dict(plen=20000, wsb=15), WS), (dict(plen=20000, ws=P + 8), ALIGN),
])
def test_attention_refuses(L, kw, code):
    assert L.lfm2sc_attn_cached8(*{**ATT, **kw}.values()) == code
    assert L.lfm2sc_last_error().decode().startswith("lfm2sc_attn_cached8")


def test_attention_no_work_and_workspace(L):
    nothing = {x: None for x in ("q", "kp", "vp", "ksc", "vsc", "prefix", "table", "len", "out", "ws")}
    assert L.lfm2sc_attn_cached8(*{**ATT, **nothing, "N": 0}.values()) == OK
    assert L.lfm2sc_attn_cached8(*{**ATT, **nothing, "L": 0}.values()) == OK
    size = L.lfm2sc_attn_cached8_workspace_bytes
    assert size(0, 64, 32, 8, 1, 1, 100, 100) == 0           # few keys: one launch
    big = size(0, 128, 24, 8, 64, 1, 0, 16384)
    assert big >= 64 * 24 * (128 + 2) * 4 * 2                # two splits or more
    for bad in ((1, 64, 32, 8, 64, 1, 0, 4096), (0, 96, 32, 8, 64, 1, 0, 4096), (0, 64, 7, 8, 64, 1, 0, 4096), (0, 64, 32, 8, 0, 1, 0, 4096),
                (0, 64, 32, 8, 64, 0, 0, 4096), (0, 64, 32, 8, 64, 1, -1, 4096), (0, 64, 32, 8, 64, 1, 0, -1), (0, 64, 32, 8, 64, 1, 1 << 30, 0),
                (0, 64, 32, 8, 1 << 28, 1, 0, 4096), (0, 64, 32, 8, (1 << 31) - 1, (1 << 31) - 1, 0, 4096)):
        assert size(*bad) == 0, bad
    # a smaller batch needs no more than the workspace of a larger one gives at the same split
    assert L.lfm2sc_attn_cached8(*{**ATT, "D": 64, "plen": 20000, "wsb": size(0, 64, 8, 2, 3, 1, 20000, 32) - 1}.values()) == WS
