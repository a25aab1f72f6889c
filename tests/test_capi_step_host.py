"""Argument errors of the step operators come back before any launch (CPU)."""
from __future__ import annotations

import ctypes

import pytest

F = ctypes.c_void_p(4096)            # never dereferenced: validation fails first
F2 = ctypes.c_void_p(4096 + 4)       # not 16-byte aligned
FV = ctypes.c_void_p(4096 + 16 * 128)


@pytest.fixture(scope="module")
def lib():
    import os
    from speculative_verify_attention_kv_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from speculative_verify_attention_kv_gb300 import splash_kv
    return splash_kv.LIB


def call(fn, names, base, kw):
    assert set(kw) <= set(names)
    a = dict(base)
    a.update(kw)
    return fn(*[a[k] for k in names])


TABLES = "ctx T B n P pages tab maxp cnt cnto free cap fc fco q new pos slots st s".split()
TABLES_OK = dict(ctx=F, T=F, B=2, n=4, P=16, pages=8, tab=F, maxp=4, cnt=F, cnto=F, free=F, cap=8,
                 fc=F, fco=F, q=F, new=F, pos=F, slots=F, st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(n=-1), -1), (dict(pages=-1), -1), (dict(maxp=0), -1), (dict(cap=-1), -1),
    (dict(pages=2 ** 27), -1),                         # page * 16 past 32 bits
    (dict(maxp=2 ** 27), -1), (dict(P=32), -2),
    *[({k: None}, -1) for k in "ctx T tab cnt cnto free fc fco q new pos slots".split()],
])
def test_build_tables(lib, kw, code):
    assert call(lib.splash_build_tables, TABLES, TABLES_OK, kw) == code


RELEASE = "keep B tab maxp P cnt cnto free cap fc fco off st s".split()
RELEASE_OK = dict(keep=F, B=2, tab=F, maxp=4, P=16, cnt=F, cnto=F, free=F, cap=8, fc=F, fco=F, off=F,
                  st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(maxp=0), -1), (dict(cap=-1), -1), (dict(P=8), -2),
    *[({k: None}, -1) for k in "keep tab cnt cnto free fc fco off".split()],
])
def test_release_pages(lib, kw, code):
    assert call(lib.splash_release_pages, RELEASE, RELEASE_OK, kw) == code


QKV = ("q k v dt n qs qh ks kh vs vh hq hkv D qw kw eps f ax R il rs pos A slots qo kp vp ksc vsc P "
       "pages st s").split()
QKV_OK = dict(q=F, k=F, v=F, dt=1, n=4, qs=2048, qh=128, ks=2048, kh=128, vs=2048, vh=128, hq=8, hkv=2,
              D=128, qw=None, kw=None, eps=1e-6, f=F, ax=None, R=128, il=0, rs=1.0, pos=F, A=1,
              slots=F, qo=F, kp=F, vp=FV, ksc=F, vsc=F, P=16, pages=8, st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(pages=-1), -1), (dict(R=-16), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(P=32), -2), (dict(D=96), -2), (dict(dt=2), -2), (dict(dt=7), -2), (dict(R=144), -2),
    (dict(R=24), -2),                                   # not a multiple of 16
    (dict(A=0), -1), (dict(rs=float("inf")), -1), (dict(rs=float("nan")), -1),
    (dict(vp=F), -1),                                   # not the V half of the pool
    (dict(q=F2), -1), (dict(k=F2), -1), (dict(v=F2), -1), (dict(qo=F2), -1),
    (dict(qs=2049), -1), (dict(kh=4), -1), (dict(dt=0, vs=2), -1), (dict(ks=-2048), -1),
    *[({k: None}, -1) for k in "q k v f pos slots qo kp vp ksc vsc".split()],
    (dict(n=0), 0),
])
def test_qkv_append(lib, kw, code):
    assert call(lib.splash_qkv_append, QKV, QKV_OK, kw) == code


GATHER = "kp vp ksc vsc slots n hkv D P pages ko vo dt st s".split()
GATHER_OK = dict(kp=F, vp=FV, ksc=F, vsc=F, slots=F, n=4, hkv=2, D=128, P=16, pages=8, ko=F, vo=F, dt=1,
                 st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(hkv=0), -1), (dict(pages=-1), -1), (dict(P=4), -2), (dict(D=32), -2),
    (dict(dt=2), -2), (dict(vp=F), -1), (dict(ko=F2), -1), (dict(vo=F2), -1),
    *[({k: None}, -1) for k in "kp vp ksc vsc slots ko vo".split()],
    (dict(n=0), 0),
])
def test_kv_gather(lib, kw, code):
    assert call(lib.splash_kv_gather, GATHER, GATHER_OK, kw) == code


CHOOSE = ("z dt zs n V q B maxT tok state ss rep pres freq bo bi bv nb m ms nm mr out os t ws wsb st "
          "s").split()
CHOOSE_OK = dict(z=F, dt=1, zs=1000, n=4, V=1000, q=F, B=2, maxT=4, tok=F, state=F, ss=1024, rep=F,
                 pres=F, freq=F, bo=F, bi=F, bv=F, nb=3, m=F, ms=32, nm=4, mr=None, out=F, os=1000, t=F,
                 ws=F, wsb=1 << 20, st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(B=-1), -1), (dict(V=0), -1), (dict(V=2 ** 30 + 1), -1), (dict(maxT=-1), -1),
    (dict(nb=-1), -1), (dict(nm=-1), -1), (dict(dt=3), -2), (dict(maxT=129), -2),
    (dict(zs=999), -1), (dict(z=ctypes.c_void_p(4097)), -1), (dict(ws=ctypes.c_void_p(4096 + 64)), -1),
    (dict(ss=999), -1), (dict(ss=1010), -1), (dict(state=F2), -1), (dict(state=None), -1),
    (dict(tok=None), -1), (dict(bi=None), -1), (dict(bv=None), -1), (dict(ms=31), -1), (dict(nm=3), -1),
    (dict(m=None, mr=F), -1), (dict(os=999), -1),
    (dict(out=ctypes.c_void_p(4096)), -1),              # in place needs fp32
    (dict(dt=0, out=ctypes.c_void_p(4096), os=1001), -1),
    *[({k: None}, -1) for k in "z q t ws".split()],
    (dict(n=0), 0), (dict(B=0), 0), (dict(maxT=0), 0),
])
def test_choose_targets(lib, kw, code):
    base = dict(CHOOSE_OK, out=ctypes.c_void_p(1 << 20))
    assert call(lib.splash_choose_targets, CHOOSE, base, kw) == code


HIST = "tok n q B acc state ss V prompt reset st s".split()
HIST_OK = dict(tok=F, n=4, q=F, B=2, acc=None, state=F, ss=1024, V=1000, prompt=0, reset=0, st=None,
               s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(B=-1), -1), (dict(V=0), -1), (dict(ss=999), -1), (dict(ss=1000), -1),
    (dict(state=F2), -1), (dict(tok=None), -1), (dict(q=None), -1), (dict(state=None), -1),
    (dict(n=0), 0), (dict(B=0), 0),
])
def test_token_state_add(lib, kw, code):
    assert call(lib.splash_token_state_add, HIST, HIST_OK, kw) == code


def test_sizes(lib):
    assert [lib.splash_token_state_stride(v) for v in (0, -1, 1, 64, 65)] == [0, 0, 64, 64, 128]
    f = lib.splash_choose_targets_workspace_size
    assert f(-1, 10) == 0 and f(4, 0) == 0 and f(0, 10) == 0
    assert f(4, 1000) == 8 * 4 * 2 and f(2, 1025) == 8 * 2 * 3
