"""Argument errors of the tree operators come back before any launch (CPU)."""
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


MASKS = "par n q ctx B maxT m ms dep pos st s".split()
MASKS_OK = dict(par=F, n=4, q=F, ctx=F, B=2, maxT=40, m=F, ms=2, dep=F, pos=F, st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(B=-1), -1), (dict(maxT=-1), -1), (dict(ms=1), -1),
    (dict(maxT=257, ms=9), -2), (dict(ctx=None), -1),
    *[({k: None}, -1) for k in "par q m".split()],
    (dict(n=0), 0), (dict(B=0), 0), (dict(maxT=0), 0),
])
def test_tree_masks(lib, kw, code):
    assert call(lib.splash_tree_masks, MASKS, MASKS_OK, kw) == code


ATTN = ("q n kp vp ksc vsc tab maxp ctx T m ms B hq hkv D P pages maxT sm out lse ws wsb st s "
        "ctas").split()
ATTN_OK = dict(q=F, n=4, kp=F, vp=FV, ksc=F, vsc=F, tab=F, maxp=4, ctx=F, T=F, m=F, ms=1, B=2, hq=8,
               hkv=2, D=128, P=16, pages=8, maxT=4, sm=0.1, out=F, lse=F, ws=F, wsb=1 << 40, st=None,
               s=None, ctas=0)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(B=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(hq=7), -1),
    (dict(maxT=-1), -1), (dict(maxp=0), -1), (dict(maxp=2 ** 27), -1), (dict(pages=-1), -1),
    (dict(ctas=-1), -1), (dict(ctas=1024), -1), (dict(ms=0), -1), (dict(maxT=33), -1),
    (dict(n=2 ** 30), -1), (dict(D=96), -2), (dict(P=32), -2), (dict(maxT=257, ms=9), -2),
    (dict(hq=2 ** 21, hkv=2 ** 20, n=1), -2),
    (dict(sm=0.0), -1), (dict(sm=float("inf")), -1), (dict(sm=float("nan")), -1), (dict(vp=F), -1),
    (dict(ws=ctypes.c_void_p(4096 + 64)), -1),
    *[({k: F2}, -1) for k in "q kp ksc vsc out".split()],
    *[({k: None}, -1) for k in "q kp vp ksc vsc tab ctx T m out lse ws".split()],
    (dict(n=0), 0), (dict(B=0), 0), (dict(maxT=0), 0),
])
def test_verify_attention_tree(lib, kw, code):
    assert call(lib.splash_verify_attention_tree, ATTN, ATTN_OK, kw) == code


ACCEPT = "tok par tgt n q ctx ctxo acc nxt rows toks B maxT st s".split()
ACCEPT_OK = dict(tok=F, par=F, tgt=F, n=4, q=F, ctx=F, ctxo=F, acc=F, nxt=F, rows=F, toks=F, B=2, maxT=4,
                 st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(B=-1), -1), (dict(maxT=-1), -1), (dict(maxT=257), -2),
    *[({k: None}, -1) for k in "tok par tgt q ctx ctxo acc nxt rows".split()],
    (dict(B=0), 0),
])
def test_accept_tree(lib, kw, code):
    assert call(lib.splash_accept_tree, ACCEPT, ACCEPT_OK, kw) == code


POOL = 8 * 2 * 2 * 16 * 128
COMPACT = "kp vp ksc vsc cl sl L slots rows n q acc B hkv D P pages st s".split()
COMPACT_OK = dict(kp=F, vp=FV, ksc=F, vsc=F, cl=POOL, sl=8 * 2 * 16, L=3, slots=F, rows=F, n=4, q=F,
                  acc=F, B=2, hkv=2, D=128, P=16, pages=8, st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(B=-1), -1), (dict(hkv=0), -1), (dict(L=-1), -1), (dict(pages=-1), -1),
    (dict(pages=2 ** 27), -1), (dict(cl=POOL - 16), -1), (dict(cl=POOL + 8), -1), (dict(sl=255), -1),
    (dict(D=96), -2), (dict(P=32), -2), (dict(vp=F), -1), (dict(kp=F2), -1),
    (dict(B=2 ** 30, L=4), -1),
    *[({k: None}, -1) for k in "kp vp ksc vsc slots rows q acc".split()],
    (dict(n=0), 0), (dict(B=0), 0), (dict(L=0), 0),
])
def test_kv_compact(lib, kw, code):
    assert call(lib.splash_kv_compact, COMPACT, COMPACT_OK, kw) == code


LOGP = "z dt zs n V rows m tok lp ent k ids tlp ws wsb st s".split()
LOGP_OK = dict(z=F, dt=1, zs=1000, n=4, V=1000, rows=None, m=4, tok=F, lp=F, ent=F, k=5, ids=F, tlp=F,
               ws=F, wsb=1 << 20, st=None, s=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(m=-1), -1), (dict(V=0), -1), (dict(V=2 ** 30 + 1, zs=2 ** 31), -1),
    (dict(k=-1), -1), (dict(k=33), -2), (dict(dt=3), -2), (dict(dt=-1), -2), (dict(zs=999), -1),
    (dict(m=5), -1),                                    # more outputs than rows, no list
    (dict(z=ctypes.c_void_p(4097)), -1), (dict(ws=F2), -1), (dict(tok=None), -1), (dict(lp=None), -1),
    (dict(ids=None), -1), (dict(tlp=None), -1), (dict(wsb=100), -3),
    *[({k: None}, -1) for k in "z ws".split()],
    (dict(n=0, m=0), 0), (dict(m=0), 0),
])
def test_token_logprobs(lib, kw, code):
    assert call(lib.splash_token_logprobs, LOGP, LOGP_OK, kw) == code


def test_sizes(lib):
    f = lib.splash_token_logprobs_workspace_size
    assert f(0, 10) == 0 and f(-1, 10) == 0 and f(4, 0) == 0 and f(4, 2 ** 30 + 1) == 0
    assert f(1, 1000) >= 16 * 2 and f(2, 131072) < 2 * 32 * (131072 // 512 + 2)
    g = lib.splash_verify_attention_tree_workspace_size
    assert g(-1, 4, 8, 2, 128, 4, 0) == 0 and g(2, 4, 8, 2, 96, 4, 0) == 0
    assert g(2, 4, 8, 2, 128, 257, 0) == 0 and g(2, 4, 7, 2, 128, 4, 0) == 0
