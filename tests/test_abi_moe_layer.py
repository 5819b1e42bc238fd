"""Refusals of the MoE layer's entry points: bad arguments are reported before any CUDA call
(no GPU needed), empty problems are no-ops."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(os.path.join(ROOT, "fp8_mxfp4_grouped_gb300", "libhg.so")):
        from fp8_mxfp4_grouped_gb300 import build
        build.build()
    from fp8_mxfp4_grouped_gb300 import hg
    return hg


def _caller(f, names, ok):
    def call(**kw):
        a = dict(ok, **kw)
        return f(*[a[n] if n in INTS else ctypes.c_void_p(a[n]) for n in names], None)
    return call


INTS = {"M", "k", "K", "N", "rows", "F", "E", "x_rows", "renorm"}
BAD, SHAPE, OK = 1, 2, 0


def test_codes(lib):
    assert (lib.HG_ERR_INVALID_ARG, lib.HG_ERR_UNSUPPORTED_SHAPE, lib.HG_OK) == (BAD, SHAPE, OK)


def test_dispatch_tokens(lib):
    call = _caller(lib.lib.hg_dispatch_tokens, ["x", "d2s", "w", "M", "k", "K", "rows_"],
                   dict(x=0x1000, d2s=0x2000, w=0x3000, M=4, k=2, K=64, rows_=0x4000))
    for kw in (dict(M=-1), dict(k=0), dict(K=0), dict(x=0), dict(d2s=0), dict(rows_=0),
               dict(x=0x1008), dict(rows_=0x4008), dict(d2s=0x2002), dict(w=0x3002)):
        assert call(**kw) == BAD, kw
    for kw in (dict(K=60), dict(M=1 << 30)):
        assert call(**kw) == SHAPE, kw
    assert call(M=0, x=0, d2s=0, w=0, rows_=0) == OK


def test_dispatch_tokens_bwd(lib):
    call = _caller(lib.lib.hg_dispatch_tokens_bwd,
                   ["dr", "x", "d2s", "w", "M", "k", "K", "dx", "dw"],
                   dict(dr=0x1000, x=0x2000, d2s=0x3000, w=0x4000, M=4, k=2, K=64, dx=0x5000,
                        dw=0x6000))
    for kw in (dict(M=-1), dict(k=0), dict(K=0), dict(dr=0), dict(d2s=0), dict(dx=0), dict(x=0),
               dict(dw=0), dict(dr=0x1008), dict(x=0x2008), dict(dx=0x5008), dict(dw=0x6002)):
        assert call(**kw) == BAD, kw
    for kw in (dict(K=60), dict(M=1 << 30)):
        assert call(**kw) == SHAPE, kw
    assert call(M=0, dr=0, x=0, d2s=0, w=0, dx=0, dw=0) == OK


def test_combine_topk_bwd(lib):
    call = _caller(lib.lib.hg_combine_topk_bwd,
                   ["do", "y", "d2s", "w", "M", "k", "N", "dy", "dw"],
                   dict(do=0x1000, y=0x2000, d2s=0x3000, w=0x4000, M=4, k=2, N=64, dy=0x5000,
                        dw=0x6000))
    for kw in (dict(M=-1), dict(k=0), dict(N=0), dict(do=0), dict(y=0), dict(d2s=0), dict(w=0),
               dict(dy=0), dict(dw=0), dict(do=0x1008), dict(y=0x2008), dict(dy=0x5008)):
        assert call(**kw) == BAD, kw
    for kw in (dict(N=60), dict(M=1 << 30)):
        assert call(**kw) == SHAPE, kw
    assert call(M=0, do=0, y=0, d2s=0, w=0, dy=0, dw=0) == OK


def test_swiglu_quantize(lib):
    call = _caller(lib.lib.hg_swiglu_quantize, ["z", "rows", "F", "a", "as_", "q", "qs"],
                   dict(z=0x1000, rows=4, F=256, a=0x2000, as_=0x3000, q=0x4000, qs=0x5000))
    for kw in (dict(rows=-1), dict(F=0), dict(z=0), dict(a=0), dict(as_=0), dict(q=0),
               dict(qs=0), dict(z=0x1008), dict(a=0x2008), dict(q=0x4008)):
        assert call(**kw) == BAD, kw
    assert call(F=200) == SHAPE
    assert call(rows=0, z=0, a=0, as_=0, q=0, qs=0) == OK


def test_swiglu_bwd(lib):
    call = _caller(lib.lib.hg_swiglu_bwd, ["dh", "q", "qs", "rows", "F", "dz"],
                   dict(dh=0x1000, q=0x2000, qs=0x3000, rows=4, F=256, dz=0x4000))
    for kw in (dict(rows=-1), dict(F=0), dict(dh=0), dict(q=0), dict(qs=0), dict(dz=0),
               dict(dh=0x1008), dict(q=0x2008), dict(dz=0x4008)):
        assert call(**kw) == BAD, kw
    assert call(F=200) == SHAPE
    assert call(rows=0, dh=0, q=0, qs=0, dz=0) == OK


@pytest.mark.parametrize("name", ["hg_expert_matvec", "hg_expert_matvec_swiglu"])
def test_expert_matvec(lib, name):
    call = _caller(getattr(lib.lib, name),
                   ["x", "x_rows", "ids", "w", "ws", "M", "k", "E", "N", "K", "y"],
                   dict(x=0x1000, x_rows=4, ids=0x2000, w=0x3000, ws=0x4000, M=4, k=2, E=8, N=64,
                        K=256, y=0x5000))
    for kw in (dict(M=-1), dict(k=0), dict(E=0), dict(N=0), dict(K=0), dict(x_rows=5),
               dict(x=0), dict(ids=0), dict(w=0), dict(ws=0), dict(y=0), dict(x=0x1008),
               dict(ids=0x2002), dict(w=0x3010), dict(ws=0x4001), dict(y=0x5001)):
        assert call(**kw) == BAD, kw
    for kw in (dict(K=64), dict(K=320), dict(K=32896), dict(M=257, x_rows=257),
               dict(E=1 << 20, N=1 << 12)):
        assert call(**kw) == SHAPE, kw
    assert call(M=0, x_rows=0, x=0, ids=0, y=0) == OK
    if name.endswith("swiglu"):
        assert call(N=63) == SHAPE


def test_router(lib):
    call = _caller(lib.lib.hg_router_topk, ["l", "M", "E", "k", "renorm", "ids", "w"],
                   dict(l=0x1000, M=4, E=64, k=8, renorm=1, ids=0x2000, w=0x3000))
    for kw in (dict(M=-1), dict(E=0), dict(k=0), dict(k=9, E=8), dict(l=0), dict(ids=0),
               dict(w=0), dict(l=0x1002), dict(ids=0x2002), dict(w=0x3002)):
        assert call(**kw) == BAD, kw
    assert call(k=33) == SHAPE
    assert call(M=0, l=0, ids=0, w=0) == OK


def test_router_bwd(lib):
    call = _caller(lib.lib.hg_router_topk_bwd,
                   ["l", "ids", "w", "dw", "M", "E", "k", "renorm", "dl"],
                   dict(l=0x1000, ids=0x2000, w=0x3000, dw=0x4000, M=4, E=64, k=8, renorm=0,
                        dl=0x5000))
    for kw in (dict(M=-1), dict(E=0), dict(k=0), dict(k=9, E=8), dict(l=0), dict(ids=0),
               dict(w=0), dict(dw=0), dict(dl=0), dict(dl=0x5002)):
        assert call(**kw) == BAD, kw
    assert call(k=33) == SHAPE
    assert call(M=0, l=0, ids=0, w=0, dw=0, dl=0) == OK
