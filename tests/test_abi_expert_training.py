"""Refusals of the operators that training the experts adds: bad arguments are reported before any
CUDA call, tensors on the wrong device before the library is entered (no GPU needed)."""
import ctypes
import types

import pytest
import torch

from tests import test_binding_devices as devices
from tests.test_abi_moe_layer import BAD, OK, SHAPE, lib  # noqa: F401  (the fixture)
from tests.test_binding_devices import hg  # noqa: F401  (the fixture)

SIZES = {"E", "N", "K", "M", "D", "k", "rows", "acc", "f32", "bytes"}


def _caller(f, names, ok):
    def call(**kw):
        a = dict(ok, **kw)
        return f(*[a[n] if n in SIZES else ctypes.c_float(a[n]) if n == "eps"
                   else ctypes.c_void_p(a[n]) for n in names], None)
    return call


def _refuses(call, bad, shape):
    for kw in bad:
        assert call(**kw) == BAD, kw
    for kw in shape:
        assert call(**kw) == SHAPE, kw


@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_wgrad(lib, fp8):  # noqa: F811
    names = ["dy", "x", *(["s"] if fp8 else []), "off", "E", "N", "K", "rows", "acc", "dw", "f32",
             "ws", "bytes"]
    call = _caller(getattr(lib.lib, "hg_grouped_wgrad_fp8" if fp8 else "hg_grouped_wgrad"), names,
                   dict(dy=0x1000, x=0x2000, s=0x3000, off=0x4000, E=4, N=64, K=256, rows=100,
                        acc=0, dw=0x5000, f32=1, ws=0x6000 if fp8 else 0,
                        bytes=2 * 256 * 100 if fp8 else 0))
    _refuses(call, [dict(E=0), dict(N=0), dict(K=0), dict(rows=-1), dict(dy=0), dict(x=0),
                    dict(off=0), dict(dw=0), dict(dy=0x1008), dict(x=0x2008), dict(off=0x4002),
                    dict(dw=0x5008), dict(acc=1, f32=0), *([dict(s=0)] if fp8 else []),
                    # one tile and many rows: parts, and a workspace for them
                    dict(E=1, N=256, K=256, rows=1 << 16),
                    dict(E=1, N=256, K=256, rows=1 << 16, ws=0x6000, bytes=1000),
                    dict(E=1, N=256, K=256, rows=1 << 16, ws=0x6004, bytes=1 << 30)],
             [dict(E=513), dict(N=60), dict(K=260), dict(N=(1 << 30) + 8), dict(K=(1 << 30) + 128),
              dict(E=512, N=1 << 30, K=1 << 20), dict(N=1 << 30, rows=1 << 20),
              dict(rows=(1 << 31) - 1, ws=0x6000, bytes=1 << 60)])
    if fp8:                                               # the decoded rows need a workspace
        _refuses(call, [dict(ws=0), dict(bytes=2 * 256 * 100 - 1), dict(ws=0x6008)], [dict(K=264)])


def test_grouped_wgrad_workspace(lib):  # noqa: F811
    f = lib.hg_grouped_wgrad_workspace_bytes
    assert f(32, 4096, 6144, 16384) == 0                  # tiles enough
    assert f(1, 256, 256, 100) == 0                       # too few rows to cut
    need = f(1, 256, 512, 1 << 16)
    assert need > 0 and need % (4 * 256 * 512) == 0
    assert f(0, 256, 256, 1 << 16) == 0 and f(1, 256, 256, -1) == 0
    fp8 = lib.hg_grouped_wgrad_fp8_workspace_bytes        # the same and the decoded rows
    for E, K, rows in ((32, 6144, 16384), (1, 512, 1 << 16), (3, 128, 0)):
        assert fp8(E, 256, K, rows) == f(E, 256, K, rows) + 2 * K * rows
    assert fp8(1, 256, 256, -1) == 0
    # shapes that the call refuses, one of which has 2^64 tiles
    most = (1 << 31) - 1
    for shape in ((1 << 18, most, most, 100), (most, most, most, most), (1, 260, 256, 100),
                  (513, 256, 256, 100), (1, 1 << 30, 256, 1 << 20)):
        assert f(*shape) == 0 and fp8(*shape) == 0, shape
    assert fp8(1, 256, 264, 100) == 0


def test_quantize_weights(lib):  # noqa: F811
    call = _caller(lib.lib.hg_quantize_weights,
                   ["w", "f32", "E", "N", "K", "q", "s", "qt", "st"],
                   dict(w=0x1000, f32=1, E=2, N=64, K=96, q=0x2000, s=0x3000, qt=0x4000, st=0x5000))
    _refuses(call, [dict(E=-1), dict(N=0), dict(K=0), dict(w=0), dict(q=0), dict(s=0), dict(qt=0),
                    dict(st=0), dict(w=0x1008), dict(q=0x2008), dict(qt=0x4008)],
             [dict(K=40), dict(N=40), dict(E=1 << 20, N=1 << 12), dict(E=1 << 10, N=1 << 20, K=1 << 14),
              # columns and rows that a last tile would number past 2^31
              dict(E=1, N=32, K=(1 << 31) - 32), dict(E=1, N=(1 << 31) - 32, K=32)])
    assert call(E=0, w=0, q=0, s=0, qt=0, st=0) == OK


def test_dequantize_weights(lib):  # noqa: F811
    call = _caller(lib.lib.hg_dequantize_weights, ["q", "s", "E", "N", "K", "w", "f32"],
                   dict(q=0x2000, s=0x3000, E=2, N=5, K=96, w=0x1000, f32=0))
    _refuses(call, [dict(E=-1), dict(N=0), dict(K=0), dict(w=0), dict(q=0), dict(s=0),
                    dict(w=0x1008), dict(q=0x2008)], [dict(K=40), dict(E=1 << 20, N=1 << 12),
                                                 dict(E=1, N=32, K=(1 << 31) - 32)])
    assert call(E=0, w=0, q=0, s=0) == OK


def test_rmsnorm_quantize(lib):  # noqa: F811
    call = _caller(lib.lib.hg_rmsnorm_quantize,
                   ["x", "res", "gain", "M", "D", "eps", "sum", "y", "a", "s", "r"],
                   dict(x=0x1000, res=0x2000, gain=0x3000, M=4, D=256, eps=1e-6, sum=0x4000,
                        y=0x5000, a=0x6000, s=0x7000, r=0x8000))
    _refuses(call, [dict(M=-1), dict(D=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                    dict(eps=float("inf")), dict(eps=1e-31), dict(x=0), dict(gain=0), dict(res=0),
                    dict(sum=0), dict(a=0), dict(s=0), dict(x=0x1008), dict(res=0x2008),
                    dict(gain=0x3008), dict(sum=0x4008), dict(y=0x5008), dict(a=0x6008),
                    dict(r=0x8002)],
             [dict(D=200), dict(D=100, a=0, s=0), dict(D=16512), dict(D=1 << 30)])
    assert call(M=0, x=0, res=0, gain=0, sum=0, y=0, a=0, s=0, r=0) == OK


def test_rmsnorm_bwd(lib):  # noqa: F811
    need = lib.hg_rmsnorm_bwd_workspace_bytes(4, 256)
    assert need >= 256 * 4 and lib.hg_rmsnorm_bwd_workspace_bytes(1 << 20, 256) >= need
    for M, D in ((0, 256), (4, 0), (4, 12), (4, 16392)):
        assert lib.hg_rmsnorm_bwd_workspace_bytes(M, D) == 0
    call = _caller(lib.lib.hg_rmsnorm_bwd,
                   ["dy", "ds", "sum", "gain", "r", "M", "D", "dx", "dg", "ws", "bytes"],
                   dict(dy=0x1000, ds=0x2000, sum=0x3000, gain=0x4000, r=0x5000, M=4, D=256,
                        dx=0x6000, dg=0x7000, ws=0x8000, bytes=need))
    _refuses(call, [dict(M=-1), dict(D=0), dict(dy=0), dict(sum=0), dict(gain=0), dict(r=0),
                    dict(dx=0), dict(ws=0), dict(bytes=need - 1), dict(ws=0x8008), dict(dy=0x1008),
                    dict(ds=0x2008), dict(sum=0x3008), dict(gain=0x4008), dict(r=0x5002),
                    dict(dx=0x6008), dict(dg=0x7002)],
             [dict(D=12), dict(D=16392)])
    assert call(M=0, dy=0, ds=0, sum=0, gain=0, r=0, dx=0, dg=0, ws=0) == OK


def test_dispatch_acts(lib):  # noqa: F811
    call = _caller(lib.lib.hg_dispatch_acts, ["a", "s", "d2s", "M", "k", "K", "ra", "rs"],
                   dict(a=0x1000, s=0x2001, d2s=0x3000, M=4, k=2, K=256, ra=0x4000, rs=0x5001))
    _refuses(call, [dict(M=-1), dict(k=0), dict(K=0), dict(a=0), dict(s=0), dict(d2s=0), dict(ra=0),
                    dict(rs=0), dict(a=0x1008), dict(ra=0x4008), dict(d2s=0x3002)],
             [dict(K=200), dict(M=1 << 30), dict(K=(1 << 30) + 128)])
    assert call(M=0, a=0, s=0, d2s=0, ra=0, rs=0) == OK


# ------------------------------------------------------- in the binding ---

class OnGpu(devices.OnGpu):
    def __init__(self, shape, dtype, device):
        super().__init__(shape, dtype, device)
        self.shape, self.dtype = torch.Size(shape), dtype

    def element_size(self):
        return self.dtype.itemsize


B, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
NORM = [((3, 256), B), ((256,), B)]
CALLS = {
    "hg_dispatch_acts": (lambda f, t: f(t[0], t[1], 2, *t[2:]),
                         [((3, 256), U8), ((3, 2), U8), ((6,), I32), ((6, 256), U8), ((6, 2), U8)]),
    "hg_rmsnorm_quantize": (lambda f, t: f(t[0], t[1], t[2], y=t[3], a_fp8=t[4], a_scale=t[5],
                                           summed=t[6], rstd=t[7]),
                            [*NORM, ((3, 256), B), ((3, 256), B), ((3, 256), U8), ((3, 2), U8),
                             ((3, 256), B), ((3,), F32)]),
    "hg_rmsnorm_bwd": (lambda f, t: f(*t[:4], dsum=t[4], dx=t[5], dgain=t[6], workspace=t[7]),
                       [((3, 256), B), ((3, 256), B), ((256,), B), ((3,), F32), ((3, 256), B),
                        ((3, 256), B), ((256,), F32), ((1 << 20,), U8)]),
    "hg_quantize_weights": (lambda f, t: f(t[0], True, *t[1:]),
                            [((2, 64, 96), F32), ((2, 64, 48), U8), ((2, 64, 3), U8),
                             ((2, 96, 32), U8), ((2, 96, 2), U8)]),
    "hg_dequantize_weights": (lambda f, t: f(t[0], t[1], out=t[2]),
                              [((2, 64, 48), U8), ((2, 64, 3), U8), ((2, 64, 96), B)]),
    "hg_grouped_wgrad": (lambda f, t: f(*t[:3], dw=t[3], workspace=t[4]),
                         [((9, 64), B), ((9, 72), B), ((3,), I32), ((2, 64, 72), F32), ((4,), U8)]),
    "hg_grouped_wgrad_fp8": (lambda f, t: f(*t[:4], dw=t[4], accumulate=True, workspace=t[5]),
                             [((9, 64), B), ((9, 128), U8), ((9, 1), U8), ((3,), I32),
                              ((2, 64, 128), F32), ((9 * 128 * 2,), U8)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_call_goes_to_the_tensors_gpu(hg, monkeypatch, name):  # noqa: F811
    call, tensors = CALLS[name]
    record = devices.Recorder()
    monkeypatch.setattr(hg.lib, name, record)
    for device, entered in ((0, []), (1, [1])):
        hg.entered.clear()
        call(getattr(hg, name), [OnGpu(*t, device) for t in tensors])
        assert hg.entered == entered and record.calls[-1][-1] == 0x5000 + device
    stream = types.SimpleNamespace(cuda_stream=0x7000, device_index=1)
    f = getattr(hg, name)
    call(lambda *a, **kw: f(*a, **kw, stream=stream), [OnGpu(*t, 1) for t in tensors])
    assert record.calls[-1][-1] == 0x7000


@pytest.mark.parametrize("name", CALLS)
def test_tensors_elsewhere_are_refused(hg, monkeypatch, name):  # noqa: F811
    call, tensors = CALLS[name]
    record = devices.Recorder()
    monkeypatch.setattr(hg.lib, name, record)
    for i in range(len(tensors)):
        for other in (-1, 1):                               # on the CPU, on another GPU
            with pytest.raises(AssertionError):
                call(getattr(hg, name), [OnGpu(*t, other if i == j else 0)
                                         for j, t in enumerate(tensors)])
    assert not record.calls


@pytest.mark.parametrize("name", CALLS)
def test_other_types_and_shapes_are_refused(hg, monkeypatch, name):  # noqa: F811
    call, tensors = CALLS[name]
    record = devices.Recorder()
    monkeypatch.setattr(hg.lib, name, record)
    for i, (shape, dtype) in enumerate(tensors):
        if dtype == U8 and len(shape) == 1:                 # a workspace: any type, large enough
            continue
        for other in ((shape, torch.float64), ((*shape[:-1], shape[-1] - 1), dtype)):
            with pytest.raises(AssertionError):
                call(getattr(hg, name), [OnGpu(*(other if i == j else t), 0)
                                         for j, t in enumerate(tensors)])
    assert not record.calls


def test_a_workspace_too_small_is_refused(hg, monkeypatch):  # noqa: F811
    record = devices.Recorder()
    monkeypatch.setattr(hg.lib, "hg_rmsnorm_bwd", record)
    call, tensors = CALLS["hg_rmsnorm_bwd"]
    with pytest.raises(AssertionError):
        call(hg.hg_rmsnorm_bwd, [OnGpu(*t, 0) for t in tensors[:-1]] + [OnGpu((64,), U8, 0)])
    call, tensors = CALLS["hg_grouped_wgrad_fp8"]
    monkeypatch.setattr(hg.lib, "hg_grouped_wgrad_fp8", record)
    with pytest.raises(AssertionError):
        call(hg.hg_grouped_wgrad_fp8, [OnGpu(*t, 0) for t in tensors[:-1]] + [OnGpu((64,), U8, 0)])
    with pytest.raises(AssertionError):                     # nothing to add to
        hg.hg_grouped_wgrad(*[OnGpu(*t, 0) for t in CALLS["hg_grouped_wgrad"][1][:3]],
                            accumulate=True)
    assert not record.calls
