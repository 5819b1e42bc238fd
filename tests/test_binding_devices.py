"""Where the binding of the MoE layer's operators sends a call: tensors that are not on a GPU, or not
on the same one, are refused before the library is entered; a call on another GPU than the current
one is made with that GPU current, on its stream.  No GPU needed: the library's functions are
replaced by one that records its arguments."""
import contextlib
import subprocess
import sys
import types

import pytest
import torch

from tests.test_abi_moe_layer import ROOT, lib  # noqa: F401  (lib is the fixture)


class Recorder:
    def __init__(self):
        self.calls = []

    def __call__(self, *args):
        self.calls.append(args)
        return 0


class OnGpu:
    """Stands for a tensor: its attributes, without memory behind it."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device_ = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device_

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


B, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
# every call with its tensors' shapes and types, outputs given
CALLS = {
    "hg_dispatch_tokens": (lambda f, t: f(t[0], 2, t[1], t[2], out=t[3]),
                           [((3, 64), B), ((6,), I32), ((3, 2), F32), ((6, 64), B)]),
    "hg_dispatch_tokens_bwd": (lambda f, t: f(t[0], 2, t[1], t[2], t[3], t[4], t[5]),
                               [((6, 64), B), ((6,), I32), ((3, 2), F32), ((3, 64), B),
                                ((3, 64), B), ((3, 2), F32)]),
    "hg_combine_topk_bwd": (lambda f, t: f(*t),
                            [((3, 64), B), ((6, 64), B), ((6,), I32), ((3, 2), F32), ((6, 64), B),
                             ((3, 2), F32)]),
    "hg_swiglu_quantize": (lambda f, t: f(t[0], True, *t[1:]),
                           [((3, 512), B), ((3, 256), U8), ((3, 2), U8), ((3, 512), U8),
                            ((3, 4), U8)]),
    "hg_swiglu_bwd": (lambda f, t: f(*t), [((3, 256), B), ((3, 512), U8), ((3, 4), U8),
                                           ((3, 512), B)]),
    "hg_expert_matvec": (lambda f, t: f(*t), [((3, 128), B), ((3, 2), I32), ((4, 16, 64), U8),
                                              ((4, 16, 4), U8), ((6, 16), B)]),
    "hg_expert_matvec_swiglu": (lambda f, t: f(*t), [((3, 128), B), ((3, 2), I32),
                                                     ((4, 16, 64), U8), ((4, 16, 4), U8),
                                                     ((6, 8), B)]),
    "hg_router_topk": (lambda f, t: f(t[0], 2, True, t[1], t[2]),
                       [((3, 8), F32), ((3, 2), I32), ((3, 2), F32)]),
    "hg_router_topk_bwd": (lambda f, t: f(*t[:4], True, t[4]),
                           [((3, 8), F32), ((3, 2), I32), ((3, 2), F32), ((3, 2), F32),
                            ((3, 8), F32)]),
}


@pytest.fixture
def hg(lib, monkeypatch):  # noqa: F811
    entered = []

    @contextlib.contextmanager
    def device(index):
        entered.append(index)
        monkeypatch.setattr(lib, "_get_device", lambda: index)
        yield
        monkeypatch.setattr(lib, "_get_device", lambda: 0)

    monkeypatch.setattr(lib, "_get_device", lambda: 0)
    monkeypatch.setattr(lib, "_raw_stream", lambda index: 0x5000 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    lib.entered = entered
    yield lib
    del lib.entered


@pytest.mark.parametrize("name", CALLS)
def test_call_goes_to_the_tensors_gpu(hg, monkeypatch, name):
    call, tensors = CALLS[name]
    record = Recorder()
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
def test_tensors_elsewhere_are_refused(hg, monkeypatch, name):
    call, tensors = CALLS[name]
    record = Recorder()
    monkeypatch.setattr(hg.lib, name, record)
    for i in range(len(tensors)):
        for other in (-1, 1):                               # on the CPU, on another GPU
            with pytest.raises(AssertionError):
                call(getattr(hg, name), [OnGpu(*t, other if i == j else 0)
                                         for j, t in enumerate(tensors)])
    stream = types.SimpleNamespace(cuda_stream=0x7000, device_index=1)
    f = getattr(hg, name)
    with pytest.raises(AssertionError):
        call(lambda *a, **kw: f(*a, **kw, stream=stream), [OnGpu(*t, 0) for t in tensors])
    assert not record.calls


def test_cpu_tensors_are_refused(lib):  # noqa: F811
    with pytest.raises(AssertionError):
        lib.hg_router_topk(torch.zeros(2, 4), 2)
    with pytest.raises(AssertionError):
        lib.hg_swiglu_quantize(torch.zeros(2, 256, dtype=B), False)


def test_import_without_torchs_private_names(lib):  # noqa: F811
    # a torch built without CUDA has neither
    code = ("import torch; del torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice; "
            "from fp8_mxfp4_grouped_gb300 import hg; "
            "assert hg._raw_stream is hg._stream_handle; "
            "assert hg._get_device is torch.cuda.current_device; print(hg.lib.hg_version())")
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0, done.stderr
