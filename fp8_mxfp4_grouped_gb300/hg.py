"""Python binding of libhg (the C ABI in include/hg.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  Tensors are torch CUDA tensors (device memory and
streams only); their data pointers are passed straight through ctypes.
There is no fallback: if the library is missing, importing this module
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhg.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m fp8_mxfp4_grouped_gb300.build` (nvcc, sm_103a)")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_u32 = ctypes.c_uint32
_sz = ctypes.c_size_t

lib.hg_status_string.argtypes = [ctypes.c_int]
lib.hg_status_string.restype = ctypes.c_char_p
lib.hg_version.argtypes = []
lib.hg_version.restype = ctypes.c_int
lib.hg_shutdown.argtypes = []
lib.hg_shutdown.restype = ctypes.c_int
lib.hg_plan_workspace_bytes.argtypes = [_i32, _i32, _i32]
lib.hg_plan_workspace_bytes.restype = _sz
lib.hg_plan_block_threads.argtypes = [_i32, _i32]
lib.hg_plan_block_threads.restype = _i32
lib.hg_plan_launches.argtypes = [_i32, _i32, _i32]
lib.hg_plan_launches.restype = _i32
lib.hg_plan_expert_offsets.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p, _sz, _p]
lib.hg_plan_expert_offsets.restype = ctypes.c_int
lib.hg_grouped_w4a8_gemm.argtypes = [_p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _p, _p]
lib.hg_grouped_w4a8_gemm.restype = ctypes.c_int
lib.hg_grouped_w4a8_gemm_mmajor.argtypes = [_p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _p, _p]
lib.hg_grouped_w4a8_gemm_mmajor.restype = ctypes.c_int
lib.hg_quantize_gather_acts.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p]
lib.hg_quantize_gather_acts.restype = ctypes.c_int
lib.hg_quantize_scatter_acts.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p]
lib.hg_quantize_scatter_acts.restype = ctypes.c_int
lib.hg_combine_topk.argtypes = [_p, _p, _p, _i32, _i32, _i32, _p, _p]
lib.hg_combine_topk.restype = ctypes.c_int
lib.hg_get_device_status.argtypes = [_p, ctypes.POINTER(_u32)]
lib.hg_get_device_status.restype = ctypes.c_int
lib.hg_selftest_wait_timeout.argtypes = [_u32, _p]
lib.hg_selftest_wait_timeout.restype = ctypes.c_int
lib.hg_set_wait_timeout_us.argtypes = [_u32]
lib.hg_set_wait_timeout_us.restype = None
lib.hg_gemm_token_tile.argtypes = [_i32, _i32, _i32, _i32]
lib.hg_gemm_token_tile.restype = _i32
lib.hg_gemm_ctas.argtypes = [_i32, _i32, _i32, _i32]
lib.hg_gemm_ctas.restype = _i32
lib.hg_set_gemm_variant.argtypes = [_i32]
lib.hg_set_gemm_variant.restype = _i32
lib.hg_gemm_host_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
lib.hg_gemm_host_workspace_bytes.restype = _sz
lib.hg_grouped_w4a8_gemm_host.argtypes = [_p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _p,
                                          _p, _p, _p, _sz, _p]
lib.hg_grouped_w4a8_gemm_host.restype = ctypes.c_int

lib.hg_dispatch_tokens.argtypes = [_p, _p, _p, _i32, _i32, _i32, _p, _p]
lib.hg_dispatch_tokens.restype = ctypes.c_int
lib.hg_dispatch_tokens_bwd.argtypes = [_p, _p, _p, _p, _i32, _i32, _i32, _p, _p, _p]
lib.hg_dispatch_tokens_bwd.restype = ctypes.c_int
lib.hg_combine_topk_bwd.argtypes = [_p, _p, _p, _p, _i32, _i32, _i32, _p, _p, _p]
lib.hg_combine_topk_bwd.restype = ctypes.c_int
lib.hg_swiglu_quantize.argtypes = [_p, _i32, _i32, _p, _p, _p, _p, _p]
lib.hg_swiglu_quantize.restype = ctypes.c_int
lib.hg_swiglu_bwd.argtypes = [_p, _p, _p, _i32, _i32, _p, _p]
lib.hg_swiglu_bwd.restype = ctypes.c_int
lib.hg_expert_matvec.argtypes = [_p, _i32, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _p, _p]
lib.hg_expert_matvec.restype = ctypes.c_int
lib.hg_expert_matvec_swiglu.argtypes = lib.hg_expert_matvec.argtypes
lib.hg_expert_matvec_swiglu.restype = ctypes.c_int
lib.hg_router_topk.argtypes = [_p, _i32, _i32, _i32, _i32, _p, _p, _p]
lib.hg_router_topk.restype = ctypes.c_int
lib.hg_router_topk_bwd.argtypes = [_p, _p, _p, _p, _i32, _i32, _i32, _i32, _p, _p]
lib.hg_router_topk_bwd.restype = ctypes.c_int

HG_OK = 0
HG_ERR_INVALID_ARG = 1
HG_ERR_UNSUPPORTED_SHAPE = 2
HG_ERR_RESOURCE = 3
HG_ERR_CUDA = 4
HG_ERR_TIMEOUT = 5
HG_ERR_BAD_OFFSETS = 6
HG_ERR_BAD_IDS = 7


class HgError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.hg_status_string(status).decode()} ({status})")


def _check(status: int, what: str):
    if status != HG_OK:
        raise HgError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# The calls of a decoding step take a few microseconds on the GPU: what they do
# on the host is kept as short.  Addresses go to ctypes as plain integers, and
# the current device and its stream's handle are asked for below torch.cuda,
# where this torch has that (one without CUDA has not).
def _stream_handle(device):
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _addr(t):
    return None if t is None else t.data_ptr()


def _device(like, *others):
    """The GPU that all of these inputs (None aside) are on."""
    device = like.get_device()
    assert device >= 0, "tensors must be on a GPU"
    for t in others:
        assert t is None or t.get_device() == device, "tensors must be on the same GPU"
    return device


def _run(fn, what, device, stream, *args):
    """One call of the library on the tensors' GPU, which need not be the current one, on
    `stream` or that GPU's current stream."""
    if device != _get_device():
        with torch.cuda.device(device):
            return _run(fn, what, device, stream, *args)
    if stream is None:
        stream = _raw_stream(device)
    else:
        assert stream.device_index == device, "the stream must belong to the tensors' GPU"
        stream = stream.cuda_stream
    _check(fn(*args, stream), what)


def _out(given, shape, dtype, like, stream):
    """The caller's output tensor, checked, or a new one that belongs to `stream`."""
    if given is not None:
        assert given.dtype == dtype and given.shape == shape and given.is_contiguous()
        assert given.get_device() == like.get_device(), "tensors must be on the same GPU"
        return given
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def hg_shutdown() -> None:
    """Drop the library's per-device caches (see include/hg.h)."""
    _check(lib.hg_shutdown(), "hg_shutdown")


def hg_plan_workspace_bytes(M: int, top_k: int, E: int) -> int:
    return int(lib.hg_plan_workspace_bytes(M, top_k, E))


def hg_plan_block_threads(E: int, smem_limit_bytes: int) -> int:
    return int(lib.hg_plan_block_threads(E, smem_limit_bytes))


def hg_plan_launches(M: int, top_k: int, E: int) -> int:
    return int(lib.hg_plan_launches(M, top_k, E))


def hg_plan_expert_offsets(topk_ids: torch.Tensor, E: int, expert_offsets=None,
                           sorted_to_src=None, src_to_sorted=None, workspace=None,
                           stream=None):
    """Routing plan on the GPU. Returns (expert_offsets, sorted_to_src, src_to_sorted)."""
    assert topk_ids.dtype == torch.int32 and topk_ids.is_contiguous() and topk_ids.dim() == 2
    M, k = topk_ids.shape
    dev = topk_ids.device
    R = M * k
    if expert_offsets is None:
        expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    if sorted_to_src is None:
        sorted_to_src = torch.empty(R, dtype=torch.int32, device=dev)
    if src_to_sorted is None:
        src_to_sorted = torch.empty(R, dtype=torch.int32, device=dev)
    need = hg_plan_workspace_bytes(M, k, E)
    if workspace is None:
        workspace = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    st = lib.hg_plan_expert_offsets(_ptr(topk_ids), M, k, E, _ptr(expert_offsets),
                                    _ptr(sorted_to_src), _ptr(src_to_sorted), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "hg_plan_expert_offsets")
    return expert_offsets, sorted_to_src, src_to_sorted


def hg_grouped_w4a8_gemm(a_fp8: torch.Tensor, a_scale: torch.Tensor, w_fp4: torch.Tensor,
                         w_scale: torch.Tensor, expert_offsets: torch.Tensor, out=None,
                         stream=None) -> torch.Tensor:
    """Grouped-contiguous W4A8 GEMM. Returns out [rows, N] as torch.bfloat16."""
    E, N, K2 = w_fp4.shape
    K = 2 * K2
    rows = a_fp8.shape[0]
    for t in (a_fp8, a_scale, w_fp4, w_scale, expert_offsets):
        assert t.is_contiguous()
    assert a_fp8.shape == (rows, K) and a_scale.shape == (rows, K // 128)
    assert w_scale.shape == (E, N, K // 32) and expert_offsets.numel() == E + 1
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=a_fp8.device)
    st = lib.hg_grouped_w4a8_gemm(_ptr(a_fp8), _ptr(a_scale), _ptr(w_fp4), _ptr(w_scale),
                                  _ptr(expert_offsets), E, N, K, rows, _ptr(out),
                                  _stream(stream))
    _check(st, "hg_grouped_w4a8_gemm")
    return out


def hg_gemm_host_workspace_bytes(M: int, top_k: int, E: int, N: int, K: int) -> int:
    return int(lib.hg_gemm_host_workspace_bytes(M, top_k, E, N, K))


def hg_grouped_w4a8_gemm_host(topk_ids: torch.Tensor, a_fp8: torch.Tensor, a_scale: torch.Tensor,
                              w_fp4: torch.Tensor, w_scale: torch.Tensor, E: int,
                              out: torch.Tensor, workspace: torch.Tensor,
                              expert_offsets=None, sorted_to_src=None, stream=None):
    """Plan + GEMM from host buffers (CPU tensors, page-locked for asynchronous
    copies): topk_ids int32 [M, top_k], a_fp8 uint8 [M*top_k, K] in the plan's
    order, a_scale uint8 [M*top_k, K/128], out bfloat16 [M*top_k, N]; optional
    host outputs expert_offsets int32 [E+1] and sorted_to_src int32 [M*top_k].
    Weights and workspace (uint8, hg_gemm_host_workspace_bytes) are on the
    device.  Asynchronous on `stream`: the host outputs are valid once the
    stream has reached the end of the call."""
    M, k = topk_ids.shape
    R = M * k
    _, N, K2 = w_fp4.shape
    K = 2 * K2
    for t in (topk_ids, a_fp8, a_scale, out):
        assert not t.is_cuda and t.is_contiguous()
    for t in (expert_offsets, sorted_to_src):
        assert t is None or (not t.is_cuda and t.is_contiguous())
    assert topk_ids.dtype == torch.int32
    assert a_fp8.shape == (R, K) and a_scale.shape == (R, K // 128) and out.shape == (R, N)
    assert expert_offsets is None or expert_offsets.numel() == E + 1
    assert sorted_to_src is None or sorted_to_src.numel() == R
    assert workspace.is_cuda and workspace.dtype == torch.uint8
    st = lib.hg_grouped_w4a8_gemm_host(_ptr(topk_ids), _ptr(a_fp8), _ptr(a_scale), _ptr(w_fp4),
                                       _ptr(w_scale), M, k, E, N, K, _ptr(out),
                                       _ptr(expert_offsets), _ptr(sorted_to_src), _ptr(workspace),
                                       workspace.numel(), _stream(stream))
    _check(st, "hg_grouped_w4a8_gemm_host")
    return out


def hg_grouped_w4a8_gemm_mmajor(a_fp8: torch.Tensor, a_scale_mmajor: torch.Tensor,
                                w_fp4: torch.Tensor, w_scale: torch.Tensor,
                                expert_offsets: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """The GEMM with activation scales laid out [K/128, rows]. Returns out [rows, N] bf16."""
    E, N, K2 = w_fp4.shape
    K = 2 * K2
    rows = a_fp8.shape[0]
    for t in (a_fp8, a_scale_mmajor, w_fp4, w_scale, expert_offsets):
        assert t.is_contiguous()
    assert a_fp8.shape == (rows, K) and a_scale_mmajor.shape == (K // 128, rows)
    assert w_scale.shape == (E, N, K // 32) and expert_offsets.numel() == E + 1
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=a_fp8.device)
    st = lib.hg_grouped_w4a8_gemm_mmajor(_ptr(a_fp8), _ptr(a_scale_mmajor), _ptr(w_fp4),
                                         _ptr(w_scale), _ptr(expert_offsets), E, N, K, rows,
                                         _ptr(out), _stream(stream))
    _check(st, "hg_grouped_w4a8_gemm_mmajor")
    return out


def hg_quantize_gather_acts(x_bf16: torch.Tensor, top_k: int, sorted_to_src: torch.Tensor,
                            a_fp8=None, a_scale=None, stream=None):
    """BF16 [M, K] tokens -> (E4M3 [M*top_k, K], E8M0 [M*top_k, K/128]) in sorted order."""
    assert x_bf16.dtype == torch.bfloat16 and x_bf16.is_contiguous() and x_bf16.dim() == 2
    M, K = x_bf16.shape
    R = M * top_k
    if a_fp8 is None:
        a_fp8 = torch.empty((R, K), dtype=torch.uint8, device=x_bf16.device)
    if a_scale is None:
        a_scale = torch.empty((R, K // 128), dtype=torch.uint8, device=x_bf16.device)
    st = lib.hg_quantize_gather_acts(_ptr(x_bf16), M, K, top_k, _ptr(sorted_to_src), _ptr(a_fp8),
                                     _ptr(a_scale), _stream(stream))
    _check(st, "hg_quantize_gather_acts")
    return a_fp8, a_scale


def hg_quantize_scatter_acts(x_bf16: torch.Tensor, top_k: int, src_to_sorted: torch.Tensor,
                             a_fp8=None, a_scale=None, stream=None):
    """BF16 [M, K] tokens -> (E4M3 [M*top_k, K], E8M0 [M*top_k, K/128]); token t's codes
    go to rows src_to_sorted[t*top_k + j]."""
    assert x_bf16.dtype == torch.bfloat16 and x_bf16.is_contiguous() and x_bf16.dim() == 2
    M, K = x_bf16.shape
    R = M * top_k
    if a_fp8 is None:
        a_fp8 = torch.empty((R, K), dtype=torch.uint8, device=x_bf16.device)
    if a_scale is None:
        a_scale = torch.empty((R, K // 128), dtype=torch.uint8, device=x_bf16.device)
    st = lib.hg_quantize_scatter_acts(_ptr(x_bf16), M, K, top_k, _ptr(src_to_sorted),
                                      _ptr(a_fp8), _ptr(a_scale), _stream(stream))
    _check(st, "hg_quantize_scatter_acts")
    return a_fp8, a_scale


def hg_combine_topk(y_bf16: torch.Tensor, src_to_sorted: torch.Tensor, topk_weights: torch.Tensor,
                    out=None, stream=None) -> torch.Tensor:
    """out[t] = sum_j w[t, j] * y[src_to_sorted[t*k + j]]  (FP32 sum, BF16 result)."""
    M, k = topk_weights.shape
    N = y_bf16.shape[1]
    assert topk_weights.dtype == torch.float32 and topk_weights.is_contiguous()
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=y_bf16.device)
    st = lib.hg_combine_topk(_ptr(y_bf16), _ptr(src_to_sorted), _ptr(topk_weights), M, k, N,
                             _ptr(out), _stream(stream))
    _check(st, "hg_combine_topk")
    return out


def hg_dispatch_tokens(x_bf16: torch.Tensor, top_k: int, src_to_sorted: torch.Tensor,
                       topk_weights=None, out=None, stream=None) -> torch.Tensor:
    """rows[src_to_sorted[t*k + j]] = w[t, j] * x[t] (w = 1 without weights), BF16 [M*top_k, K].
    Rows that no entry names are not written."""
    M, K = x_bf16.shape
    assert x_bf16.dtype == _BF16 and x_bf16.is_contiguous()
    assert src_to_sorted.dtype == _I32 and src_to_sorted.numel() == M * top_k
    assert src_to_sorted.is_contiguous()
    assert topk_weights is None or (topk_weights.dtype == _F32 and
                                    topk_weights.shape == (M, top_k) and
                                    topk_weights.is_contiguous())
    device = _device(x_bf16, src_to_sorted, topk_weights)
    out = _out(out, (M * top_k, K), _BF16, x_bf16, stream)
    _run(lib.hg_dispatch_tokens, "hg_dispatch_tokens", device, stream, x_bf16.data_ptr(),
         src_to_sorted.data_ptr(), _addr(topk_weights), M, top_k, K, out.data_ptr())
    return out


def hg_dispatch_tokens_bwd(drows: torch.Tensor, top_k: int, src_to_sorted: torch.Tensor,
                           topk_weights=None, x_bf16=None, dx=None, dweights=None, stream=None):
    """Gradient of hg_dispatch_tokens: (dx [M, K] BF16, dweights [M, top_k] float32).
    dweights is None unless the forward input x_bf16 is given."""
    R, K = drows.shape
    M = src_to_sorted.numel() // top_k
    assert drows.dtype == _BF16 and drows.is_contiguous() and R == M * top_k
    assert src_to_sorted.dtype == _I32 and src_to_sorted.numel() == R
    assert src_to_sorted.is_contiguous()
    assert topk_weights is None or (topk_weights.dtype == _F32 and
                                    topk_weights.shape == (M, top_k) and
                                    topk_weights.is_contiguous())
    device = _device(drows, src_to_sorted, topk_weights, x_bf16)
    dx = _out(dx, (M, K), _BF16, drows, stream)
    if x_bf16 is not None:
        assert x_bf16.dtype == _BF16 and x_bf16.shape == (M, K) and x_bf16.is_contiguous()
        dweights = _out(dweights, (M, top_k), _F32, drows, stream)
    else:
        assert dweights is None
    _run(lib.hg_dispatch_tokens_bwd, "hg_dispatch_tokens_bwd", device, stream, drows.data_ptr(),
         _addr(x_bf16), src_to_sorted.data_ptr(), _addr(topk_weights), M, top_k, K, dx.data_ptr(),
         _addr(dweights))
    return dx, dweights


def hg_combine_topk_bwd(dout: torch.Tensor, y_bf16: torch.Tensor, src_to_sorted: torch.Tensor,
                        topk_weights: torch.Tensor, dy=None, dweights=None, stream=None):
    """Gradient of hg_combine_topk: (dy [M*top_k, N] BF16, dweights [M, top_k] float32)."""
    M, k = topk_weights.shape
    N = dout.shape[1]
    assert dout.dtype == _BF16 and dout.shape == (M, N) and dout.is_contiguous()
    assert y_bf16.dtype == _BF16 and y_bf16.shape == (M * k, N) and y_bf16.is_contiguous()
    assert topk_weights.dtype == _F32 and topk_weights.is_contiguous()
    assert src_to_sorted.dtype == _I32 and src_to_sorted.numel() == M * k
    assert src_to_sorted.is_contiguous()
    device = _device(dout, y_bf16, topk_weights, src_to_sorted)
    dy = _out(dy, (M * k, N), _BF16, dout, stream)
    dweights = _out(dweights, (M, k), _F32, dout, stream)
    _run(lib.hg_combine_topk_bwd, "hg_combine_topk_bwd", device, stream, dout.data_ptr(),
         y_bf16.data_ptr(), src_to_sorted.data_ptr(), topk_weights.data_ptr(), M, k, N,
         dy.data_ptr(), dweights.data_ptr())
    return dy, dweights


def hg_swiglu_quantize(z_bf16: torch.Tensor, checkpoint: bool = True, a_fp8=None, a_scale=None,
                       z_fp8=None, z_scale=None, stream=None):
    """silu(g) * u of z = (g, u) [rows, 2F] as the next GEMM's (a_fp8, a_scale), and with
    `checkpoint` z itself in 8 bits (z_fp8, z_scale), else None in their places."""
    rows, F2 = z_bf16.shape
    assert z_bf16.dtype == _BF16 and z_bf16.is_contiguous() and F2 % 2 == 0
    F = F2 // 2
    device = _device(z_bf16)
    a_fp8 = _out(a_fp8, (rows, F), _U8, z_bf16, stream)
    a_scale = _out(a_scale, (rows, F // 128), _U8, z_bf16, stream)
    if checkpoint:
        z_fp8 = _out(z_fp8, (rows, F2), _U8, z_bf16, stream)
        z_scale = _out(z_scale, (rows, F2 // 128), _U8, z_bf16, stream)
    else:
        assert z_fp8 is None and z_scale is None
    _run(lib.hg_swiglu_quantize, "hg_swiglu_quantize", device, stream, z_bf16.data_ptr(), rows, F,
         a_fp8.data_ptr(), a_scale.data_ptr(), _addr(z_fp8), _addr(z_scale))
    return a_fp8, a_scale, z_fp8, z_scale


def hg_swiglu_bwd(dh: torch.Tensor, z_fp8: torch.Tensor, z_scale: torch.Tensor, dz=None,
                  stream=None) -> torch.Tensor:
    """Gradient of silu(g) * u from the 8-bit checkpoint of (g, u): dz [rows, 2F] BF16."""
    rows, F = dh.shape
    assert dh.dtype == _BF16 and dh.is_contiguous()
    assert z_fp8.dtype == _U8 and z_fp8.shape == (rows, 2 * F) and z_fp8.is_contiguous()
    assert z_scale.dtype == _U8 and z_scale.shape == (rows, 2 * F // 128)
    assert z_scale.is_contiguous()
    device = _device(dh, z_fp8, z_scale)
    dz = _out(dz, (rows, 2 * F), _BF16, dh, stream)
    _run(lib.hg_swiglu_bwd, "hg_swiglu_bwd", device, stream, dh.data_ptr(), z_fp8.data_ptr(),
         z_scale.data_ptr(), rows, F, dz.data_ptr())
    return dz


def _expert_matvec(fn, what, cols, x_bf16, topk_ids, w_fp4, w_scale, out, stream):
    M, k = topk_ids.shape
    E, N, K2 = w_fp4.shape
    K = 2 * K2
    assert x_bf16.dtype == _BF16 and x_bf16.is_contiguous() and x_bf16.shape[1] == K
    assert topk_ids.dtype == _I32 and topk_ids.is_contiguous()
    assert w_fp4.dtype == _U8 and w_fp4.is_contiguous()
    assert w_scale.dtype == _U8 and w_scale.is_contiguous()
    assert w_scale.shape == (E, N, K // 32)
    device = _device(x_bf16, topk_ids, w_fp4, w_scale)
    out = _out(out, (M * k, cols(N)), _BF16, x_bf16, stream)
    _run(fn, what, device, stream, x_bf16.data_ptr(), x_bf16.shape[0], topk_ids.data_ptr(),
         w_fp4.data_ptr(), w_scale.data_ptr(), M, k, E, N, K, out.data_ptr())
    return out


def hg_expert_matvec(x_bf16: torch.Tensor, topk_ids: torch.Tensor, w_fp4: torch.Tensor,
                     w_scale: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """y[t*k + j] = W[topk_ids[t, j]] x: BF16 [M*top_k, N].  x_bf16 has M rows (shared by a
    token's slots) or M*top_k (one a slot)."""
    return _expert_matvec(lib.hg_expert_matvec, "hg_expert_matvec", lambda N: N, x_bf16, topk_ids,
                          w_fp4, w_scale, out, stream)


def hg_expert_matvec_swiglu(x_bf16: torch.Tensor, topk_ids: torch.Tensor, w_fp4: torch.Tensor,
                            w_scale: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """silu(y[:, :N/2]) * y[:, N/2:] of hg_expert_matvec's y: BF16 [M*top_k, N/2]."""
    return _expert_matvec(lib.hg_expert_matvec_swiglu, "hg_expert_matvec_swiglu",
                          lambda N: N // 2, x_bf16, topk_ids, w_fp4, w_scale, out, stream)


def hg_router_topk(logits: torch.Tensor, top_k: int, renormalize: bool = True, ids=None,
                   weights=None, stream=None):
    """(topk_ids int32 [M, top_k], topk_weights float32 [M, top_k]) of float32 logits [M, E]."""
    M, E = logits.shape
    assert logits.dtype == _F32 and logits.is_contiguous()
    device = _device(logits)
    ids = _out(ids, (M, top_k), _I32, logits, stream)
    weights = _out(weights, (M, top_k), _F32, logits, stream)
    _run(lib.hg_router_topk, "hg_router_topk", device, stream, logits.data_ptr(), M, E, top_k,
         int(renormalize), ids.data_ptr(), weights.data_ptr())
    return ids, weights


def hg_router_topk_bwd(logits: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                       dweights: torch.Tensor, renormalize: bool = True, dlogits=None,
                       stream=None) -> torch.Tensor:
    """Gradient of hg_router_topk with respect to the logits: float32 [M, E]."""
    M, E = logits.shape
    k = topk_ids.shape[1]
    assert logits.dtype == _F32 and logits.is_contiguous()
    assert topk_ids.dtype == _I32 and topk_ids.shape == (M, k) and topk_ids.is_contiguous()
    for t in (topk_weights, dweights):
        assert t.dtype == _F32 and t.shape == (M, k) and t.is_contiguous()
    device = _device(logits, topk_ids, topk_weights, dweights)
    dlogits = _out(dlogits, (M, E), _F32, logits, stream)
    _run(lib.hg_router_topk_bwd, "hg_router_topk_bwd", device, stream, logits.data_ptr(),
         topk_ids.data_ptr(), topk_weights.data_ptr(), dweights.data_ptr(), M, E, k,
         int(renormalize), dlogits.data_ptr())
    return dlogits


def hg_get_device_status(stream=None):
    """(status, detail) of the device status word; synchronises the stream."""
    detail = _u32(0)
    st = lib.hg_get_device_status(_stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def hg_selftest_wait_timeout(timeout_us: int, stream=None):
    _check(lib.hg_selftest_wait_timeout(timeout_us, _stream(stream)), "hg_selftest_wait_timeout")


def hg_set_wait_timeout_us(timeout_us: int):
    lib.hg_set_wait_timeout_us(timeout_us)


def hg_gemm_token_tile(E: int, N: int, K: int, rows: int) -> int:
    return int(lib.hg_gemm_token_tile(E, N, K, rows))


def hg_gemm_ctas(E: int, N: int, K: int, rows: int) -> int:
    return int(lib.hg_gemm_ctas(E, N, K, rows))


def hg_set_gemm_variant(variant: int) -> int:
    prev = int(lib.hg_set_gemm_variant(variant))
    if prev < 0:
        raise ValueError(f"invalid GEMM variant {variant}")
    return prev
