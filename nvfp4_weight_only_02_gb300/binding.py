"""Thin ctypes binding of libnvfp4.so (argument marshalling only).

Every function here takes CUDA tensors of the current device, checks devices,
dtypes and shapes, and passes
raw device pointers, sizes and the current CUDA stream to the C ABI declared
in include/nvfp4.h.  All arithmetic happens in the library's CUDA kernels;
if the library is missing, loading fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

_lib = None
_lock = threading.Lock()

OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_UNSUPPORTED_DEVICE, ERR_CUDA, \
    ERR_NONFINITE, ERR_TIMEOUT, ERR_INDEX = range(10)
OUT_BF16, OUT_FP32 = 0, 1
FORMAT_MXFP4, FORMAT_NVFP4 = 0, 1

EXPORTS = [
    "nvfp4_workspace_bytes", "nvfp4_quantize", "nvfp4_dequantize", "nvfp4_w4a16_lora_gemm",
    "nvfp4_round_scales", "nvfp4_get_device_status", "nvfp4_status_string", "nvfp4_encode_debug",
    "nvfp4_quotient_check", "nvfp4_w4a16_lora_gemm_static", "nvfp4_wait_selftest", "nvfp4_gemm_kernel",
    "nvfp4_scale_qlora_gemm", "nvfp4_w4a16_lora_gemm_dgrad", "nvfp4_dgrad_workspace_bytes",
    "nvfp4_lora_grads", "nvfp4_lora_grads_workspace_bytes", "nvfp4_gemm_list_workspace_bytes",
    "nvfp4_w4a16_lora_gemm_list", "nvfp4_tiled_scale_bytes", "nvfp4_tile_scales", "nvfp4_mx_quantize",
    "nvfp4_mx_dequantize", "nvfp4_w4a4_workspace_bytes", "nvfp4_w4a4_gemm", "nvfp4_mx_linear_workspace_bytes",
    "nvfp4_mx_linear", "nvfp4_mx_linear_backward_workspace_bytes", "nvfp4_mx_linear_backward", "nvfp4_distill_topk",
    "nvfp4_distill_wait_selftest",
]


class Projection(ctypes.Structure):
    """struct nvfp4_projection (one entry of nvfp4_w4a16_lora_gemm_list)."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales_e4m3", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("lora_a_bf16", ctypes.c_void_p),
                ("lora_b_bf16", ctypes.c_void_p), ("noise_fp32", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("lora_scale", ctypes.c_float)]


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libnvfp4.so (building it with nvcc when it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if build_if_missing and _build.is_stale():
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"libnvfp4.so not found at {path}; run nvfp4_weight_only_02_gb300/build.py")
        lib = ctypes.CDLL(path)
        P, i64, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32
        st = ctypes.c_int
        sig = {
            "nvfp4_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i64]),
            "nvfp4_quantize": (st, [P, i64, i64, P, P, P, ctypes.c_int, P, ctypes.c_size_t, P]),
            "nvfp4_dequantize": (st, [P, P, P, i64, i64, P, ctypes.c_int, P]),
            "nvfp4_w4a16_lora_gemm": (st, [P, i64, i64, i64, P, P, P, P, P, i64, ctypes.c_float, P, P,
                                           ctypes.c_int, P, ctypes.c_size_t, P]),
            "nvfp4_round_scales": (st, [P, P, i64, i64, P, P, ctypes.c_size_t, P]),
            "nvfp4_get_device_status": (st, [P, P]),
            "nvfp4_status_string": (ctypes.c_char_p, [st]),
            "nvfp4_encode_debug": (st, [P, i64, ctypes.c_int, P, P]),
            "nvfp4_quotient_check": (st, [u32, u32, P, P]),
            "nvfp4_w4a16_lora_gemm_static": (st, [P, i64, i64, i64, P, P, P, P, P, i64, ctypes.c_float,
                                                  P, P, ctypes.c_int, P]),
            "nvfp4_wait_selftest": (st, [P, ctypes.c_int, P]),
            "nvfp4_gemm_kernel": (ctypes.c_char_p, [i64, i64, i64, i64]),
            "nvfp4_scale_qlora_gemm": (st, [P, i64, i64, i64, P, P, P, P, P, P, i64, ctypes.c_float, P, P,
                                            ctypes.c_int, P, ctypes.c_size_t, P]),
            "nvfp4_w4a16_lora_gemm_dgrad": (st, [P, i64, i64, i64, P, P, P, P, P, i64, ctypes.c_float, P, P,
                                                 ctypes.c_int, P, ctypes.c_size_t, P]),
            "nvfp4_dgrad_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i64]),
            "nvfp4_lora_grads": (st, [P, P, P, i64, i64, i64, P, P, i64, ctypes.c_float, P, P, P, ctypes.c_size_t,
                                      P]),
            "nvfp4_lora_grads_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64, i64]),
            "nvfp4_gemm_list_workspace_bytes": (ctypes.c_size_t, [P, ctypes.c_int, i64, i64]),
            "nvfp4_w4a16_lora_gemm_list": (st, [P, ctypes.c_int, i64, i64, ctypes.c_int, P, ctypes.c_size_t, P]),
            "nvfp4_tiled_scale_bytes": (ctypes.c_size_t, [i64, i64, ctypes.c_int]),
            "nvfp4_tile_scales": (st, [P, i64, i64, ctypes.c_int, P, P]),
            "nvfp4_mx_quantize": (st, [P, ctypes.c_int, i64, i64, i64, P, P, P, P, P, P, P]),
            "nvfp4_mx_dequantize": (st, [P, P, i64, i64, P, ctypes.c_int, P]),
            "nvfp4_w4a4_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64]),
            "nvfp4_w4a4_gemm": (st, [ctypes.c_int, P, P, P, P, P, P, i64, i64, i64, P, ctypes.c_int, P,
                                     ctypes.c_size_t, P]),
            "nvfp4_mx_linear_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64]),
            "nvfp4_mx_linear": (st, [P, ctypes.c_int, i64, i64, i64, i64, P, P, P, ctypes.c_int, P, ctypes.c_size_t,
                                     P]),
            "nvfp4_mx_linear_backward_workspace_bytes": (ctypes.c_size_t, [i64, i64, i64]),
            "nvfp4_mx_linear_backward": (st, [P, ctypes.c_int, i64, i64, i64, i64, P, P, P, P, P, ctypes.c_int, P,
                                              ctypes.c_int, P, ctypes.c_size_t, P]),
            "nvfp4_distill_topk": (st, [P, ctypes.c_int, i64, i64, i64, P, ctypes.c_int, P, ctypes.c_int, i64,
                                        ctypes.c_float, ctypes.c_int, P, P, i64, P, P, i64, P, ctypes.c_size_t, P]),
            "nvfp4_distill_wait_selftest": (st, [P, ctypes.c_int, i64, i64, P, P, i64, ctypes.c_int, P, P, P, P,
                                                 ctypes.c_size_t, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
        return lib


def gemm_kernel(M: int, N: int, K: int, r: int = 0):
    """Kernel family nvfp4_w4a16_lora_gemm runs for these sizes (None if unsupported)."""
    name = load().nvfp4_gemm_kernel(M, N, K, r)
    return None if name is None else name.decode()


def status_string(status: int) -> str:
    return load().nvfp4_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise NVFP4Error(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


# index of the current device, and the raw handle of a device's current stream (no Stream object is built)
_current = getattr(torch._C, "_cuda_getDevice", None)
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device_of(t, name):
    """Index of t's device, which has to be the current one: kernels run on its stream, and an address of another
    device or of the host would fault there."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current():
        raise ValueError(f"{name} must be on the current device, cuda:{_current()}, got cuda:{dev}")
    return dev


def _space(workspace):
    if workspace is None:
        return None
    _device_of(workspace, "workspace")
    return ctypes.c_void_p(workspace.data_ptr())


def _need(t, dtype, shape, name, dev=None):
    """dev: the current device, where the caller has it at hand."""
    if t.get_device() != (_current() if dev is None else dev):
        _device_of(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------ workspace
def nvfp4_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(load().nvfp4_workspace_bytes(M, N, K, r))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled workspace (the library keeps it zeroed between calls)."""
    n = max(256, (int(nbytes) + 255) // 256 * 256)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def nvfp4_get_device_status(workspace: torch.Tensor) -> int:
    return int(load().nvfp4_get_device_status(_space(workspace), _stream()))


# ------------------------------------------------------------------ entry points
def nvfp4_quantize(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                   tensor_scale: torch.Tensor, use_given_tensor_scale: bool,
                   workspace: torch.Tensor):
    N, K = w.shape
    _need(w, torch.bfloat16, (N, K), "w")
    _need(codes, torch.uint8, (N, K // 2), "codes")
    _need(scales, torch.uint8, (N, K // 16), "scales")
    _need(tensor_scale, torch.float32, (1,), "tensor_scale")
    st = load().nvfp4_quantize(_ptr(w), N, K, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
                               int(bool(use_given_tensor_scale)), _space(workspace),
                               workspace.numel(), _stream())
    _check(st, "nvfp4_quantize")


def nvfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, tensor_scale: torch.Tensor,
                     out: torch.Tensor):
    N, K2 = codes.shape
    K = K2 * 2
    _need(scales, torch.uint8, (N, K // 16), "scales")
    _need(tensor_scale, torch.float32, (1,), "tensor_scale")
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out must be float32 or bfloat16")
    _need(out, out.dtype, (N, K), "out")
    st = load().nvfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(tensor_scale), N, K, _ptr(out),
                                 OUT_FP32 if out.dtype == torch.float32 else OUT_BF16, _stream())
    _check(st, "nvfp4_dequantize")


def nvfp4_w4a16_lora_gemm(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                          tensor_scale: torch.Tensor, lora_a, lora_b, lora_scale: float,
                          noise, y: torch.Tensor, workspace: torch.Tensor):
    M, K = x.shape
    N = codes.shape[0]
    _need(x, torch.bfloat16, (M, K), "x")
    _need(codes, torch.uint8, (N, K // 2), "codes")
    _need(scales, torch.uint8, (N, K // 16), "scales")
    _need(tensor_scale, torch.float32, (1,), "tensor_scale")
    r = 0
    if lora_a is not None:
        r = lora_a.shape[0]
        _need(lora_a, torch.bfloat16, (r, K), "lora_a")
        _need(lora_b, torch.bfloat16, (N, r), "lora_b")
    if noise is not None:
        _need(noise, torch.float32, (K,), "noise")
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("y must be float32 or bfloat16")
    _need(y, y.dtype, (M, N), "y")
    st = load().nvfp4_w4a16_lora_gemm(
        _ptr(x), M, N, K, _ptr(codes), _ptr(scales), _ptr(tensor_scale), _ptr(lora_a),
        _ptr(lora_b), r, float(lora_scale), _ptr(noise), _ptr(y),
        OUT_FP32 if y.dtype == torch.float32 else OUT_BF16, _space(workspace), workspace.numel(),
        _stream())
    _check(st, "nvfp4_w4a16_lora_gemm")


def _projection_array(entries):
    """entries: (x, codes, scales, tensor_scale, lora_a, lora_b, lora_scale, noise, y) tuples of CUDA
    tensors (lora_a, lora_b, noise may be None).  Returns (ctypes array, M, r, y dtype code)."""
    if len(entries) == 0:
        raise ValueError("empty projection list")
    M = entries[0][0].shape[0]
    r = 0 if entries[0][4] is None else entries[0][4].shape[0]
    ydt = entries[0][8].dtype
    if ydt not in (torch.float32, torch.bfloat16):
        raise ValueError("y must be float32 or bfloat16")
    arr = (Projection * len(entries))()
    dev = _current()
    for i, (x, codes, scales, ts, a, b, s, z, y) in enumerate(entries):
        K = x.shape[1]
        N = codes.shape[0]
        _need(x, torch.bfloat16, (M, K), f"x[{i}]", dev)
        _need(codes, torch.uint8, (N, K // 2), f"codes[{i}]", dev)
        _need(scales, torch.uint8, (N, K // 16), f"scales[{i}]", dev)
        _need(ts, torch.float32, (1,), f"tensor_scale[{i}]", dev)
        if (a is None) != (r == 0):
            raise ValueError("every entry of a list has the same LoRA rank")
        if a is not None:
            _need(a, torch.bfloat16, (r, K), f"lora_a[{i}]", dev)
            _need(b, torch.bfloat16, (N, r), f"lora_b[{i}]", dev)
        if z is not None:
            _need(z, torch.float32, (K,), f"noise[{i}]", dev)
        _need(y, ydt, (M, N), f"y[{i}]", dev)
        arr[i] = Projection(_ptr(x), _ptr(codes), _ptr(scales), _ptr(ts), _ptr(a), _ptr(b), _ptr(z), _ptr(y),
                            N, K, float(s))
    return arr, M, r, OUT_FP32 if ydt == torch.float32 else OUT_BF16


def nvfp4_gemm_list_workspace_bytes(entries) -> int:
    arr, M, r, _ = _projection_array(entries)
    return int(load().nvfp4_gemm_list_workspace_bytes(arr, len(entries), M, r))


def nvfp4_w4a16_lora_gemm_list(entries, workspace: torch.Tensor):
    """Independent projections of one token count in one call (see _projection_array for an entry)."""
    arr, M, r, ydt = _projection_array(entries)
    st = load().nvfp4_w4a16_lora_gemm_list(arr, len(entries), M, r, ydt, _space(workspace), workspace.numel(),
                                           _stream())
    _check(st, "nvfp4_w4a16_lora_gemm_list")


def nvfp4_round_scales(scale_param: torch.Tensor, tensor_scale: torch.Tensor,
                       scales: torch.Tensor, workspace: torch.Tensor):
    N, KB = scale_param.shape
    _need(scale_param, torch.float32, (N, KB), "scale_param")
    _need(scales, torch.uint8, (N, KB), "scales")
    _need(tensor_scale, torch.float32, (1,), "tensor_scale")
    st = load().nvfp4_round_scales(_ptr(scale_param), _ptr(tensor_scale), N, KB * 16,
                                   _ptr(scales), _space(workspace), workspace.numel(), _stream())
    _check(st, "nvfp4_round_scales")


def nvfp4_scale_qlora_gemm(x: torch.Tensor, codes: torch.Tensor, scale_param: torch.Tensor,
                           tensor_scale: torch.Tensor, scales: torch.Tensor, lora_a, lora_b,
                           lora_scale: float, noise, y: torch.Tensor, workspace: torch.Tensor):
    M, K = x.shape
    N = codes.shape[0]
    _need(x, torch.bfloat16, (M, K), "x")
    _need(codes, torch.uint8, (N, K // 2), "codes")
    _need(scale_param, torch.float32, (N, K // 16), "scale_param")
    _need(scales, torch.uint8, (N, K // 16), "scales")
    _need(tensor_scale, torch.float32, (1,), "tensor_scale")
    r = 0
    if lora_a is not None:
        r = lora_a.shape[0]
        _need(lora_a, torch.bfloat16, (r, K), "lora_a")
        _need(lora_b, torch.bfloat16, (N, r), "lora_b")
    if noise is not None:
        _need(noise, torch.float32, (K,), "noise")
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("y must be float32 or bfloat16")
    _need(y, y.dtype, (M, N), "y")
    st = load().nvfp4_scale_qlora_gemm(
        _ptr(x), M, N, K, _ptr(codes), _ptr(scale_param), _ptr(tensor_scale), _ptr(scales),
        _ptr(lora_a), _ptr(lora_b), r, float(lora_scale), _ptr(noise), _ptr(y),
        OUT_FP32 if y.dtype == torch.float32 else OUT_BF16, _space(workspace), workspace.numel(),
        _stream())
    _check(st, "nvfp4_scale_qlora_gemm")


def nvfp4_encode_debug(x: torch.Tensor, which: int) -> torch.Tensor:
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    st = load().nvfp4_encode_debug(_ptr(x), x.numel(), int(which), _ptr(out), _stream())
    _check(st, "nvfp4_encode_debug")
    return out


def nvfp4_wait_selftest(workspace: torch.Tensor, which: int):
    _check(load().nvfp4_wait_selftest(_space(workspace), int(which), _stream()), "nvfp4_wait_selftest")


def nvfp4_quotient_check(sig_lo: int, sig_hi: int) -> int:
    cnt = torch.zeros(1, dtype=torch.int64, device="cuda")
    st = load().nvfp4_quotient_check(sig_lo, sig_hi, _ptr(cnt), _stream())
    _check(st, "nvfp4_quotient_check")
    return int(cnt.item())


# ------------------------------------------------------------------ conveniences
class QuantizedWeight:
    """Device buffers of one NVFP4 weight: codes, scales and tensor scale."""

    def __init__(self, codes, scales, tensor_scale):
        self.codes, self.scales, self.tensor_scale = codes, scales, tensor_scale

    @property
    def shape(self):
        return self.codes.shape[0], self.codes.shape[1] * 2


def quantize(w: torch.Tensor, tensor_scale=None, workspace=None) -> QuantizedWeight:
    N, K = w.shape
    dev = w.device
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
    ts = torch.zeros(1, dtype=torch.float32, device=dev)
    if tensor_scale is not None:
        ts.fill_(float(tensor_scale))
    ws = workspace if workspace is not None else new_workspace(256, dev)
    nvfp4_quantize(w, codes, scales, ts, tensor_scale is not None, ws)
    return QuantizedWeight(codes, scales, ts)


def dequantize(q: QuantizedWeight, dtype=torch.float32) -> torch.Tensor:
    out = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
    nvfp4_dequantize(q.codes, q.scales, q.tensor_scale, out)
    return out


def nvfp4_dgrad_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(load().nvfp4_dgrad_workspace_bytes(M, N, K, r))


def nvfp4_w4a16_lora_gemm_dgrad(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                                tensor_scale: torch.Tensor, lora_a, lora_b, lora_scale: float,
                                noise, dx: torch.Tensor, workspace: torch.Tensor):
    M, N = dy.shape
    K = codes.shape[1] * 2
    _need(dy, torch.bfloat16, (M, N), "dy")
    _need(codes, torch.uint8, (N, K // 2), "codes")
    _need(scales, torch.uint8, (N, K // 16), "scales")
    _need(tensor_scale, torch.float32, (1,), "tensor_scale")
    r = 0
    if lora_a is not None:
        r = lora_a.shape[0]
        _need(lora_a, torch.bfloat16, (r, K), "lora_a")
        _need(lora_b, torch.bfloat16, (N, r), "lora_b")
    if noise is not None:
        _need(noise, torch.float32, (K,), "noise")
    if dx.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dx must be float32 or bfloat16")
    _need(dx, dx.dtype, (M, K), "dx")
    st = load().nvfp4_w4a16_lora_gemm_dgrad(
        _ptr(dy), M, N, K, _ptr(codes), _ptr(scales), _ptr(tensor_scale), _ptr(lora_a),
        _ptr(lora_b), r, float(lora_scale), _ptr(noise), _ptr(dx),
        OUT_FP32 if dx.dtype == torch.float32 else OUT_BF16, _space(workspace), workspace.numel(),
        _stream())
    _check(st, "nvfp4_w4a16_lora_gemm_dgrad")


def gemm_dgrad(dy, q: "QuantizedWeight", lora_a=None, lora_b=None, lora_scale=0.0, noise=None,
               out_dtype=torch.float32, workspace=None) -> torch.Tensor:
    """dX = (dY deq(W) + s (dY B) A) diag(z), the input gradient of gemm()."""
    M, N = dy.shape
    K = q.shape[1]
    r = 0 if lora_a is None else lora_a.shape[0]
    dx = torch.empty((M, K), dtype=out_dtype, device=dy.device)
    ws = workspace if workspace is not None else new_workspace(nvfp4_dgrad_workspace_bytes(M, N, K, r),
                                                              dy.device)
    nvfp4_w4a16_lora_gemm_dgrad(dy, q.codes, q.scales, q.tensor_scale, lora_a, lora_b, lora_scale, noise,
                                dx, ws)
    return dx


def nvfp4_lora_grads_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(load().nvfp4_lora_grads_workspace_bytes(M, N, K, r))


def nvfp4_lora_grads(x: torch.Tensor, noise, dy: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                     lora_scale: float, grad_a: torch.Tensor, grad_b: torch.Tensor, workspace: torch.Tensor):
    M, K = x.shape
    N = dy.shape[1]
    r = lora_a.shape[0]
    _need(x, torch.bfloat16, (M, K), "x")
    _need(dy, torch.bfloat16, (M, N), "dy")
    _need(lora_a, torch.bfloat16, (r, K), "lora_a")
    _need(lora_b, torch.bfloat16, (N, r), "lora_b")
    _need(grad_a, torch.float32, (r, K), "grad_a")
    _need(grad_b, torch.float32, (N, r), "grad_b")
    if noise is not None:
        _need(noise, torch.float32, (K,), "noise")
    st = load().nvfp4_lora_grads(_ptr(x), _ptr(noise), _ptr(dy), M, N, K, _ptr(lora_a), _ptr(lora_b), r,
                                 float(lora_scale), _ptr(grad_a), _ptr(grad_b), _space(workspace),
                                 workspace.numel(), _stream())
    _check(st, "nvfp4_lora_grads")


def lora_grads(x, dy, lora_a, lora_b, lora_scale, noise=None, workspace=None):
    """(dA (r, K), dB (N, r)) float32: dA = s (dY B)^T X', dB = s dY^T (X' A^T)."""
    M, K = x.shape
    N = dy.shape[1]
    r = lora_a.shape[0]
    ga = torch.empty((r, K), dtype=torch.float32, device=x.device)
    gb = torch.empty((N, r), dtype=torch.float32, device=x.device)
    ws = workspace if workspace is not None else new_workspace(nvfp4_lora_grads_workspace_bytes(M, N, K, r),
                                                              x.device)
    nvfp4_lora_grads(x, noise, dy, lora_a, lora_b, lora_scale, ga, gb, ws)
    return ga, gb


def gemm_list(items, out_dtype=torch.float32, workspace=None):
    """items: (x, q, lora_a, lora_b, lora_scale, noise) tuples (q a QuantizedWeight; lora_a, lora_b,
    noise may be None).  Returns the list of outputs, each M x N."""
    entries = []
    for x, q, a, b, s, z in items:
        y = torch.empty((x.shape[0], q.shape[0]), dtype=out_dtype, device=x.device)
        entries.append((x, q.codes, q.scales, q.tensor_scale, a, b, s, z, y))
    ws = workspace if workspace is not None else new_workspace(nvfp4_gemm_list_workspace_bytes(entries),
                                                              entries[0][0].device)
    nvfp4_w4a16_lora_gemm_list(entries, ws)
    return [e[8] for e in entries]


def gemm(x, q: QuantizedWeight, lora_a=None, lora_b=None, lora_scale=0.0, noise=None,
         out_dtype=torch.float32, workspace=None) -> torch.Tensor:
    M, K = x.shape
    N = q.shape[0]
    r = 0 if lora_a is None else lora_a.shape[0]
    y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    ws = workspace if workspace is not None else new_workspace(nvfp4_workspace_bytes(M, N, K, r),
                                                              x.device)
    nvfp4_w4a16_lora_gemm(x, q.codes, q.scales, q.tensor_scale, lora_a, lora_b, lora_scale, noise,
                          y, ws)
    return y


# ------------------------------------------------------------------ 4-bit activations
# One decode call is a few microseconds on the device, so these wrappers keep
# the host side short: sizes are computed here, pointers go over as integers.
_DTYPE_CODE = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}
_U8, _F32 = torch.uint8, torch.float32


def _out_code(dtype, name):
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code


def _raw_stream():
    return _raw(_current())


def _call(name, *args):
    st = getattr(_lib or load(), name)(*args)
    if st != OK:
        raise NVFP4Error(st, name)


def _matrix(t, name, dev):
    """Checks a 2-D matrix on the current device, dev, whose rows are contiguous; returns (rows, cols, row stride in
    elements, type code)."""
    if t.get_device() != dev:
        _device_of(t, name)
    code = _DTYPE_CODE.get(t.dtype)
    shape = t.shape
    if code is None or len(shape) != 2:
        _out_code(t.dtype, name)
        raise ValueError(f"{name} must have 2 dimensions, got {len(shape)}")
    rows, cols = shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return rows, cols, ld if rows > 1 else cols, code


def _addr(t):
    return None if t is None else t.data_ptr()


def _bad_scratch(workspace):
    _device_of(workspace, "workspace")
    raise ValueError("workspace must be a contiguous torch.uint8 tensor")


def _operand_elsewhere(index, dev):
    raise ValueError(f"operands must be on the current device, cuda:{dev}, got cuda:{index}")


def nvfp4_tiled_scale_bytes(rows: int, cols: int, fmt: int) -> int:
    return int(load().nvfp4_tiled_scale_bytes(rows, cols, int(fmt)))


class _Fp4Operand:
    """A 4-bit operand: codes (rows, cols/2) uint8 with the blocks along cols, and tiled scales (1-D uint8)."""

    format, block = None, None

    def __init__(self, codes, scales, tensor_scale=None):
        if not (codes.is_cuda and scales.is_cuda):
            raise ValueError("codes and scales must be CUDA tensors")
        if scales.get_device() != codes.get_device():
            raise ValueError("codes and scales must be on one device")
        if codes.dtype != _U8 or scales.dtype != _U8:
            raise ValueError("codes and scales must be torch.uint8")
        if codes.dim() != 2 or not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes must be a contiguous matrix and scales contiguous")
        rows, half = codes.shape
        cols = 2 * half
        # tiles of 128 rows x 4 blocks, 512 bytes each
        tiles = (rows + 127) // 128 * ((cols // self.block + 3) // 4)
        if cols % self.block or tiles == 0 or scales.dim() != 1 or scales.numel() != 512 * tiles:
            raise ValueError(f"scales must hold {512 * tiles} bytes in one dimension, and codes whole blocks of "
                             f"{self.block}")
        if tensor_scale is not None:
            _need(tensor_scale, _F32, (1,), "tensor_scale")
            if tensor_scale.get_device() != codes.get_device():
                raise ValueError("codes and tensor_scale must be on one device")
        self.codes, self.scales, self.tensor_scale = codes, scales, tensor_scale
        self.rows, self.cols, self.index = rows, cols, codes.get_device()

    @property
    def shape(self):
        return self.rows, self.cols

    @property
    def device(self):
        return self.codes.device

    def addresses(self):
        """Of the codes and of the scales."""
        return self.codes.data_ptr(), self.scales.data_ptr()

    @classmethod
    def from_row_major(cls, codes, scales, *tensor_scale):
        """From row-major scales (rows, cols/block), as a checkpoint or nvfp4_quantize has them."""
        rows, cols = codes.shape[0], codes.shape[1] * 2
        _need(codes, _U8, (rows, cols // 2), "codes")
        _need(scales, _U8, (rows, cols // cls.block), "scales")
        tiled = torch.empty(nvfp4_tiled_scale_bytes(rows, cols, cls.format), dtype=_U8, device=codes.device)
        _call("nvfp4_tile_scales", _addr(scales), rows, cols, cls.format, _addr(tiled), _raw_stream())
        return cls(codes, tiled, *tensor_scale)


class MxOperand(_Fp4Operand):
    """MXFP4: blocks of 32, E8M0 scales."""

    format, block = FORMAT_MXFP4, 32

    def __init__(self, codes, scales):
        super().__init__(codes, scales)

    def dequantize(self, dtype=torch.float32):
        if self.index != _current():
            _operand_elsewhere(self.index, _current())
        out = torch.empty(self.shape, dtype=dtype, device=self.device)
        _call("nvfp4_mx_dequantize", *self.addresses(), self.rows, self.cols, _addr(out), _out_code(dtype, "dtype"),
              _raw_stream())
        return out


class _MxMade(MxOperand):
    """An operand for mx_quantize to fill: one buffer with the codes first, then the scales, 16-byte aligned; the
    tensors are made when they are asked for."""

    tensor_scale = None

    def __init__(self, rows, cols, device, index):
        self.rows, self.cols, self.index = rows, cols, index
        self._at = (rows * cols // 2 + 15) & ~15
        self._nscales = (rows + 127) // 128 * ((cols + 127) // 128) * 512
        self._buffer = torch.empty(self._at + self._nscales, dtype=_U8, device=device)

    def addresses(self):
        base = self._buffer.data_ptr()
        return base, base + self._at

    @property
    def device(self):
        return self._buffer.device

    @property
    def codes(self):
        return self._buffer.as_strided((self.rows, self.cols // 2), (self.cols // 2, 1))

    @property
    def scales(self):
        return self._buffer.as_strided((self._nscales,), (1,), self._at)


class Nvfp4Operand(_Fp4Operand):
    """NVFP4: blocks of 16, E4M3 scales, a tensor scale."""

    format, block = FORMAT_NVFP4, 16

    @classmethod
    def from_weight(cls, q: QuantizedWeight):
        """The library's NVFP4 weight (or an activation quantised the same way) as an operand; shares its codes."""
        return cls.from_row_major(q.codes, q.scales, q.tensor_scale)


class MxQuantized:
    """What mx_quantize returns: .row and .col are MxOperands (blocks along the columns, along the rows and
    transposed), .values and .values_t bf16 matrices of x's shape; each None when it was not asked for."""

    __slots__ = ("row", "col", "values", "values_t")

    def __init__(self, row, col, values, values_t):
        self.row, self.col, self.values, self.values_t = row, col, values, values_t


def mx_quantize(x: torch.Tensor, rowwise=True, colwise=False, codes=True, values=False) -> MxQuantized:
    """MXFP4 quantisation of x (rows, cols), bf16 or float32, along its columns (rowwise) and/or its rows (colwise).
    codes: return operands for products; values: return x as the codes stand for it (bf16), e.g. for a
    straight-through forward."""
    index = _current()
    rows, cols, ld, dt = _matrix(x, "x", index)
    dev = x.device
    rows32 = (rows + 31) // 32 * 32
    row = col = v = vt = q = qs = qt = qts = None
    if codes:
        # a buffer each: what is kept for a backward pass does not hold the other direction
        if rowwise:
            row = _MxMade(rows, cols, dev, index)
            q, qs = row.addresses()
        if colwise:
            col = _MxMade(cols, rows32, dev, index)
            qt, qts = col.addresses()
    if values:
        if rowwise:
            v = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
        if colwise:
            vt = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    _call("nvfp4_mx_quantize", x.data_ptr(), dt, rows, cols, ld, q, qs, _addr(v), qt, qts, _addr(vt), _raw(index))
    return MxQuantized(row, col, v, vt)


def nvfp4_w4a4_workspace_bytes(M: int, N: int, K: int) -> int:
    return (_lib or load()).nvfp4_w4a4_workspace_bytes(M, N, K)


def nvfp4_mx_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return (_lib or load()).nvfp4_mx_linear_workspace_bytes(M, N, K)


def nvfp4_mx_linear_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    return (_lib or load()).nvfp4_mx_linear_backward_workspace_bytes(M, N, K)


def w4a4_gemm(a, w, out_dtype=torch.float32, workspace=None) -> torch.Tensor:
    """Y (M, N) = A W^T of two operands of one format (MxOperand or Nvfp4Operand)."""
    if a.format != w.format:
        raise ValueError("a and w must have the same format")
    M, N, K = a.rows, w.rows, a.cols
    if K != w.cols:
        raise ValueError(f"a and w must have the same number of columns, got {K} and {w.cols}")
    ydt = _DTYPE_CODE.get(out_dtype)
    if ydt is None:
        _out_code(out_dtype, "out_dtype")
    dev = _current()
    if a.index != dev or w.index != dev:
        _operand_elsewhere(a.index if a.index != dev else w.index, dev)
    ws = workspace
    if ws is None:
        ws = new_workspace(nvfp4_w4a4_workspace_bytes(M, N, K), a.device)
    elif ws.get_device() != dev or ws.dtype is not _U8 or not ws.is_contiguous():
        _bad_scratch(ws)
    y = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _call("nvfp4_w4a4_gemm", a.format, *a.addresses(), _addr(a.tensor_scale), *w.addresses(), _addr(w.tensor_scale),
          M, N, K, y.data_ptr(), ydt, ws.data_ptr(), ws.numel(), _raw(dev))
    return y


def mx_linear(x: torch.Tensor, w: MxOperand, out_dtype=torch.float32, workspace=None) -> torch.Tensor:
    """Y (M, N) = Q(X) W^T: x (M, K) bf16 or float32, quantised to MXFP4 on the way."""
    dev = _current()
    M, K, ld, dt = _matrix(x, "x", dev)
    ydt = _DTYPE_CODE.get(out_dtype)
    if ydt is None:
        _out_code(out_dtype, "out_dtype")
    if not isinstance(w, MxOperand) or K != w.cols:
        raise ValueError("w must be an MxOperand with x's number of columns")
    if w.index != dev:
        _operand_elsewhere(w.index, dev)
    N = w.rows
    ws = workspace
    if ws is None:
        ws = new_workspace(nvfp4_mx_linear_workspace_bytes(M, N, K), x.device)
    elif ws.get_device() != dev or ws.dtype is not _U8 or not ws.is_contiguous():
        _bad_scratch(ws)
    y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _call("nvfp4_mx_linear", x.data_ptr(), dt, ld, M, N, K, *w.addresses(), y.data_ptr(), ydt,
          ws.data_ptr(), ws.numel(), _raw(dev))
    return y


def mx_linear_backward(dy: torch.Tensor, x_col, w_col, dx_dtype=torch.float32, dw_dtype=torch.float32,
                       workspace=None):
    """(dX (M, K), dW (N, K)) of Y = X W^T with straight-through MXFP4 quantisers.  dy (M, N) bf16 or float32;
    x_col, w_col: mx_quantize(..., colwise=True).col of X and W.  w_col None: no dX; x_col None: no dW."""
    dev = _current()
    M, N, ld, dt = _matrix(dy, "dy", dev)
    xdt, wdt = _out_code(dx_dtype, "dx_dtype"), _out_code(dw_dtype, "dw_dtype")
    if x_col is None and w_col is None:
        raise ValueError("one of x_col and w_col is needed")
    K = (x_col if x_col is not None else w_col).rows
    M32 = (M + 31) // 32 * 32
    if x_col is not None and (not isinstance(x_col, MxOperand) or x_col.shape != (K, M32)):
        raise ValueError(f"x_col must be an MxOperand of shape {(K, M32)}")
    if w_col is not None and (not isinstance(w_col, MxOperand) or w_col.shape != (K, N)):
        raise ValueError(f"w_col must be an MxOperand of shape {(K, N)}")
    for operand in (x_col, w_col):
        if operand is not None and operand.index != dev:
            _operand_elsewhere(operand.index, dev)
    xp = (None, None) if x_col is None else x_col.addresses()
    wp = (None, None) if w_col is None else w_col.addresses()
    ws = workspace
    if ws is None:
        ws = new_workspace(nvfp4_mx_linear_backward_workspace_bytes(M, N, K), dy.device)
    elif ws.get_device() != dev or ws.dtype is not _U8 or not ws.is_contiguous():
        _bad_scratch(ws)
    dx = torch.empty((M, K), dtype=dx_dtype, device=dy.device) if w_col is not None else None
    dw = torch.empty((N, K), dtype=dw_dtype, device=dy.device) if x_col is not None else None
    _call("nvfp4_mx_linear_backward", dy.data_ptr(), dt, ld, M, N, K, *xp, *wp, _addr(dx), xdt, _addr(dw), wdt,
          ws.data_ptr(), ws.numel(), _raw(dev))
    return dx, dw


# ------------------------------------------------------------------ distillation
_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}


def nvfp4_distill_topk(z, index, teacher, temperature, tail, row_weight, grad_loss, loss, dz, workspace):
    """The C entry point on tensors; loss or dz may be None (see include/nvfp4.h)."""
    dev = _current()
    T, V, ldz, zdt = _matrix(z, "z", dev)
    tdt = _out_code(teacher.dtype, "teacher")
    ib = _INDEX_BYTES.get(index.dtype)
    shape = index.shape
    if ib is None or len(shape) != 2:
        raise ValueError("index must be a 2-dimensional int32 or int64 tensor")
    k = shape[1]
    if index.get_device() != dev or teacher.get_device() != dev:
        _device_of(index, "index")
        _device_of(teacher, "teacher")
    if shape[0] != T or teacher.shape != shape or not (index.is_contiguous() and teacher.is_contiguous()):
        raise ValueError(f"index and teacher must be contiguous CUDA tensors of one shape ({T}, k), got "
                         f"{tuple(shape)} and {tuple(teacher.shape)}")
    if row_weight is not None:
        _need(row_weight, _F32, (T,), "row_weight", dev)
    ng = 0
    if grad_loss is not None:
        ng = grad_loss.numel()
        _need(grad_loss, _F32, (T,) if ng != 1 else grad_loss.shape, "grad_loss", dev)
    if loss is not None:
        _need(loss, _F32, (T,), "loss", dev)
    lddz = V
    if dz is not None:
        rows, cols, lddz, ddt = _matrix(dz, "dz", dev)
        if ddt != zdt or rows != T or cols != V:
            raise ValueError("dz must have z's type and shape")
    if workspace is not None and not (workspace.get_device() == dev and workspace.dtype is _U8 and
                                      workspace.is_contiguous()):
        _bad_scratch(workspace)
    _call("nvfp4_distill_topk", z.data_ptr(), zdt, T, V, ldz, index.data_ptr(), ib, teacher.data_ptr(), tdt, k,
          temperature, 1 if tail else 0, _addr(row_weight), _addr(grad_loss), ng, _addr(loss), _addr(dz), lddz,
          _addr(workspace), 0 if workspace is None else workspace.numel(), _raw(dev))


def distill_topk_loss(z, index, teacher, temperature=1.0, tail=False, row_weight=None, workspace=None):
    """Loss per row (T,) float32 of student logits z (T, V) against the teacher's top entries (T, k): index (int32 or
    int64, negative: unused slot) and teacher (logits, or log-probabilities with tail=True, where the teacher's
    remaining mass is one more class)."""
    loss = torch.empty(z.shape[0], dtype=torch.float32, device=z.device)
    nvfp4_distill_topk(z, index, teacher, temperature, tail, row_weight, None, loss, None, workspace)
    return loss


def distill_topk_loss_grad(z, index, teacher, temperature=1.0, tail=False, row_weight=None, grad_loss=None,
                           out=None, workspace=None):
    """(loss (T,), dz (T, V)) in one pass over z; dz = grad_loss (T values, one, or None for 1) times d loss / d z.
    out: where dz goes (z itself for an update in place)."""
    loss = torch.empty(z.shape[0], dtype=torch.float32, device=z.device)
    dz = out if out is not None else torch.empty_like(z, memory_format=torch.contiguous_format)
    nvfp4_distill_topk(z, index, teacher, temperature, tail, row_weight, grad_loss, loss, dz, workspace)
    return loss, dz


def distill_topk_grad(z, index, teacher, grad_loss=None, temperature=1.0, tail=False, row_weight=None, out=None,
                      workspace=None):
    """dz alone, for a backward pass whose incoming gradient was not known with the loss."""
    dz = out if out is not None else torch.empty_like(z, memory_format=torch.contiguous_format)
    nvfp4_distill_topk(z, index, teacher, temperature, tail, row_weight, grad_loss, None, dz, workspace)
    return dz


def nvfp4_distill_wait_selftest(z, index, teacher, tail=False, row_weight=None, loss=None, dz=None, workspace=None):
    """The distillation kernels with waits that give up at once (see include/nvfp4.h): z (T, V) contiguous."""
    dev = _current()
    T, V, ldz, zdt = _matrix(z, "z", dev)
    k = index.shape[1]
    _need(z, z.dtype, (T, V), "z")
    _need(index, torch.int32, (T, k), "index")
    _need(teacher, _F32, (T, k), "teacher")
    if row_weight is not None:
        _need(row_weight, _F32, (T,), "row_weight")
    if loss is not None:
        _need(loss, _F32, (T,), "loss")
    if dz is not None:
        _need(dz, z.dtype, (T, V), "dz")
    if workspace is not None and not (workspace.get_device() == dev and workspace.dtype is _U8 and
                                      workspace.is_contiguous()):
        _bad_scratch(workspace)
    _call("nvfp4_distill_wait_selftest", z.data_ptr(), zdt, T, V, index.data_ptr(), teacher.data_ptr(), k,
          1 if tail else 0, _addr(row_weight), _addr(loss), _addr(dz), _addr(workspace),
          0 if workspace is None else workspace.numel(), _raw(dev))
