"""Python binding of libptq.so, the GB300 (sm_103a) PTQ1_0 ternary matmul
library (C ABI in include/ptq.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or a call fails,
these functions raise.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from . import _build

LIB_PATH = _build.LIB

PTQ_F32 = 0
PTQ_BF16 = 1

STATUS = {
    0: "PTQ_OK", 1: "PTQ_ERR_NULL", 2: "PTQ_ERR_SHAPE", 3: "PTQ_ERR_ALIGN", 4: "PTQ_ERR_VALUE",
    5: "PTQ_ERR_UNSUPPORTED", 6: "PTQ_ERR_WORKSPACE", 7: "PTQ_ERR_CUDA", 8: "PTQ_ERR_TIMEOUT",
    9: "PTQ_ERR_RANGE",
}

# Every symbol include/ptq.h declares.
EXPORTS = ("ptq1_pack", "ptq1_unpack", "ptq_fwht", "ptq_matmul_workspace_bytes", "ptq_matmul",
           "ptq_rotate_matmul_workspace_bytes", "ptq_rotate_matmul",
           "ptq_rotate_matmul_host_workspace_bytes", "ptq_rotate_matmul_host", "ptq_ffn_workspace_bytes",
           "ptq_ffn", "ptq_ffn_noalloc", "ptq_ffn_stack_workspace_bytes", "ptq_ffn_stack",
           "ptq_ffn_stack_ex", "ptq_ffn_stack_route", "ptq2_pack", "ptq2_unpack",
           "ptq_matmul_pq2_workspace_bytes", "ptq_matmul_pq2", "ptq_embed", "ptq_embed_ptq1",
           "ptq_kv_write", "ptq_kv_read", "ptq_attn_decode_workspace_bytes", "ptq_attn_decode",
           "ptq_attn_prefill_workspace_bytes", "ptq_attn_prefill",
           "ptq_route", "ptq_gemv_plan", "ptq_matmul_bf16_accumulator", "ptq_matmul_f32_peel",
           "ptq_selftest_timeout",
           "ptq_selftest_grid_timeout",
           "ptq_device_check", "ptq_status_str", "ptq_last_error")

# Size of the built-in scratch array behind ptq_ffn_noalloc (include/ptq.h).
FFN_NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


class PTQError(RuntimeError):
    def __init__(self, status: int, call: str, message: str):
        self.status = status
        self.name = STATUS.get(status, f"status {status}")
        super().__init__(f"{call}: {self.name}: {message}")


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int


def load(path: str | None = None):
    """Load libptq.so (building it first if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        _build.build()
    L = ctypes.CDLL(path)
    L.ptq1_pack.argtypes = [_P, _P, _I64, _I64]
    L.ptq1_unpack.argtypes = [_P, _P, _I64, _I64, _P]
    L.ptq_fwht.argtypes = [_P, _P, _P, _I64, _I64, _I32, _P]
    L.ptq_matmul_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    L.ptq_matmul_workspace_bytes.restype = ctypes.c_size_t
    L.ptq_matmul.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_size_t, _P]
    L.ptq_rotate_matmul_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    L.ptq_rotate_matmul_workspace_bytes.restype = ctypes.c_size_t
    L.ptq_rotate_matmul_host_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    L.ptq_rotate_matmul_host_workspace_bytes.restype = ctypes.c_size_t
    L.ptq_rotate_matmul_host.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P,
                                         ctypes.c_size_t, _P]
    L.ptq_rotate_matmul_host.restype = _I32
    L.ptq_rotate_matmul.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_size_t,
                                    _P]
    L.ptq_ffn_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    L.ptq_ffn_workspace_bytes.restype = ctypes.c_size_t
    L.ptq_ffn.argtypes = [_P] * 8 + [_I64, _I64, _I64, _I32, _P, ctypes.c_size_t, _P]
    L.ptq_ffn_noalloc.argtypes = [_P] * 8 + [_I64, _I64, _I64, _I32, _P]
    L.ptq_ffn_stack_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    L.ptq_ffn_stack_workspace_bytes.restype = ctypes.c_size_t
    L.ptq_ffn_stack.argtypes = [_P, _I64, _P, _I64, _I64, _I64, ctypes.c_float, _I32, _P,
                                ctypes.c_size_t, _P]
    L.ptq_ffn_stack_ex.argtypes = [_P, _I64, _P, _I64, _I64, _I64, ctypes.c_float, _I32, _P,
                                   ctypes.c_size_t, ctypes.c_uint, _P]
    L.ptq_ffn_stack_route.argtypes = [_I64, _I64, _I64, _I32, ctypes.POINTER(ctypes.c_char_p)]
    L.ptq2_pack.argtypes = [_P, _P, _I64, _I64]
    L.ptq2_unpack.argtypes = [_P, _P, _I64, _I64, _P]
    L.ptq_matmul_pq2_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    L.ptq_matmul_pq2_workspace_bytes.restype = ctypes.c_size_t
    L.ptq_matmul_pq2.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, ctypes.c_size_t, _P]
    L.ptq_embed.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P]
    L.ptq_embed_ptq1.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P]
    S = ctypes.c_size_t
    L.ptq_kv_write.argtypes = [_P, _P, _P, _I64, _I64, _P, _I64, _I32, _P]
    L.ptq_kv_read.argtypes = [_P, _P, _I64, _P, _P, _I64, _I64, _I32, _P]
    L.ptq_attn_decode_workspace_bytes.argtypes = [_I64] * 4 + [_I32]
    L.ptq_attn_decode_workspace_bytes.restype = S
    L.ptq_attn_decode.argtypes = ([_P, _I64, _P, _P, _I64, _P, _P, _P, _I64, _I64, ctypes.c_float,
                                   _I32, _P, S, _P])
    L.ptq_attn_prefill_workspace_bytes.argtypes = [_I64] * 6 + [_I32]
    L.ptq_attn_prefill_workspace_bytes.restype = S
    L.ptq_attn_prefill.argtypes = ([_P] * 3 + [_I64] * 3 + [_P] * 4 + [_I64] * 6 +
                                   [ctypes.c_float, ctypes.c_uint, _I32, _P, S, _P])
    for name in ("ptq_kv_write", "ptq_kv_read", "ptq_attn_decode", "ptq_attn_prefill"):
        getattr(L, name).restype = _I32
    L.ptq_route.argtypes = [_I64, _I32, ctypes.POINTER(ctypes.c_char_p)]
    L.ptq_gemv_plan.argtypes = [_I64, _I64, _I64, _I32, ctypes.POINTER(ctypes.c_int32)]
    L.ptq_matmul_f32_peel.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P]
    L.ptq_matmul_f32_peel.restype = _I32
    L.ptq_matmul_bf16_accumulator.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, _P,
                                              ctypes.c_size_t, _P]
    L.ptq_device_check.argtypes = [_P]
    L.ptq_selftest_timeout.argtypes = [_P]
    L.ptq_selftest_grid_timeout.argtypes = [_P]
    L.ptq_status_str.argtypes = [_I32]
    L.ptq_status_str.restype = ctypes.c_char_p
    L.ptq_last_error.argtypes = []
    L.ptq_last_error.restype = ctypes.c_char_p
    for name in ("ptq1_pack", "ptq1_unpack", "ptq_fwht", "ptq_matmul", "ptq_rotate_matmul", "ptq_ffn",
                 "ptq_ffn_noalloc", "ptq_ffn_stack", "ptq_ffn_stack_ex", "ptq_ffn_stack_route", "ptq2_pack",
                 "ptq2_unpack", "ptq_matmul_pq2", "ptq_embed",
                 "ptq_embed_ptq1", "ptq_route", "ptq_gemv_plan", "ptq_device_check",
                 "ptq_selftest_timeout", "ptq_selftest_grid_timeout"):
        getattr(L, name).restype = _I32
    _lib = L
    return L


def _check(status: int, call: str) -> None:
    if status != 0:
        msg = load().ptq_last_error().decode(errors="replace")
        raise PTQError(status, call, msg)


def _stream(stream=None, device=None) -> int:
    """The raw handle of `stream`, else of PyTorch's current stream on
    `device` (an index; the current device when None)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if device is None or _raw_stream is None:
        import torch

        _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or  # no Stream object per call
                       (lambda d: torch.cuda.current_stream(d).cuda_stream))
        if device is None:
            device = torch.cuda.current_device()
    return _raw_stream(device)


_raw_stream = None


def _new(like, shape, dtype, stream, returned=True):
    """An uninitialised tensor beside `like` for a call queued on `stream`.  It
    is allocated on that stream, whose work alone then gets its memory before
    the call has run or after the tensor is dropped; one that is returned is
    marked as used on the current stream too."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch

    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, like.device)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if returned:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _nowhere():
    return -1


def _misplaced(t, name, on):
    """Refuses a tensor that is not on the CUDA device of index `on`."""
    d = getattr(t, "get_device", _nowhere)()
    if d < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on another device: cuda:{d}, not cuda:{on}")


def _dev(t, dtype=None, name="tensor", on=None):
    if on is None:
        if not getattr(t, "is_cuda", False):
            raise TypeError(f"{name} must be a CUDA tensor")
    elif getattr(t, "get_device", _nowhere)() != on:
        _misplaced(t, name, on)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _act_dtype(t):
    if not _act_dtypes:
        import torch

        _act_dtypes.update({torch.float32: PTQ_F32, torch.bfloat16: PTQ_BF16})
    dt = _act_dtypes.get(t.dtype)
    if dt is None:
        raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")
    return dt


_act_dtypes = {}


# ---- host encoder ------------------------------------------------------------

def pack(trits: np.ndarray) -> np.ndarray:
    """ptq1_pack: N x K int8 trits -> N x (K/128*26) uint8 (host)."""
    trits = np.ascontiguousarray(trits, dtype=np.int8)
    if trits.ndim != 2:
        raise ValueError("trits must be 2-D")
    N, K = trits.shape
    out = np.empty((N, (K // 128) * 26 if K % 128 == 0 else 0), np.uint8)
    _check(load().ptq1_pack(ctypes.c_void_p(trits.ctypes.data), ctypes.c_void_p(out.ctypes.data),
                            N, K), "ptq1_pack")
    return out


# ---- device calls --------------------------------------------------------------

def unpack(wq, K: int, stream=None):
    import torch

    N = wq.shape[0]
    out = _new(wq, (N, K), torch.int8, stream)
    _check(load().ptq1_unpack(_dev(wq, torch.uint8, "wq"), _dev(out), N, K, _stream(stream)),
           "ptq1_unpack")
    return out


def fwht(x, signs, out=None, stream=None):
    """Signed 1024-wide rotation of the rows of x (in place when out is x)."""
    import torch

    y = _new(x, x.shape, x.dtype, stream) if out is None else out
    M, K = x.shape
    _check(load().ptq_fwht(_dev(x, None, "x"), _dev(y, x.dtype, "out"), _dev(signs, torch.int8, "signs"),
                           M, K, _act_dtype(x), _stream(stream)), "ptq_fwht")
    return y


def matmul_workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    return int(load().ptq_matmul_workspace_bytes(M, N, K, dtype))


def matmul(wq, scales, x, out=None, workspace=None, stream=None):
    """y = x W^T, W the PTQ1_0 weight (N x K); x M x K (float32 or bfloat16).
    The scratch the call needs (ptq_matmul_workspace_bytes) is allocated by
    PyTorch here when `workspace` is not given."""
    import torch

    M, K = x.shape
    N = wq.shape[0]
    dt = _act_dtype(x)
    y = _new(x, (M, N), x.dtype, stream) if out is None else out
    need = matmul_workspace_bytes(M, N, K, dt)
    if workspace is None and need > 0:
        workspace = _new(x, need, torch.uint8, stream, returned=False)
    ws = _dev(workspace, None, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().ptq_matmul(_dev(wq, torch.uint8, "wq"), _dev(scales, torch.int16, "scales"),
                             _dev(x, None, "x"), _dev(y, x.dtype, "out"), M, N, K, dt, ws,
                             ws_bytes, _stream(stream)), "ptq_matmul")
    return y


def matmul_bf16_accumulator(wq, scales, x, stream=None):
    """Test export: the bf16 prefill GEMM's fp32 accumulator (y = x W^T with
    x bfloat16, y float32), the same kernel as matmul() on bfloat16 input
    without the output's bf16 rounding."""
    import torch

    M, K = x.shape
    N = wq.shape[0]
    y = _new(x, (M, N), torch.float32, stream)
    need = matmul_workspace_bytes(M, N, K, PTQ_BF16)
    ws = _new(x, need, torch.uint8, stream, returned=False) if need > 0 else None
    _check(load().ptq_matmul_bf16_accumulator(
        _dev(wq, torch.uint8, "wq"), _dev(scales, torch.int16, "scales"),
        _dev(x, torch.bfloat16, "x"), _dev(y, torch.float32, "out"), M, N, K,
        _dev(ws, None, "workspace") if ws is not None else None, need, _stream(stream)),
        "ptq_matmul_bf16_accumulator")
    return y


def pq2_pack(trits: np.ndarray) -> np.ndarray:
    """ptq2_pack: N x K int8 trits -> N x (K/128*32) uint8 PQ2_0 codes (host)."""
    trits = np.ascontiguousarray(trits, dtype=np.int8)
    if trits.ndim != 2:
        raise ValueError("trits must be 2-D")
    N, K = trits.shape
    out = np.empty((N, K // 4 if K % 128 == 0 else 0), np.uint8)
    _check(load().ptq2_pack(ctypes.c_void_p(trits.ctypes.data), ctypes.c_void_p(out.ctypes.data),
                            N, K), "ptq2_pack")
    return out


def pq2_unpack(wq, K: int, stream=None):
    import torch

    N = wq.shape[0]
    out = _new(wq, (N, K), torch.int8, stream)
    _check(load().ptq2_unpack(_dev(wq, torch.uint8, "wq"), _dev(out), N, K, _stream(stream)),
           "ptq2_unpack")
    return out


def matmul_pq2_workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    return int(load().ptq_matmul_pq2_workspace_bytes(M, N, K, dtype))


def matmul_pq2(wq, scales, x, out=None, workspace=None, stream=None):
    """y = x W^T over PQ2_0 weights (ptq_matmul_pq2); as matmul otherwise."""
    import torch

    M, K = x.shape
    N = wq.shape[0]
    dt = _act_dtype(x)
    y = _new(x, (M, N), x.dtype, stream) if out is None else out
    need = matmul_pq2_workspace_bytes(M, N, K, dt)
    if workspace is None and need > 0:
        workspace = _new(x, need, torch.uint8, stream, returned=False)
    ws = _dev(workspace, None, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().ptq_matmul_pq2(_dev(wq, torch.uint8, "wq"), _dev(scales, torch.int16, "scales"),
                                 _dev(x, None, "x"), _dev(y, x.dtype, "out"), M, N, K, dt, ws,
                                 ws_bytes, _stream(stream)), "ptq_matmul_pq2")
    return y


def rotate_matmul_workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    return int(load().ptq_rotate_matmul_workspace_bytes(M, N, K, dtype))


def rotate_matmul_host_workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    return int(load().ptq_rotate_matmul_host_workspace_bytes(M, N, K, dtype))


def rotate_matmul_host(wq, scales, x_host, signs, y_host, workspace, stream=None):
    """ptq_rotate_matmul_host: x_host (M x K) and y_host (M x N) are CPU
    tensors (page-locked for asynchronous copies) of one dtype, float32 or
    bfloat16; the copies and the product are queued on the stream, and
    y_host is valid once it is synchronised."""
    import torch

    M, K = x_host.shape
    N = wq.shape[0]
    dt = _act_dtype(x_host)
    for t, name in ((x_host, "x_host"), (y_host, "y_host")):
        if t.is_cuda or not t.is_contiguous() or t.dtype != x_host.dtype:
            raise TypeError(f"{name} must be a contiguous CPU tensor of the activations' dtype")
    if tuple(y_host.shape) != (M, N):
        raise ValueError(f"y_host must be {M} x {N}")
    _check(load().ptq_rotate_matmul_host(
        _dev(wq, torch.uint8, "wq"), _dev(scales, torch.int16, "scales"), x_host.data_ptr(),
        _dev(signs, torch.int8, "signs"), y_host.data_ptr(), M, N, K, dt,
        _dev(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream, wq.device.index)), "ptq_rotate_matmul_host")
    return y_host


def rotate_matmul(wq, scales, x, signs, out=None, workspace=None, stream=None):
    """y = (R x) W^T: the signed rotation of `x` (not modified), then the
    PTQ1_0 matmul; fused into one kernel on the fp32 M = 1 route.  The
    scratch is allocated by PyTorch here when `workspace` is not given."""
    import torch

    M, K = x.shape
    N = wq.shape[0]
    dt = _act_dtype(x)
    y = _new(x, (M, N), x.dtype, stream) if out is None else out
    if workspace is None:
        workspace = _new(x, max(1, rotate_matmul_workspace_bytes(M, N, K, dt)), torch.uint8, stream,
                         returned=False)
    _check(load().ptq_rotate_matmul(_dev(wq, torch.uint8, "wq"),
                                    _dev(scales, torch.int16, "scales"), _dev(x, None, "x"),
                                    _dev(signs, torch.int8, "signs"), _dev(y, x.dtype, "out"), M, N,
                                    K, dt, _dev(workspace, None, "workspace"),
                                    workspace.numel() * workspace.element_size(), _stream(stream)),
           "ptq_rotate_matmul")
    return y


def ffn_workspace_bytes(M: int, H: int, I: int, dtype: int) -> int:
    return int(load().ptq_ffn_workspace_bytes(M, H, I, dtype))


def ffn(wgu_q, wgu_s, wd_q, wd_s, signs_in, signs_mid, x, out=None, workspace=None, stream=None):
    """The feed-forward block: rotate, gate+up, SwiGLU, rotate, down."""
    import torch

    M, H = x.shape
    I = signs_mid.shape[0]
    dt = _act_dtype(x)
    need = ffn_workspace_bytes(M, H, I, dt)
    if workspace is None:
        workspace = _new(x, max(need, 1), torch.uint8, stream, returned=False)
    y = _new(x, x.shape, x.dtype, stream) if out is None else out
    _check(load().ptq_ffn(_dev(wgu_q, torch.uint8, "wgu_q"), _dev(wgu_s, torch.int16, "wgu_s"),
                          _dev(wd_q, torch.uint8, "wd_q"), _dev(wd_s, torch.int16, "wd_s"),
                          _dev(signs_in, torch.int8, "signs_in"),
                          _dev(signs_mid, torch.int8, "signs_mid"), _dev(x, None, "x"),
                          _dev(y, x.dtype, "out"), M, H, I, dt, _dev(workspace, None, "workspace"),
                          workspace.numel() * workspace.element_size(), _stream(stream)),
           "ptq_ffn")
    return y


class FfnLayer(ctypes.Structure):
    """One layer of ptq_ffn_stack (include/ptq.h): device addresses."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("wgu_q", "wgu_s", "wd_q", "wd_s", "signs_in", "signs_mid", "norm_w")]


def ffn_stack_workspace_bytes(M: int, H: int, I: int, dtype: int) -> int:
    return int(load().ptq_ffn_stack_workspace_bytes(M, H, I, dtype))


def ffn_stack_route(M: int, H: int, I: int, dtype: int) -> str:
    """The implementation ptq_ffn_stack uses for (M, H, I, dtype) here."""
    name = ctypes.c_char_p()
    _check(load().ptq_ffn_stack_route(M, H, I, dtype, ctypes.byref(name)), "ptq_ffn_stack_route")
    return name.value.decode()


PTQ_STACK_DETERMINISTIC = 1


def ffn_stack(layers, norm_w, x, eps: float, act=None, workspace=None, stream=None,
              deterministic: bool = False):
    """L chained pre-norm feed-forward blocks over the fp32 residual stream x
    (M x H, updated in place and returned): x += ffn_l(rmsnorm(x) * g_l).
    `layers`: per layer (wgu_q, wgu_s, wd_q, wd_s, signs_in, signs_mid) as for
    ffn(); `norm_w`: per layer an H-vector of fp32 gains.  `act` is the
    blocks' activation dtype, torch.float32 (default) or torch.bfloat16.
    `deterministic` takes the bitwise-reproducible per-layer path."""
    import torch

    if len(layers) != len(norm_w):
        raise ValueError("layers and norm_w differ in length")
    M, H = x.shape
    L = len(layers)
    I = layers[0][5].shape[0] if L else 1024
    dt = _act_dtype(torch.empty(0, dtype=act or torch.float32))
    need = ffn_stack_workspace_bytes(M, H, I, dt)
    if workspace is None:
        workspace = _new(x, max(need, 1), torch.uint8, stream, returned=False)
    arr = (FfnLayer * max(L, 1))()
    names = ("wgu_q", "wgu_s", "wd_q", "wd_s", "signs_in", "signs_mid")
    types = (torch.uint8, torch.int16, torch.uint8, torch.int16, torch.int8, torch.int8)
    for l, (lay, g) in enumerate(zip(layers, norm_w)):
        ptrs = [_dev(t, ty, f"layers[{l}].{n}") for t, ty, n in zip(lay, types, names)]
        ptrs.append(_dev(g, torch.float32, f"norm_w[{l}]"))
        arr[l] = FfnLayer(*ptrs)
    _check(load().ptq_ffn_stack_ex(ctypes.cast(arr, ctypes.c_void_p), L,
                                   _dev(x, torch.float32, "x"), M, H, I, float(eps), dt,
                                   _dev(workspace, None, "workspace"),
                                   workspace.numel() * workspace.element_size(),
                                   PTQ_STACK_DETERMINISTIC if deterministic else 0, _stream(stream)),
           "ptq_ffn_stack")
    return x


def ffn_noalloc(wgu_q, wgu_s, wd_q, wd_s, signs_in, signs_mid, x, out=None, stream=None):
    """The feed-forward block without a workspace: for callers that cannot
    allocate device memory (graph capture, real-time loops, memory owned by
    another allocator).  Its scratch is one built-in device array of
    FFN_NOALLOC_SCRATCH_BYTES shared by all calls, so calls that overlap on
    the GPU race; larger shapes raise PTQ_ERR_WORKSPACE.  Only `out` (if not
    given) is allocated here, by PyTorch, before the call."""
    import torch

    M, H = x.shape
    I = signs_mid.shape[0]
    y = _new(x, x.shape, x.dtype, stream) if out is None else out
    _check(load().ptq_ffn_noalloc(_dev(wgu_q, torch.uint8, "wgu_q"), _dev(wgu_s, torch.int16, "wgu_s"),
                                  _dev(wd_q, torch.uint8, "wd_q"), _dev(wd_s, torch.int16, "wd_s"),
                                  _dev(signs_in, torch.int8, "signs_in"),
                                  _dev(signs_mid, torch.int8, "signs_mid"), _dev(x, None, "x"),
                                  _dev(y, x.dtype, "out"), M, H, I, _act_dtype(x), _stream(stream)),
           "ptq_ffn_noalloc")
    return y


def embed(table, ids, signs, out=None, stream=None):
    """out[m] = R^T table[ids[m]]: the lookup on a rotated embedding table
    (ptq_embed).  table: V x H float32 or bfloat16; ids: M int32 token ids;
    ids outside [0, V) give rows of NaN."""
    import torch

    dt = _act_dtype(table)
    V, H = table.shape
    M = ids.numel()
    y = _new(table, (M, H), table.dtype, stream) if out is None else out
    _check(load().ptq_embed(_dev(table, None, "table"), _dev(ids, torch.int32, "ids"),
                            _dev(signs, torch.int8, "signs"), _dev(y, table.dtype, "out"), M, V, H,
                            dt, _stream(stream)), "ptq_embed")
    return y


def embed_ptq1(wq, scales, ids, signs, out_dtype=None, out=None, stream=None):
    """ptq_embed_ptq1: the same lookup on a PTQ1_0 table (wq V x H/128*26
    uint8, scales V x H/128 int16 bit patterns); out_dtype float32 (default)
    or bfloat16."""
    import torch

    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    dt = PTQ_F32 if out_dtype == torch.float32 else PTQ_BF16 if out_dtype == torch.bfloat16 else None
    if dt is None:
        raise TypeError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    V, H = scales.shape[0], scales.shape[1] * 128
    M = ids.numel()
    y = _new(wq, (M, H), out_dtype, stream) if out is None else out
    _check(load().ptq_embed_ptq1(_dev(wq, torch.uint8, "wq"), _dev(scales, None, "scales"),
                                 _dev(ids, torch.int32, "ids"), _dev(signs, torch.int8, "signs"),
                                 _dev(y, out_dtype, "out"), M, V, H, dt, _stream(stream)),
           "ptq_embed_ptq1")
    return y


# ---- attention over a paged key-value cache --------------------------------------

PTQ_KV_BF16 = 0
PTQ_KV_I8 = 1
PTQ_ATTN_CAUSAL = 1


class _KvCacheStruct(ctypes.Structure):
    """ptq_kv_cache (include/ptq.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] +
                [(n, ctypes.c_int64) for n in ("pages", "page_tokens", "kv_heads", "head_dim")] +
                [("type", ctypes.c_int)])


class KVCache:
    """A paged key-value cache over the caller's tensors: k and v are pages x
    kv_heads x page_tokens x head_dim, bfloat16, or int8 with k_scale and
    v_scale (pages x kv_heads x page_tokens float32).  Keeps the tensors alive;
    copies nothing, and hands their addresses to the library: none is replaced."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch

        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be pages x kv_heads x page_tokens x head_dim, of one type")
        on = k.get_device() if k.is_cuda else None
        if k.dtype == torch.int8:
            for s in (k_scale, v_scale):
                if s is None or s.shape != k.shape[:3]:
                    raise ValueError("an int8 cache needs k_scale and v_scale, one scale for each row")
            self.type = PTQ_KV_I8
            scales = (_dev(k_scale, torch.float32, "k_scale", on), _dev(v_scale, torch.float32, "v_scale", on))
        elif k.dtype == torch.bfloat16:
            if k_scale is not None or v_scale is not None:
                raise ValueError("a bfloat16 cache takes no scales")
            self.type = PTQ_KV_BF16
            scales = (None, None)
        else:
            raise TypeError(f"a cache is bfloat16 or int8, got {k.dtype}")
        self._on = on
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._int32, self._bfloat16 = torch.int32, torch.bfloat16
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = k.shape
        self._struct = _KvCacheStruct(_dev(k, None, "k", on), _dev(v, None, "v", on), *scales, self.pages,
                                      self.page_tokens, self.kv_heads, self.head_dim, self.type)
        self._ref = ctypes.addressof(self._struct)

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{name} of a KVCache is not replaced: make a new one")
        self.__dict__[name] = value

    @classmethod
    def empty(cls, pages, kv_heads, page_tokens, head_dim, dtype, device="cuda"):
        """A new cache of torch.bfloat16 or torch.int8 rows."""
        import torch

        shape = (pages, kv_heads, page_tokens, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.float32, device=device)
                           for _ in range(2)))


def _heads(t, name, dtype, on, shape=None):
    """The address and token stride of a tokens x heads x head_dim tensor whose
    heads are contiguous within a token (tokens may be any stride apart)."""
    if getattr(t, "get_device", _nowhere)() != on:
        _misplaced(t, name, on)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    s = t.shape
    if len(s) != 3 or (shape is not None and s != shape):
        raise ValueError(f"{name} must be {'tokens x heads x head_dim' if shape is None else tuple(shape)}, "
                         f"got {tuple(s)}")
    n, h, d = s
    if t.is_contiguous():
        return t.data_ptr(), h * d
    s = t.stride()
    if (s[2] != 1 and d != 1) or (s[1] != d and h != 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (s[0] if n > 1 else h * d)


def kv_write(cache, k, v, slots, stream=None):
    """Stores the rows k and v (tokens x kv_heads x head_dim, float32 or
    bfloat16; heads contiguous, tokens any stride apart) at the int32 `slots`
    of the cache, rounded or quantised as the cache is; a slot outside the
    cache skips its token."""
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    dtype = k.dtype
    on = cache._on
    kp, ks = _heads(k, "k", dtype, on, shape)
    vp, vs = _heads(v, "v", dtype, on, shape)
    _check(load().ptq_kv_write(cache._ref, kp, vp, ks, vs, _dev(slots, cache._int32, "slots", on), shape[0],
                               _act_dtype(k), _stream(stream, on)), "ptq_kv_write")


def kv_read(cache, slots, dtype=None, k=None, v=None, stream=None):
    """The values that the int32 `slots` of the cache stand for, as (k, v) of
    float32 or bfloat16 (default, where neither k nor v is given); into the
    given k and v (as for kv_write) or new tensors.  A slot outside the cache gives NaN."""
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    if dtype is None:
        given = v if k is None else k
        dtype = cache._bfloat16 if given is None else given.dtype
    on = cache._on
    sp = _dev(slots, cache._int32, "slots", on)
    if k is None:
        k = slots.new_empty(shape, dtype=dtype) if stream is None else _new(slots, shape, dtype, stream)
    if v is None:
        v = slots.new_empty(shape, dtype=dtype) if stream is None else _new(slots, shape, dtype, stream)
    kp, ks = _heads(k, "k", dtype, on, shape)
    vp, vs = _heads(v, "v", dtype, on, shape)
    _check(load().ptq_kv_read(cache._ref, sp, shape[0], kp, vp, ks, vs, _act_dtype(k),
                              _stream(stream, on)), "ptq_kv_read")
    return k, v


def attn_decode_workspace_bytes(B: int, q_heads: int, kv_heads: int, head_dim: int, dtype: int) -> int:
    return int(load().ptq_attn_decode_workspace_bytes(B, q_heads, kv_heads, head_dim, dtype))


def _attn_buffers(q, out, lse, workspace, need, stream, on):
    """The output, the addresses of out and lse, the workspace, its address and size."""
    if out is None:
        out = _new(q, q.shape, q.dtype, stream)
    elif out.shape != q.shape:
        raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
    op = _dev(out, q.dtype, "out", on)
    lp = wp = None
    wb = 0
    if lse is not None:
        import torch

        if lse.shape != q.shape[:2]:
            raise ValueError(f"lse must be {tuple(q.shape[:2])}, got {tuple(lse.shape)}")
        lp = _dev(lse, torch.float32, "lse", on)
    if workspace is None and (wb := need()) > 0:
        import torch

        workspace = _new(q, wb, torch.uint8, stream, returned=False)
    if workspace is not None:
        wp, wb = _dev(workspace, None, "workspace", on), workspace.nbytes
    return out, op, lp, wp, wb, workspace


def attn_decode(q, cache, table, lens, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token of each sequence over its cached tokens.
    q: sequences x q_heads x head_dim, float32 or bfloat16; table: sequences x
    pages int32 page numbers; lens: int32 token counts.  `scale` defaults to
    head_dim ** -0.5; `lse` (sequences x q_heads float32), when given, receives
    the log-sum-exp of the scaled scores.  out and the workspace are allocated
    by PyTorch when not given."""
    dt = _act_dtype(q)
    on = cache._on
    qp, qs = _heads(q, "q", q.dtype, on)
    B, Hq, D = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q has head_dim {D}, the cache {cache.head_dim}")
    ts, int32 = table.shape, cache._int32
    if len(ts) != 2 or ts[0] != B or lens.shape != (B,):
        raise ValueError("table must be sequences x pages, lens one count for each sequence")
    out, op, lp, wp, wb, keep = _attn_buffers(
        q, out, lse, workspace, lambda: attn_decode_workspace_bytes(B, Hq, cache.kv_heads, D, dt), stream, on)
    _check(load().ptq_attn_decode(qp, qs, cache._ref, _dev(table, int32, "table", on), ts[1],
                                  _dev(lens, int32, "lens", on), op, lp, B, Hq,
                                  D ** -0.5 if scale is None else scale, dt, wp, wb,
                                  _stream(stream, on)), "ptq_attn_decode")
    return out


def attn_prefill_workspace_bytes(B: int, Tq: int, Tk: int, q_heads: int, kv_heads: int, head_dim: int,
                                 dtype: int) -> int:
    return int(load().ptq_attn_prefill_workspace_bytes(B, Tq, Tk, q_heads, kv_heads, head_dim, dtype))


def attn_prefill(q, k, v, cu_q, cu_k, causal=True, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention of packed prompts.  q: queries x q_heads x head_dim, k and v:
    keys x kv_heads x head_dim, bfloat16; cu_q and cu_k: int32 offsets of the
    sequences in them (one more than there are sequences).  With `causal`
    query i of nq sees the keys j <= i + nk - nq of its sequence.  scale, out,
    lse and workspace as for attn_decode."""
    import torch

    dt, dtype, shape = _act_dtype(q), q.dtype, k.shape
    on = q.get_device() if getattr(q, "is_cuda", False) else _misplaced(q, "q", 0)
    qp, qs = _heads(q, "q", dtype, on)
    kp, ks = _heads(k, "k", dtype, on)
    vp, vs = _heads(v, "v", dtype, on, shape)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = shape
    if Dk != D:
        raise ValueError(f"q has head_dim {D}, k {Dk}")
    B = cu_q.numel() - 1
    if B < 0 or cu_q.shape != cu_k.shape:
        raise ValueError("cu_q and cu_k must have one offset more than there are sequences")
    out, op, lp, wp, wb, keep = _attn_buffers(
        q, out, lse, workspace, lambda: attn_prefill_workspace_bytes(B, Tq, Tk, Hq, Hkv, D, dt),
        stream, on)
    _check(load().ptq_attn_prefill(qp, kp, vp, qs, ks, vs, _dev(cu_q, torch.int32, "cu_q", on),
                                   _dev(cu_k, torch.int32, "cu_k", on), op, lp, B, Tq, Tk, Hq, Hkv, D,
                                   D ** -0.5 if scale is None else scale,
                                   PTQ_ATTN_CAUSAL if causal else 0, dt, wp, wb,
                                   _stream(stream, on)), "ptq_attn_prefill")
    return out


def route(M: int, dtype: int) -> str:
    name = ctypes.c_char_p()
    _check(load().ptq_route(M, dtype, ctypes.byref(name)), "ptq_route")
    return name.value.decode()


def matmul_f32_peel(wq, scales, x, out=None, stream=None):
    """Test export: the fp32 route's SIMT peel GEMV (ptq_matmul_f32_peel),
    y = x W^T with x float32 (already rotated), on any shape."""
    import torch

    M, K = x.shape
    N = wq.shape[0]
    y = _new(x, (M, N), torch.float32, stream) if out is None else out
    _check(load().ptq_matmul_f32_peel(
        _dev(wq, torch.uint8, "wq"), _dev(scales, torch.int16, "scales"),
        _dev(x, torch.float32, "x"), _dev(y, torch.float32, "out"), M, N, K, _stream(stream)),
        "ptq_matmul_f32_peel")
    return y


def gemv_plan(M: int, N: int, K: int, pq2: bool = False) -> dict:
    """The launch of the fp32 decode GEMV for (M, N, K) on the current device
    (ptq_gemv_plan): CTAs, cluster size (0: none), K-chunks, kernels."""
    out = (ctypes.c_int32 * 4)()
    _check(load().ptq_gemv_plan(M, N, K, int(pq2), out), "ptq_gemv_plan")
    return {"ctas": out[0], "cluster": out[1], "chunks": out[2], "kernels": out[3]}


def selftest_timeout(stream=None) -> None:
    """Runs the bounded wait that is made to run out (ptq_selftest_timeout);
    the next device_check raises PTQ_ERR_TIMEOUT."""
    _check(load().ptq_selftest_timeout(_stream(stream)), "ptq_selftest_timeout")


def selftest_grid_timeout(stream=None) -> None:
    """Runs the persistent stack's grid barrier with one CTA that never
    arrives (ptq_selftest_grid_timeout); the next device_check raises
    PTQ_ERR_TIMEOUT."""
    _check(load().ptq_selftest_grid_timeout(_stream(stream)), "ptq_selftest_grid_timeout")


def device_check(stream=None) -> None:
    _check(load().ptq_device_check(_stream(stream)), "ptq_device_check")
