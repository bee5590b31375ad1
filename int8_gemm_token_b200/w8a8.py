"""ctypes binding of libw8a8 (include/w8a8.h) over torch CUDA tensors.

Argument marshalling only: every function here checks tensor dtypes/shapes,
passes raw device pointers, sizes and the current CUDA stream to the C entry
point of the same name, and raises W8A8Error when it returns a non-OK status.
All compute runs in the library's kernels; there is no fallback. If
libw8a8.so is missing or cannot load, the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os
import re
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libw8a8.so")
HEADER = os.path.join(ROOT, "include", "w8a8.h")

OK = 0
BF16, FP32, I32 = 0, 1, 2
DECODE_MAX_M = 64  # calls with at most this many tokens take the weight-streaming decode kernel
STATUS_NAMES = {}


class W8A8Error(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


_lock = threading.Lock()
_lib = None

_P, _I64, _I32, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
_SIGNATURES = {
    "w8a8_status_string": (ctypes.c_char_p, [_I32]),
    "w8a8_quant_weight_per_channel": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]),
    "w8a8_calibrate_static": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]),
    "w8a8_quant_per_token": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "w8a8_quant_per_tensor": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P]),
    "w8a8_dequant_per_tensor": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _I32, _P]),
    "w8a8_gemm_dequant": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I32, _P, _SZ, _P]),
    "w8a8_gemm_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "w8a8_linear_static": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I32, _P, _SZ, _P]),
    "w8a8_gemm_requant": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P]),
    "w8a8_linear_static_requant": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P,
                                          _SZ, _P]),
    "w8a8_linear_static_noalloc": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I32, _P]),
    "int8_outlier_split": (_I32, [_P, _I64, _I64, _I64, _F, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "int8_outlier_split_workspace_size": (_SZ, [_I64]),
    "int8_mixed_decomp_gemm": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _I32, _P]),
    "int8_mixed_decomp_gemm_tc": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _I32,
                                         _P, _SZ, _P]),
    "int8_mixed_decomp_gemm_tc_workspace_size": (_SZ, [_I64, _I64, _I32]),
    "w8a8_kv_append": (_I32, [_P, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I32, _I32, _P, _I64, _I64,
                              _I32, _P, _P]),
    "w8a8_kv_gather": (_I32, [_P, _P, _I64, _I32, _I32, _P, _P, _I64, _P, _P, _I32, _P]),
    "w8a8_kv_attention": (_I32, [_P, _P, _I64, _P, _I64, _I64, _I32, _P, _P, _P, _SZ, _P]),
    "w8a8_kv_attention_requant": (_I32, [_P, _P, _I64, _P, _I64, _I64, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "w8a8_kv_attention_workspace_size": (_SZ, [_P, _P, _I64, _I32]),
    "w8a8_check_device_error": (_I32, [_P, _P]),
    "w8a8_debug_wait_timeout_selftest": (_I32, [ctypes.c_uint64, _P]),
}


def header_symbols() -> list[str]:
    """Names of the functions include/w8a8.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[\w]+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)


def lib() -> ctypes.CDLL:
    """Load libw8a8.so (once) and declare every entry point's signature."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m int8_gemm_token_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().w8a8_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != OK:
        raise W8A8Error(fn, status, status_string(status))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dt(dtype) -> int:
    return {torch.bfloat16: BF16, torch.float32: FP32, torch.int32: I32}[dtype]


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("expected a 2-D tensor with contiguous rows")
    return t.stride(0)


def _expect(t: torch.Tensor, dtype, shape, what: str):
    """Raise before the C call when a tensor the C side takes as a raw
    pointer of a fixed type and dense layout is not that."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _rows(t: torch.Tensor, dtype, what: str, shape=None) -> int:
    """A 2-D matrix of `dtype` whose rows are contiguous (any row stride);
    returns the row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: expected a 2-D tensor with contiguous rows, got shape {tuple(t.shape)} "
                         f"strides {tuple(t.stride())}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.stride(0)


def _vec(t, dtype, n: int, what: str, optional: bool = False):
    """A dense vector of n elements (n = 1: a device scalar, shape (1,) or ())."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{what}: required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.dim() > 1:
        raise ValueError(f"{what}: expected a contiguous {dtype} vector of {n} element(s), "
                         f"got {t.dtype} {tuple(t.shape)}")


def _on_one_gpu(*ts):
    """Every tensor a CUDA tensor on the same device (checked after the
    shapes, so shape errors are reported first)."""
    devs = {t.device for t in ts if t is not None}
    if any(d.type != "cuda" for d in devs) or len(devs) > 1:
        raise ValueError(f"expected CUDA tensors on one device, got {sorted(str(d) for d in devs)}")


def _out(out, dtype, shape, dev, allowed, what="out"):
    if out is None:
        if dtype not in allowed:
            raise ValueError(f"{what}: dtype must be one of {allowed}, got {dtype}")
        return torch.empty(shape, dtype=dtype, device=dev)
    if out.dtype not in allowed:
        raise ValueError(f"{what}: dtype must be one of {allowed}, got {out.dtype}")
    _expect(out, out.dtype, shape, what)
    return out


_GEMM_OUT = (torch.bfloat16, torch.float32, torch.int32)


# --------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# --------------------------------------------------------------------------

def w8a8_quant_weight_per_channel(W: torch.Tensor, Wq=None, s_w=None, colsum=None, stream=None):
    """W [K, N] bf16/fp32 -> (Wq int8 [N, K], s_w fp32 [N], colsum int32 [N])."""
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"W: expected bfloat16 or float32, got {W.dtype}")
    ldw = _rows(W, W.dtype, "W")
    K, N = W.shape
    dev = W.device
    Wq = torch.empty((N, K), dtype=torch.int8, device=dev) if Wq is None else Wq
    s_w = torch.empty((N,), dtype=torch.float32, device=dev) if s_w is None else s_w
    colsum = torch.empty((N,), dtype=torch.int32, device=dev) if colsum is None else colsum
    _expect(Wq, torch.int8, (N, K), "Wq")
    _vec(s_w, torch.float32, N, "s_w")
    _vec(colsum, torch.int32, N, "colsum")
    _on_one_gpu(W, Wq, s_w, colsum)
    _check("w8a8_quant_weight_per_channel", lib().w8a8_quant_weight_per_channel(
        _ptr(W), _dt(W.dtype), K, N, ldw, _ptr(Wq), _ptr(s_w), _ptr(colsum), _stream(stream)))
    return Wq, s_w, colsum


def w8a8_calibrate_static(Xcal: torch.Tensor, S=None, r=None, Z=None, stream=None):
    """MinMax calibration over Xcal [T, K] -> device scalars (S, r, Z)."""
    if Xcal.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"Xcal: expected bfloat16 or float32, got {Xcal.dtype}")
    ldx = _rows(Xcal, Xcal.dtype, "Xcal")
    T, K = Xcal.shape
    dev = Xcal.device
    S = torch.empty((1,), dtype=torch.float32, device=dev) if S is None else S
    r = torch.empty((1,), dtype=torch.float32, device=dev) if r is None else r
    Z = torch.empty((1,), dtype=torch.int32, device=dev) if Z is None else Z
    _vec(S, torch.float32, 1, "S")
    _vec(r, torch.float32, 1, "r")
    _vec(Z, torch.int32, 1, "Z")
    _on_one_gpu(Xcal, S, r, Z)
    _check("w8a8_calibrate_static", lib().w8a8_calibrate_static(
        _ptr(Xcal), _dt(Xcal.dtype), T, K, ldx, _ptr(S), _ptr(r), _ptr(Z), _stream(stream)))
    return S, r, Z


def w8a8_quant_per_token(X: torch.Tensor, Xq=None, S_x=None, stream=None):
    """bf16 X [M, K] -> (Xq int8 [M, K], S_x fp32 [M])."""
    ldx = _rows(X, torch.bfloat16, "X")
    M, K = X.shape
    Xq = torch.empty((M, K), dtype=torch.int8, device=X.device) if Xq is None else Xq
    S_x = torch.empty((M,), dtype=torch.float32, device=X.device) if S_x is None else S_x
    _expect(Xq, torch.int8, (M, K), "Xq")
    _vec(S_x, torch.float32, M, "S_x")
    _on_one_gpu(X, Xq, S_x)
    _check("w8a8_quant_per_token", lib().w8a8_quant_per_token(
        _ptr(X), M, K, ldx, _ptr(Xq), _ptr(S_x), _stream(stream)))
    return Xq, S_x


def w8a8_quant_per_tensor(X: torch.Tensor, r: torch.Tensor, Z: torch.Tensor, Xq=None, stream=None):
    """bf16 X [M, K] -> int8 codes clamp(rne(X r) + Z) [M, K]."""
    ldx = _rows(X, torch.bfloat16, "X")
    M, K = X.shape
    Xq = torch.empty((M, K), dtype=torch.int8, device=X.device) if Xq is None else Xq
    _expect(Xq, torch.int8, (M, K), "Xq")
    _vec(r, torch.float32, 1, "r")
    _vec(Z, torch.int32, 1, "Z")
    _on_one_gpu(X, Xq, r, Z)
    _check("w8a8_quant_per_tensor", lib().w8a8_quant_per_tensor(
        _ptr(X), M, K, ldx, _ptr(r), _ptr(Z), _ptr(Xq), _stream(stream)))
    return Xq


def w8a8_dequant_per_tensor(Xq: torch.Tensor, S: torch.Tensor, Z: torch.Tensor, out=None, out_dtype=torch.bfloat16,
                            stream=None):
    """int8 Xq [M, K] -> S * (Xq - Z) as bf16 or fp32 [M, K]."""
    if Xq.dtype != torch.int8:
        raise ValueError(f"Xq: expected int8 codes, got {Xq.dtype}")
    ldq = _rows(Xq, torch.int8, "Xq")
    M, K = Xq.shape
    out = _out(out, out_dtype, (M, K), Xq.device, (torch.bfloat16, torch.float32))
    _vec(S, torch.float32, 1, "S")
    _vec(Z, torch.int32, 1, "Z")
    _on_one_gpu(Xq, out, S, Z)
    _check("w8a8_dequant_per_tensor", lib().w8a8_dequant_per_tensor(
        _ptr(Xq), M, K, ldq, _ptr(S), _ptr(Z), _ptr(out), _dt(out.dtype),
        _stream(stream)))
    return out


def w8a8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().w8a8_gemm_workspace_size(M, N, K))


def new_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A workspace for w8a8_linear_static of this shape (None when the shape
    needs none). It needs no initial contents; calls on one stream may share it."""
    n = w8a8_gemm_workspace_size(M, N, K)
    if n == 0:
        return None
    return torch.empty((n,), dtype=torch.uint8, device=device or torch.device("cuda"))


def _workspace(n: int, dev, ws):
    if ws is None:
        if n == 0:
            return None, 0
        ws = torch.empty((n,), dtype=torch.uint8, device=dev)
    if not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return ws, ws.numel() * ws.element_size()


def _weight_operands(Wq, s_w, colsum, bias, K):
    """Wq int8 [N, K] dense, s_w fp32 [N], colsum int32 [N] (optional), bias fp32 [N] (optional)."""
    if Wq.dtype != torch.int8 or Wq.dim() != 2:
        raise ValueError(f"Wq: expected a 2-D int8 tensor, got {Wq.dtype} {tuple(Wq.shape)}")
    N = Wq.shape[0]
    _expect(Wq, torch.int8, (N, K), "Wq")
    _vec(s_w, torch.float32, N, "s_w")
    _vec(colsum, torch.int32, N, "colsum", optional=True)
    _vec(bias, torch.float32, N, "bias", optional=True)
    return N


def _scales(S_x, M):
    if S_x is None or S_x.numel() not in (1, M):
        raise ValueError("S_x holds one scale per row or a single per-tensor scale")
    _vec(S_x, torch.float32, S_x.numel(), "S_x")
    return 1 if S_x.numel() == M else 0  # M == 1: both readings give the same single scale


def w8a8_gemm_dequant(Xq, S_x, Wq, s_w, colsum=None, Z=None, bias=None, out=None,
                      out_dtype=torch.bfloat16, workspace=None, stream=None):
    """out [M, N] = S_x * s_w * (Xq Wq^T - Z * colsum) + bias.

    S_x is [M] (per token) or a 1-element tensor (per tensor)."""
    if Xq.dtype != torch.int8 or Xq.dim() != 2:
        raise ValueError(f"Xq: expected a 2-D int8 tensor, got {Xq.dtype} {tuple(Xq.shape)}")
    M, K = Xq.shape
    _expect(Xq, torch.int8, (M, K), "Xq")
    N = _weight_operands(Wq, s_w, colsum, bias, K)
    per_row = _scales(S_x, M)
    _vec(Z, torch.int32, 1, "Z", optional=True)
    if Z is not None and colsum is None:
        raise ValueError("colsum: required with a zero point Z")
    out = _out(out, out_dtype, (M, N), Xq.device, _GEMM_OUT)
    ws, nbytes = (None, 0) if workspace is None else _workspace(0, Xq.device, workspace)
    _on_one_gpu(Xq, S_x, Wq, s_w, colsum, Z, bias, out, ws)
    _check("w8a8_gemm_dequant", lib().w8a8_gemm_dequant(
        _ptr(Xq), _ptr(S_x), per_row, _ptr(Z), _ptr(Wq), _ptr(s_w), _ptr(colsum), _ptr(bias),
        M, N, K, _ptr(out), _dt(out.dtype), _ptr(ws), nbytes, _stream(stream)))
    return out


def _static_inputs(X, S, r, Z, Wq, s_w, colsum, bias):
    ldx = _rows(X, torch.bfloat16, "X")
    M, K = X.shape
    N = _weight_operands(Wq, s_w, colsum, bias, K)
    if colsum is None:
        raise ValueError("colsum: required (the zero-point correction)")
    _vec(S, torch.float32, 1, "S")
    _vec(r, torch.float32, 1, "r")
    _vec(Z, torch.int32, 1, "Z")
    return ldx, M, K, N


def w8a8_linear_static(X, S, r, Z, Wq, s_w, colsum, bias=None, out=None, out_dtype=torch.bfloat16,
                       workspace=None, stream=None):
    """Fused Decode linear with static per-tensor quantization of bf16 X."""
    ldx, M, K, N = _static_inputs(X, S, r, Z, Wq, s_w, colsum, bias)
    out = _out(out, out_dtype, (M, N), X.device, _GEMM_OUT)
    ws, nbytes = _workspace(w8a8_gemm_workspace_size(M, N, K), X.device, workspace)
    _on_one_gpu(X, S, r, Z, Wq, s_w, colsum, bias, out, ws)
    _check("w8a8_linear_static", lib().w8a8_linear_static(
        _ptr(X), M, K, ldx, _ptr(S), _ptr(r), _ptr(Z), _ptr(Wq), _ptr(s_w), _ptr(colsum),
        _ptr(bias), N, _ptr(out), _dt(out.dtype), _ptr(ws), nbytes, _stream(stream)))
    return out


def w8a8_gemm_requant(Xq, S_x, Wq, s_w, r_out, Z_out, colsum=None, Z=None, bias=None, out=None, stream=None):
    """w8a8_gemm_dequant whose bf16 result is quantized at once with the next
    linear's static r_out, Z_out: returns int8 [M, N] (M <= 64)."""
    if Xq.dtype != torch.int8 or Xq.dim() != 2:
        raise ValueError(f"Xq: expected a 2-D int8 tensor, got {Xq.dtype} {tuple(Xq.shape)}")
    M, K = Xq.shape
    _expect(Xq, torch.int8, (M, K), "Xq")
    N = _weight_operands(Wq, s_w, colsum, bias, K)
    per_row = _scales(S_x, M)
    _vec(Z, torch.int32, 1, "Z", optional=True)
    if Z is not None and colsum is None:
        raise ValueError("colsum: required with a zero point Z")
    _vec(r_out, torch.float32, 1, "r_out")
    _vec(Z_out, torch.int32, 1, "Z_out")
    out = _out(out, torch.int8, (M, N), Xq.device, (torch.int8,))
    _on_one_gpu(Xq, S_x, Wq, s_w, colsum, Z, bias, r_out, Z_out, out)
    _check("w8a8_gemm_requant", lib().w8a8_gemm_requant(
        _ptr(Xq), _ptr(S_x), per_row, _ptr(Z), _ptr(Wq), _ptr(s_w), _ptr(colsum), _ptr(bias), M, N, K,
        _ptr(r_out), _ptr(Z_out), _ptr(out), _stream(stream)))
    return out


def w8a8_linear_static_requant(X, S, r, Z, Wq, s_w, colsum, r_out, Z_out, bias=None, out=None, workspace=None,
                               stream=None):
    """Decode linear whose bf16 result is quantized at once with the next
    linear's static r_out, Z_out: returns int8 [M, N] (M <= 64)."""
    ldx, M, K, N = _static_inputs(X, S, r, Z, Wq, s_w, colsum, bias)
    _vec(r_out, torch.float32, 1, "r_out")
    _vec(Z_out, torch.int32, 1, "Z_out")
    out = _out(out, torch.int8, (M, N), X.device, (torch.int8,))
    ws, nbytes = _workspace(w8a8_gemm_workspace_size(M, N, K), X.device, workspace)
    _on_one_gpu(X, S, r, Z, Wq, s_w, colsum, bias, r_out, Z_out, out, ws)
    _check("w8a8_linear_static_requant", lib().w8a8_linear_static_requant(
        _ptr(X), M, K, ldx, _ptr(S), _ptr(r), _ptr(Z), _ptr(Wq), _ptr(s_w), _ptr(colsum), _ptr(bias), N,
        _ptr(r_out), _ptr(Z_out), _ptr(out), _ptr(ws), nbytes, _stream(stream)))
    return out


def w8a8_linear_static_noalloc(X, S, r, Z, Wq, s_w, colsum, bias=None, out=None, out_dtype=torch.bfloat16,
                               stream=None):
    """w8a8_linear_static with the library's own fixed scratch instead of a
    caller workspace (M <= 32, N <= 32768, K <= 16384)."""
    ldx, M, K, N = _static_inputs(X, S, r, Z, Wq, s_w, colsum, bias)
    out = _out(out, out_dtype, (M, N), X.device, _GEMM_OUT)
    _on_one_gpu(X, S, r, Z, Wq, s_w, colsum, bias, out)
    _check("w8a8_linear_static_noalloc", lib().w8a8_linear_static_noalloc(
        _ptr(X), M, K, ldx, _ptr(S), _ptr(r), _ptr(Z), _ptr(Wq), _ptr(s_w), _ptr(colsum), _ptr(bias), N,
        _ptr(out), _dt(out.dtype), _stream(stream)))
    return out


def int8_outlier_split(X, threshold: float = 6.0, cap: int = 64, Xq=None, S_x=None, idx=None,
                       n_out=None, Xo=None, workspace=None, stream=None):
    """LLM.int8() split -> (Xq, S_x, outlier_idx [cap], n_out [1], Xo [M, cap])."""
    ldx = _rows(X, torch.bfloat16, "X")
    M, K = X.shape
    cap = int(cap)
    dev = X.device
    Xq = torch.empty((M, K), dtype=torch.int8, device=dev) if Xq is None else Xq
    S_x = torch.empty((M,), dtype=torch.float32, device=dev) if S_x is None else S_x
    idx = torch.empty((max(cap, 1),), dtype=torch.int32, device=dev) if idx is None else idx
    n_out = torch.empty((1,), dtype=torch.int32, device=dev) if n_out is None else n_out
    Xo = torch.empty((M, max(cap, 1)), dtype=torch.bfloat16, device=dev) if Xo is None else Xo
    _expect(Xq, torch.int8, (M, K), "Xq")
    _vec(S_x, torch.float32, M, "S_x")
    _vec(n_out, torch.int32, 1, "n_out")
    if idx.dtype != torch.int32 or idx.numel() < cap or not idx.is_contiguous():
        raise ValueError(f"idx: expected a contiguous int32 tensor of at least {cap} elements")
    _expect(Xo, torch.bfloat16, (M, max(cap, 1)), "Xo")
    ws, nbytes = _workspace(int(lib().int8_outlier_split_workspace_size(K)), dev, workspace)
    _on_one_gpu(X, Xq, S_x, idx, n_out, Xo, ws)
    _check("int8_outlier_split", lib().int8_outlier_split(
        _ptr(X), M, K, ldx, float(threshold), cap, _ptr(Xq), _ptr(S_x), _ptr(idx), _ptr(n_out),
        _ptr(Xo), _ptr(ws), nbytes, _stream(stream)))
    return Xq, S_x, idx, n_out, Xo


def _mixed(fn, Xq, S_x, Xo, idx, n_out, cap, Wq, s_w, W, bias, out, out_dtype, stream, workspace=None):
    if Xq.dtype != torch.int8 or Xq.dim() != 2:
        raise ValueError(f"Xq: expected a 2-D int8 tensor, got {Xq.dtype} {tuple(Xq.shape)}")
    M, K = Xq.shape
    cap = int(cap)
    _expect(Xq, torch.int8, (M, K), "Xq")
    N = _weight_operands(Wq, s_w, None, bias, K)
    _vec(S_x, torch.float32, M, "S_x")
    _expect(Xo, torch.bfloat16, (M, max(cap, 1)), "Xo")
    if idx.dtype != torch.int32 or idx.numel() < cap or not idx.is_contiguous():
        raise ValueError(f"idx: expected a contiguous int32 tensor of at least {cap} elements")
    _vec(n_out, torch.int32, 1, "n_out")
    ldw = _rows(W, torch.bfloat16, "W", shape=(K, N))
    out = _out(out, out_dtype, (M, N), Xq.device, (torch.bfloat16, torch.float32))
    args = [_ptr(Xq), _ptr(S_x), _ptr(Xo), _ptr(idx), _ptr(n_out), cap, _ptr(Wq), _ptr(s_w), _ptr(W),
            ldw, _ptr(bias), M, N, K, _ptr(out), _dt(out.dtype)]
    ws = None
    if fn == "int8_mixed_decomp_gemm_tc":
        ws, nbytes = _workspace(int(lib().int8_mixed_decomp_gemm_tc_workspace_size(M, N, cap)), Xq.device, workspace)
        args += [_ptr(ws), nbytes]
    _on_one_gpu(Xq, S_x, Xo, idx, n_out, Wq, s_w, W, bias, out, ws)
    _check(fn, getattr(lib(), fn)(*args, _stream(stream)))
    return out


def int8_mixed_decomp_gemm(Xq, S_x, Xo, idx, n_out, cap: int, Wq, s_w, W, bias=None, out=None,
                           out_dtype=torch.bfloat16, stream=None):
    """INT8 vector-wise product + bf16 outlier side product (fixed-order fmaf
    chain on CUDA cores), summed in the epilogue."""
    return _mixed("int8_mixed_decomp_gemm", Xq, S_x, Xo, idx, n_out, cap, Wq, s_w, W, bias, out, out_dtype, stream)


def int8_mixed_decomp_gemm_tc(Xq, S_x, Xo, idx, n_out, cap: int, Wq, s_w, W, bias=None, out=None,
                              out_dtype=torch.bfloat16, workspace=None, stream=None):
    """The same decomposition with the bf16 side product on the tensor cores
    (kind::f16 MMAs into a second TMEM accumulator); `workspace` (allocated
    when None) holds the padded side operands."""
    return _mixed("int8_mixed_decomp_gemm_tc", Xq, S_x, Xo, idx, n_out, cap, Wq, s_w, W, bias, out, out_dtype,
                  stream, workspace)


# --------------------------------------------------------------------------
# INT8 paged KV cache
# --------------------------------------------------------------------------

class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_scale", _P), ("v_scale", _P), ("num_pages", _I64),
                ("kv_heads", _I32), ("page_size", _I32), ("head_dim", _I32)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("page_table", _P), ("page_table_ld", _I64), ("seq_start", _P), ("kv_len", _P), ("batch", _I32),
                ("max_pages", _I32), ("max_q_len", _I32), ("max_kv_len", _I32)]


class _ScoresStruct(ctypes.Structure):
    _fields_ = [("scale", _F), ("softcap", _F), ("slopes", _P), ("window", _I32), ("prefix_len", _P)]


class _Described:
    """What the C calls get is taken from the attributes once, when the object
    is made. So those cannot be assigned again: the calls would not see it."""

    _taken = frozenset()

    def __setattr__(self, name, value):
        if name in self._taken:
            raise AttributeError(f"{type(self).__name__}.{name} was taken when the object was made: make another one")
        object.__setattr__(self, name, value)


class PagedKVCache(_Described):
    """An INT8 paged KV cache (w8a8_kv_cache): codes int8 [pages, kv_heads,
    page_size, head_dim] and scales fp32 [pages, kv_heads], for keys and for
    values. Checked once here; keeps the tensors alive. Their contents may
    change between calls, the tensors may be neither resized nor exchanged."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        if not isinstance(k_codes, torch.Tensor) or k_codes.dtype != torch.int8 or k_codes.dim() != 4:
            raise ValueError("k_codes: expected an int8 tensor [pages, kv_heads, page_size, head_dim]")
        shape = tuple(k_codes.shape)
        _expect(k_codes, torch.int8, shape, "k_codes")
        _expect(v_codes, torch.int8, shape, "v_codes")
        _expect(k_scale, torch.float32, shape[:2], "k_scale")
        _expect(v_scale, torch.float32, shape[:2], "v_scale")
        if shape[2] not in (16, 32, 64, 128):
            raise ValueError(f"k_codes: page size must be 16, 32, 64 or 128, got {shape[2]}")
        if shape[3] not in (64, 96, 128):
            raise ValueError(f"k_codes: head dim must be 64, 96 or 128, got {shape[3]}")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = shape
        self.device, self._dev = k_codes.device, k_codes.get_device()
        self._tensors = (k_codes, v_codes, k_scale, v_scale)
        if any(t.device != self.device for t in self._tensors):
            raise ValueError(f"expected tensors on one device, got {sorted({str(t.device) for t in self._tensors})}")
        self._c = _CacheStruct(*(t.data_ptr() for t in self._tensors), *shape)
        self._ref = ctypes.byref(self._c)
        self._taken = frozenset(vars(self))

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, device=None):
        """A cache of zeroed pages."""
        device = device or torch.device("cuda")
        codes = [torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=torch.int8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros((num_pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def _bound(x) -> int:
    """A host bound as the C int, which ctypes would cut to its low 32 bits: past the int's range the range's end
    says the same (no sequence is that long)."""
    return min(max(operator.index(x), -2 ** 31), 2 ** 31 - 1)


def _page_table(t) -> int:
    """The row stride of an int32 [batch, max_pages] page table. (Of one row or none torch may report any stride;
    the C calls want at least the row's length. Rows that overlap are no table the kernels can walk.)"""
    ld = _rows(t, torch.int32, "page_table")
    if ld >= t.shape[1]:
        return ld
    if t.shape[0] > 1:
        raise ValueError(f"page_table: rows overlap (shape {tuple(t.shape)} strides {tuple(t.stride())}); "
                         "sequences that share pages need a row each, as .contiguous() makes them")
    return t.shape[1]


class KVBatch(_Described):
    """The sequences of a call (w8a8_kv_batch): page_table int32 [batch,
    max_pages] (rows contiguous, at any distance that keeps them apart),
    seq_start int32 [batch + 1], kv_len int32 [batch], all on the device and
    read there, and the host's bounds on a sequence's new tokens and length
    (without max_kv_len what the table holds; attention of many new tokens
    takes workspace for batch * kv_heads * max_kv_len keys, see
    w8a8_kv_attention_workspace_size in the header). Checked once here; as of
    a PagedKVCache, only the tensors' contents may change."""

    def __init__(self, page_table, seq_start, kv_len, max_q_len: int, max_kv_len: int | None = None):
        ld = _page_table(page_table)
        batch, max_pages = page_table.shape
        _vec(seq_start, torch.int32, batch + 1, "seq_start")
        _vec(kv_len, torch.int32, batch, "kv_len")
        self.page_table, self.seq_start, self.kv_len = page_table, seq_start, kv_len
        self.max_q_len, self.max_kv_len = _bound(int(max_q_len)), max_kv_len
        if seq_start.device != page_table.device or kv_len.device != page_table.device:
            raise ValueError("expected page_table, seq_start and kv_len on one device")
        self.size, self._max_pages = batch, max_pages
        self._fields = (page_table.data_ptr(), ld, seq_start.data_ptr(), kv_len.data_ptr(), batch, max_pages,
                        self.max_q_len)
        self._refs = {}
        self._taken = frozenset(vars(self))

    def _for(self, cache: PagedKVCache):
        """The C struct for caches of that page size, with the longest length
        the table can hold where the caller gave none. (One for each page
        size, never written again: threads and caches may share a batch.)"""
        ref = self._refs.get(cache.page_size)
        if ref is None:
            most = self._max_pages * cache.page_size if self.max_kv_len is None else int(self.max_kv_len)
            ref = self._refs[cache.page_size] = ctypes.byref(_BatchStruct(*self._fields, _bound(most)))
        return ref


# These calls run once or more for every layer of a Decode step of a few
# microseconds, so their marshalling is kept short: each tensor is looked at
# once (dtype, shape, strides, device index) and what does not change between
# steps was checked when the PagedKVCache and KVBatch were made.

def _bad(what: str, expected: str, t):
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    return ValueError(f"{what}: expected {expected}, got {t.dtype} {tuple(t.shape)} strides {tuple(t.stride())}")


def _heads3(t, heads, d, what: str, tokens=None):
    """A bf16 tensor [tokens, heads, d] whose last axis is contiguous: its
    shape and its strides between tokens and heads in elements."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16:
        shape, stride = t.shape, t.stride()
        if len(shape) == 3 and shape[2] == d and stride[2] == 1 and (heads is None or shape[1] == heads) \
                and (tokens is None or shape[0] == tokens):
            # the stride of an axis of one (or no) element is never used; torch may report any value for it
            return shape[0], shape[1], (stride[0] if shape[0] > 1 else 0), (stride[1] if shape[1] > 1 else 0)
    raise _bad(what, f"bfloat16 [{'tokens' if tokens is None else tokens}, {'heads' if heads is None else heads}, {d}] "
                     "with a contiguous last axis", t)


def _dense(t, dtype, shape, what: str):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise _bad(what, f"a contiguous {dtype} tensor of shape {tuple(shape)}", t)


def _same_gpu(dev: int, *ts):
    """Every tensor on the GPU of that index (checked after the shapes, as in _on_one_gpu)."""
    for t in ts:
        if t is not None and t.get_device() != dev or dev < 0:
            raise ValueError(f"expected CUDA tensors on one device, got {sorted({str(t.device) for t in ts if t is not None})}")


def _allocating(stream):
    """Where what a call allocates is used on a given stream, it comes from that stream's memory: the
    current stream may still use a freed block, or be given this one while the call runs."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


_entry = {}
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without making a Stream object


def _kv_fn(name):
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(lib(), name)
    return f


def _kv_call(fn, dev: int, stream, *args):
    """Call entry point `fn` with GPU `dev` current, on the given stream or the GPU's current one."""
    f = _kv_fn(fn)
    if stream is not None:
        raw = stream.cuda_stream
    elif _current_raw_stream is not None:
        raw = _current_raw_stream(dev)
    else:
        raw = torch.cuda.current_stream(dev).cuda_stream
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = f(*args, raw)
    else:
        status = f(*args, raw)
    if status:
        _check(fn, status)


def w8a8_kv_append(k, v, cache: PagedKVCache, batch: KVBatch, cos=None, sin=None, q=None, q_out=None,
                   interleaved: bool = False, stream=None):
    """Rotate (cos, sin fp32 [positions, rot_dim / 2]), quantize and store the
    new tokens' keys and values; with q, rotate the queries into q_out (bf16
    [tokens, q_heads, head_dim], allocated when None, and then uninitialised in
    rows of no sequence; returned)."""
    d, dev = cache.head_dim, cache._dev
    tokens, _, kst, ksh = _heads3(k, cache.kv_heads, d, "k")
    _, _, vst, vsh = _heads3(v, cache.kv_heads, d, "v", tokens)
    rope_len = half = 0
    cp = sp = qp = op = None
    if cos is not None:
        if sin is None:
            raise ValueError("cos and sin: give both or neither")
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise _bad("cos", "float32 [positions, rot_dim / 2]", cos)
        shape = cos.shape
        _dense(cos, torch.float32, shape, "cos")
        _dense(sin, torch.float32, shape, "sin")
        rope_len, half = shape
        cp, sp = cos.data_ptr(), sin.data_ptr()
    elif sin is not None:
        raise ValueError("cos and sin: give both or neither")
    qst = qsh = hq = 0
    if q is not None:
        _, hq, qst, qsh = _heads3(q, None, d, "q", tokens)
        if q_out is None:
            with _allocating(stream):
                q_out = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device=q.device)
        else:
            _dense(q_out, torch.bfloat16, (tokens, hq, d), "q_out")
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    _same_gpu(dev, k, v, cos, sin, q, q_out, batch.page_table)
    _kv_call("w8a8_kv_append", dev, stream, cache._ref, batch._for(cache), tokens, k.data_ptr(), kst, ksh, v.data_ptr(),
             vst, vsh, cp, sp, rope_len, 2 * half, 1 if interleaved else 0, qp, qst, qsh, hq, op)
    return q_out


def w8a8_kv_gather(cache: PagedKVCache, page_table, first_pos, row_start, rows: int | None = None, k_out=None,
                   v_out=None, out_dtype=torch.bfloat16, stream=None):
    """Read positions first_pos[b] .. of each sequence back into rows
    row_start[b] .. row_start[b + 1] of k_out and v_out [rows, kv_heads,
    head_dim] (bf16 or fp32; both allocated for `rows` rows when neither is
    given, and then uninitialised in rows of no sequence) -> (k_out, v_out)."""
    ld = _page_table(page_table)
    batch, max_pages = page_table.shape
    _dense(first_pos, torch.int32, (batch,), "first_pos")
    _dense(row_start, torch.int32, (batch + 1,), "row_start")
    given = k_out if k_out is not None else v_out
    if given is None:
        if rows is None:
            raise ValueError("rows: required where no output is given")
        shape = (int(rows), cache.kv_heads, cache.head_dim)
        with _allocating(stream):
            given = k_out = _out(None, out_dtype, shape, cache.device, (torch.bfloat16, torch.float32), "k_out")
            v_out = torch.empty_like(k_out)
    else:
        what = "k_out" if k_out is not None else "v_out"
        if not isinstance(given, torch.Tensor) or given.dtype not in (torch.bfloat16, torch.float32) or given.dim() != 3:
            raise _bad(what, "bfloat16 or float32 [rows, kv_heads, head_dim]", given)
        shape = (given.shape[0] if rows is None else int(rows), cache.kv_heads, cache.head_dim)
        _dense(given, given.dtype, shape, what)
        if k_out is not None and v_out is not None:
            _dense(v_out, given.dtype, shape, "v_out")
    _same_gpu(cache._dev, page_table, first_pos, row_start, k_out, v_out)
    _kv_call("w8a8_kv_gather", cache._dev, stream, cache._ref, page_table.data_ptr(), ld, batch, max_pages,
             first_pos.data_ptr(), row_start.data_ptr(), shape[0],
             None if k_out is None else k_out.data_ptr(), None if v_out is None else v_out.data_ptr(),
             BF16 if given.dtype is torch.bfloat16 else FP32)
    return k_out, v_out


def w8a8_kv_attention_workspace_size(cache: PagedKVCache, batch: KVBatch, tokens: int, q_heads: int) -> int:
    """Bytes of workspace the attention calls need, on the cache's GPU."""
    f = _kv_fn("w8a8_kv_attention_workspace_size")
    if cache._dev >= 0 and cache._dev != torch.cuda.current_device():
        with torch.cuda.device(cache._dev):
            return f(cache._ref, batch._for(cache), tokens, _bound(q_heads))
    return f(cache._ref, batch._for(cache), tokens, _bound(q_heads))


def _attention(fn, q, cache, batch, scale, softcap, window, slopes, prefix_len, out, out_dtype, extra, workspace, stream):
    d, dev = cache.head_dim, cache._dev
    tokens, hq, qst, qsh = _heads3(q, None, d, "q")
    sp = pp = None
    if slopes is not None:
        _dense(slopes, torch.float32, (hq,), "slopes")
        sp = slopes.data_ptr()
    if prefix_len is not None:
        _dense(prefix_len, torch.int32, (batch.size,), "prefix_len")
        pp = prefix_len.data_ptr()
    if out is None:
        with _allocating(stream):
            out = torch.empty((tokens, hq, d), dtype=out_dtype, device=q.device)
    else:
        _dense(out, out_dtype, (tokens, hq, d), "out")
    _same_gpu(dev, q, out, slopes, prefix_len, workspace, batch.page_table, *extra)
    if workspace is None:
        nbytes = w8a8_kv_attention_workspace_size(cache, batch, tokens, hq)
        if nbytes:
            with _allocating(stream):
                workspace = torch.empty((nbytes,), dtype=torch.uint8, device=q.device)
    else:
        workspace, nbytes = _workspace(0, q.device, workspace)
    sc = _ScoresStruct(d ** -0.5 if scale is None else scale, softcap, sp, _bound(window), pp)
    _kv_call(fn, dev, stream, cache._ref, batch._for(cache), tokens, q.data_ptr(), qst, qsh, hq, ctypes.byref(sc),
             *[t.data_ptr() for t in extra], out.data_ptr(), None if workspace is None else workspace.data_ptr(), nbytes)
    return out


def w8a8_kv_attention(q, cache: PagedKVCache, batch: KVBatch, scale: float | None = None, softcap: float = 0.0,
                      window: int = 0, slopes=None, prefix_len=None, out=None, workspace=None, stream=None):
    """Causal attention of bf16 q [tokens, q_heads, head_dim] over the cache ->
    bf16 of the same shape (rows of no sequence are left as they are in a
    given `out`, and uninitialised in one that is allocated here; so are those
    of a sequence that is skipped). scale defaults to head_dim ** -0.5; slopes
    [q_heads] add -slope * (query's position - key's)."""
    return _attention("w8a8_kv_attention", q, cache, batch, scale, softcap, window, slopes, prefix_len, out,
                      torch.bfloat16, (), workspace, stream)


def w8a8_kv_attention_requant(q, cache: PagedKVCache, batch: KVBatch, r_out, Z_out, scale: float | None = None,
                              softcap: float = 0.0, window: int = 0, slopes=None, prefix_len=None, out=None,
                              workspace=None, stream=None):
    """w8a8_kv_attention whose bf16 result is quantized at once with the output
    projection's static r_out, Z_out: returns int8 [tokens, q_heads, head_dim]
    (rows of no sequence as there)."""
    _vec(r_out, torch.float32, 1, "r_out")
    _vec(Z_out, torch.int32, 1, "Z_out")
    return _attention("w8a8_kv_attention_requant", q, cache, batch, scale, softcap, window, slopes, prefix_len, out,
                      torch.int8, (r_out, Z_out), workspace, stream)


def w8a8_check_device_error(stream=None) -> int:
    """Synchronize the stream, return and clear the device status word."""
    st = ctypes.c_int32(0)
    _check("w8a8_check_device_error", lib().w8a8_check_device_error(_stream(stream), ctypes.byref(st)))
    return int(st.value)


def w8a8_debug_wait_timeout_selftest(limit_ns: int = 5_000_000, stream=None):
    _check("w8a8_debug_wait_timeout_selftest",
           lib().w8a8_debug_wait_timeout_selftest(int(limit_ns), _stream(stream)))
