"""ctypes binding of libwql.so: argument marshalling only.

Every computation happens in the CUDA kernels behind the C ABI declared in ``include/wql.h``.
Tensors are torch CUDA tensors (torch is used for device memory and streams only); the calls are
enqueued on the current torch stream of the tensors' device.  There is no CPU fallback: if the
library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libwql.so")

WQL_OK, WQL_EINVAL, WQL_EUNSUPPORTED, WQL_ECUDA, WQL_ETIMEOUT = range(5)

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_I64 = ctypes.c_int64

# name -> (restype, argtypes); this list is also what the export test checks against wql.h
SIGNATURES = {
    "wql_status_string": (ctypes.c_char_p, [_I]),
    "wql_last_error": (ctypes.c_char_p, []),
    "wql_version": (_I, []),
    "wql_device_status": (_I, [_P]),
    "wql_diag_expire_wait": (_I, [_P]),
    "wql_trace_setup": (_I, [_P, _P, ctypes.c_uint64, _I, _I]),
    "wql_awq_pack": (_I, [_P, _I, _I, _I, _P, _P, _P, _P]),
    "wql_w4a16_gemm": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "wql_w4a16_kernel_for": (_I, [_I, _I, _I, _I]),
    "wql_w4a16_gemm_silu_mul": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "wql_qrmsnorm_quant_i8": (_I, [_P, _P, _F, _I, _I, _P, _P, _P]),
    "wql_add_qrmsnorm_quant_i8": (_I, [_P, _P, _P, _F, _I, _I, _P, _P, _P, _P]),
    "wql_per_token_quant_i8": (_I, [_P, _I, _I, _P, _P, _P]),
    "wql_per_token_quant_fp8": (_I, [_P, _I, _I, _P, _P, _P]),
    "wql_w8a8_workspace_bytes": (_SZ, [_I, _I, _I]),
    "wql_w8a8_gemm": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "wql_w8a8_gemm_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "wql_w8a8_gemm_fused": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "wql_act_absmax": (_I, [_P, _P, _F, _I, _I, _P, _P]),
    "wql_smooth": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P]),
    "wql_per_channel_quant_i8": (_I, [_P, _I, _I, _P, _P, _P]),
    "wql_qrmsnorm_quant_fp8": (_I, [_P, _P, _F, _I, _I, _P, _P, _P]),
    "wql_add_qrmsnorm_quant_fp8": (_I, [_P, _P, _P, _F, _I, _I, _P, _P, _P, _P]),
    "wql_per_channel_quant_fp8": (_I, [_P, _I, _I, _P, _P, _P]),
    "wql_w8a8_gemm_fp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "wql_kv_quant_i8": (_I, [_P, ctypes.c_int64, _I, _P, _P, _P]),
    "wql_kv_dequant_i8": (_I, [_P, _P, ctypes.c_int64, _I, _P, _P]),
    "wql_kv_plan_pages": (_I, [_P, _P, _I, _I, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P]),
    "wql_kv_append_i4": (_I, [_P, _P, _I64, _I64, _I, _I, _I, _P, _P, _I64, _I, _P]),
    "wql_kv_read_i4": (_I, [_P, _I64, _I, _I, _I, _P, _I, _P, _P, _P]),
    "wql_attention_kv_i4_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "wql_attention_kv_i4": (_I, [_P, _I64, _I, _I, _I, _I, _I, _P, _I64, _I, _P, _I, _P, _F, _P, _P, _SZ, _P]),
    "wql_attention_prompt": (_I, [_P, _I64, _P, _I64, _P, _I64, _I, _I, _I, _I, _P, _I, _F, _P, _P]),
}

_lock = threading.Lock()
_lib = None


class WQLError(RuntimeError):
    def __init__(self, status: int, fn: str, detail: str):
        self.status = status
        super().__init__(f"{fn}: status {status}: {detail}")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libwql.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(
                    f"libwql.so not found at {p}; build it with weight_quantized_linear_gb300.build.build()")
            lib = ctypes.CDLL(p)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _check(status: int, fn: str) -> None:
    if status != WQL_OK:
        lib = load()
        detail = lib.wql_last_error().decode() or lib.wql_status_string(status).decode()
        raise WQLError(status, fn, detail)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---------------------------------------------------------------------------------------------
# AWQ W4A16
# ---------------------------------------------------------------------------------------------

def awq_pack(w: torch.Tensor, group: int):
    """fp32 w [K, N] -> (qweight int32 [K, N/8], scales fp16 [K/G, N], qzeros int32 [K/G, N/8]).

    qweight / qzeros hold uint32 bit patterns in int32 tensors (torch has no uint32 arithmetic).
    """
    K, N = w.shape
    _need(w, "w", torch.float32, (K, N))
    dev = w.device
    qweight = torch.empty((K, N // 8), dtype=torch.int32, device=dev)
    scales = torch.empty((K // group, N), dtype=torch.float16, device=dev)
    qzeros = torch.empty((K // group, N // 8), dtype=torch.int32, device=dev)
    _check(load().wql_awq_pack(_ptr(w), K, N, group, _ptr(qweight), _ptr(scales), _ptr(qzeros), _stream(dev)),
           "wql_awq_pack")
    return qweight, scales, qzeros


def w4a16_gemm(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, qzeros: torch.Tensor, group: int,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """y [M, N] fp16 = x [M, K] fp16 @ dequant(qweight, scales, qzeros)."""
    M, K = x.shape
    N = qweight.shape[1] * 8
    _need(x, "x", torch.float16, (M, K))
    _need(qweight, "qweight", torch.int32, (K, N // 8))
    _need(scales, "scales", torch.float16, (K // group, N))
    _need(qzeros, "qzeros", torch.int32, (K // group, N // 8))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
    _need(out, "out", torch.float16, (M, N))
    _check(load().wql_w4a16_gemm(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros), M, K, N, group, _ptr(out),
                                 _stream(x.device)), "wql_w4a16_gemm")
    return out


def w4a16_gemm_silu_mul(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, qzeros: torch.Tensor,
                        group: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Fused gate/up projection: the packed weight has N = 2I channels with gate j at channel 2j and
    up j at 2j + 1; returns y [M, I] fp16 = fp16(silu(g) * u) of the GEMM's fp16 gate and up."""
    M, K = x.shape
    N = qweight.shape[1] * 8
    _need(x, "x", torch.float16, (M, K))
    _need(qweight, "qweight", torch.int32, (K, N // 8))
    _need(scales, "scales", torch.float16, (K // group, N))
    _need(qzeros, "qzeros", torch.int32, (K // group, N // 8))
    if out is None:
        out = torch.empty((M, N // 2), dtype=torch.float16, device=x.device)
    _need(out, "out", torch.float16, (M, N // 2))
    _check(load().wql_w4a16_gemm_silu_mul(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros), M, K, N, group,
                                          _ptr(out), _stream(x.device)), "wql_w4a16_gemm_silu_mul")
    return out


def interleave_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor) -> torch.Tensor:
    """[K, I] gate and up weights -> the [K, 2I] fused weight that w4a16_gemm_silu_mul expects
    (column 2j = gate j, column 2j + 1 = up j); pack it with awq_pack."""
    if w_gate.shape != w_up.shape or w_gate.dim() != 2:
        raise ValueError("gate and up weights must both be [K, I]")
    return torch.stack([w_gate, w_up], dim=2).reshape(w_gate.shape[0], 2 * w_gate.shape[1]).contiguous()


# ---------------------------------------------------------------------------------------------
# SmoothQuant W8A8
# ---------------------------------------------------------------------------------------------

def qrmsnorm_quant_i8(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                      q: torch.Tensor | None = None, xs: torch.Tensor | None = None):
    """x [M, K] fp16, gamma [K] fp16 -> (q int8 [M, K], xs fp32 [M])."""
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    _need(gamma, "gamma", torch.float16, (K,))
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(q, "q", torch.int8, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _check(load().wql_qrmsnorm_quant_i8(_ptr(x), _ptr(gamma), float(eps), M, K, _ptr(q), _ptr(xs), _stream(x.device)),
           "wql_qrmsnorm_quant_i8")
    return q, xs


def per_token_quant_i8(x: torch.Tensor, q: torch.Tensor | None = None, xs: torch.Tensor | None = None):
    """x [M, K] fp16 -> (q int8 [M, K], xs fp32 [M]): per-token int8 of the row itself (no norm)."""
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(q, "q", torch.int8, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _check(load().wql_per_token_quant_i8(_ptr(x), M, K, _ptr(q), _ptr(xs), _stream(x.device)), "wql_per_token_quant_i8")
    return q, xs


def per_token_quant_fp8(x: torch.Tensor, q: torch.Tensor | None = None, xs: torch.Tensor | None = None):
    """x [M, K] fp16 -> (q float8_e4m3fn [M, K], xs fp32 [M]) with xs = absmax / 448."""
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    if q is None:
        q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(q, "q", torch.float8_e4m3fn, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _check(load().wql_per_token_quant_fp8(_ptr(x), M, K, _ptr(q), _ptr(xs), _stream(x.device)),
           "wql_per_token_quant_fp8")
    return q, xs


def add_qrmsnorm_quant_i8(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                          residual_out: torch.Tensor | None = None, q: torch.Tensor | None = None,
                          xs: torch.Tensor | None = None):
    """Residual-fused QRMSNorm: h = fp16(x + residual) -> (h [M, K] fp16, q int8 [M, K], xs fp32 [M]).

    residual_out receives h (it may be `residual` itself, for an in-place update)."""
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    _need(residual, "residual", torch.float16, (M, K))
    _need(gamma, "gamma", torch.float16, (K,))
    if residual_out is None:
        residual_out = torch.empty((M, K), dtype=torch.float16, device=x.device)
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(residual_out, "residual_out", torch.float16, (M, K))
    _need(q, "q", torch.int8, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _check(load().wql_add_qrmsnorm_quant_i8(_ptr(x), _ptr(residual), _ptr(gamma), float(eps), M, K, _ptr(residual_out),
                                            _ptr(q), _ptr(xs), _stream(x.device)), "wql_add_qrmsnorm_quant_i8")
    return residual_out, q, xs


def w4a16_kernel_for(M: int, K: int, N: int, group: int) -> str:
    """The kernel w4a16_gemm runs for this shape and group size: "decode" or "prefill"."""
    return "prefill" if load().wql_w4a16_kernel_for(M, K, N, group) else "decode"


def w8a8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().wql_w8a8_workspace_bytes(M, K, N))


def w8a8_gemm(q: torch.Tensor, xs: torch.Tensor, qw: torch.Tensor, ws: torch.Tensor,
              out: torch.Tensor | None = None, acc_out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y [M, N] fp16 = fp16((float(q @ qw^T) * xs) * ws); optional exact int32 acc_out [M, N]."""
    M, K = q.shape
    N = qw.shape[0]
    _need(q, "q", torch.int8, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _need(qw, "qw", torch.int8, (N, K))
    _need(ws, "ws", torch.float32, (N,))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=q.device)
    _need(out, "out", torch.float16, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, N))
    need = w8a8_workspace_bytes(M, K, N)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().wql_w8a8_gemm(_ptr(q), _ptr(xs), _ptr(qw), _ptr(ws), M, K, N, _ptr(out), _ptr(acc_out),
                                _ptr(workspace), ws_bytes, _stream(q.device)), "wql_w8a8_gemm")
    return out


def w8a8_gemm_fused(q: torch.Tensor, xs: torch.Tensor, qw: torch.Tensor, ws: torch.Tensor,
                    bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, acc_out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y [M, N] fp16 = fp16(((float(q @ qw^T) * xs) * ws + bias) + residual); bias [N] and residual
    [M, N] fp16 are optional (None leaves the term out); `out` may be `residual` (in place)."""
    M, K = q.shape
    N = qw.shape[0]
    _need(q, "q", torch.int8, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _need(qw, "qw", torch.int8, (N, K))
    _need(ws, "ws", torch.float32, (N,))
    if bias is not None:
        _need(bias, "bias", torch.float16, (N,))
    if residual is not None:
        _need(residual, "residual", torch.float16, (M, N))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=q.device)
    _need(out, "out", torch.float16, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, N))
    need = w8a8_workspace_bytes(M, K, N)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().wql_w8a8_gemm_fused(_ptr(q), _ptr(xs), _ptr(qw), _ptr(ws), _ptr(bias), _ptr(residual), M, K, N,
                                      _ptr(out), _ptr(acc_out), _ptr(workspace), ws_bytes, _stream(q.device)),
           "wql_w8a8_gemm_fused")
    return out


def w8a8_gemm_noalloc(q: torch.Tensor, xs: torch.Tensor, qw: torch.Tensor, ws: torch.Tensor,
                      out: torch.Tensor, acc_out: torch.Tensor | None = None) -> torch.Tensor:
    """w8a8_gemm for callers that cannot allocate: the library uses its built-in scratch array.

    The caller passes every input and output (``out`` is required); the call itself allocates
    nothing.  Limits and sharing rules: see wql_w8a8_gemm_noalloc in include/wql.h.
    """
    M, K = q.shape
    N = qw.shape[0]
    _need(q, "q", torch.int8, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _need(qw, "qw", torch.int8, (N, K))
    _need(ws, "ws", torch.float32, (N,))
    _need(out, "out", torch.float16, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, N))
    _check(load().wql_w8a8_gemm_noalloc(_ptr(q), _ptr(xs), _ptr(qw), _ptr(ws), M, K, N, _ptr(out), _ptr(acc_out),
                                        _stream(q.device)), "wql_w8a8_gemm_noalloc")
    return out


def act_absmax(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    _need(gamma, "gamma", torch.float16, (K,))
    out = torch.empty((K,), dtype=torch.float32, device=x.device)
    _check(load().wql_act_absmax(_ptr(x), _ptr(gamma), float(eps), M, K, _ptr(out), _stream(x.device)),
           "wql_act_absmax")
    return out


def smooth(absmax: torch.Tensor, gamma: torch.Tensor, w: torch.Tensor):
    """Returns (s fp32 [K], gamma' fp16 [K], w' fp32 [K, N])."""
    K, N = w.shape
    _need(absmax, "absmax", torch.float32, (K,))
    _need(gamma, "gamma", torch.float16, (K,))
    _need(w, "w", torch.float32, (K, N))
    s = torch.empty((K,), dtype=torch.float32, device=w.device)
    g = torch.empty((K,), dtype=torch.float16, device=w.device)
    wo = torch.empty_like(w)
    _check(load().wql_smooth(_ptr(absmax), _ptr(gamma), _ptr(w), K, N, _ptr(s), _ptr(g), _ptr(wo), _stream(w.device)),
           "wql_smooth")
    return s, g, wo


def per_channel_quant_i8(w: torch.Tensor):
    """w [K, N] fp32 -> (qw int8 [N, K], ws fp32 [N])."""
    K, N = w.shape
    _need(w, "w", torch.float32, (K, N))
    qw = torch.empty((N, K), dtype=torch.int8, device=w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    _check(load().wql_per_channel_quant_i8(_ptr(w), K, N, _ptr(qw), _ptr(ws), _stream(w.device)),
           "wql_per_channel_quant_i8")
    return qw, ws


def device_status(device: torch.device | None = None) -> None:
    """Synchronise the current stream and raise if a kernel abandoned a bounded wait."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    _check(load().wql_device_status(_stream(dev)), "wql_device_status")


def diag_expire_wait(device: torch.device | None = None) -> None:
    """Launch the failure-path diagnostic: a bounded wait that gives up (about 2 s); the next
    device_status() then raises WQLError with WQL_ETIMEOUT."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    _check(load().wql_diag_expire_wait(_stream(dev)), "wql_diag_expire_wait")


# ---- fp8 (float8_e4m3fn) variant of W8A8 ------------------------------------------------------

E4M3 = torch.float8_e4m3fn


def qrmsnorm_quant_fp8(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, q: torch.Tensor | None = None,
                       xs: torch.Tensor | None = None):
    """QRMSNorm + per-token fp8: x [M, K] fp16 -> (q float8_e4m3fn [M, K], xs fp32 [M]), xs = absmax / 448."""
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    _need(gamma, "gamma", torch.float16, (K,))
    if q is None:
        q = torch.empty((M, K), dtype=E4M3, device=x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(q, "q", E4M3, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _check(load().wql_qrmsnorm_quant_fp8(_ptr(x), _ptr(gamma), float(eps), M, K, _ptr(q), _ptr(xs), _stream(x.device)),
           "wql_qrmsnorm_quant_fp8")
    return q, xs


def add_qrmsnorm_quant_fp8(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                           residual_out: torch.Tensor | None = None, q: torch.Tensor | None = None,
                           xs: torch.Tensor | None = None):
    """Residual-fused fp8 QRMSNorm: h = fp16(x + residual) -> (h, q float8_e4m3fn [M, K], xs fp32 [M]).

    residual_out receives h (it may be `residual` itself, for an in-place update)."""
    M, K = x.shape
    _need(x, "x", torch.float16, (M, K))
    _need(residual, "residual", torch.float16, (M, K))
    _need(gamma, "gamma", torch.float16, (K,))
    if residual_out is None:
        residual_out = torch.empty((M, K), dtype=torch.float16, device=x.device)
    if q is None:
        q = torch.empty((M, K), dtype=E4M3, device=x.device)
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(residual_out, "residual_out", torch.float16, (M, K))
    _need(q, "q", E4M3, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _check(load().wql_add_qrmsnorm_quant_fp8(_ptr(x), _ptr(residual), _ptr(gamma), float(eps), M, K,
                                             _ptr(residual_out), _ptr(q), _ptr(xs), _stream(x.device)),
           "wql_add_qrmsnorm_quant_fp8")
    return residual_out, q, xs


def per_channel_quant_fp8(w: torch.Tensor, qw: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """w [K, N] fp32 -> (qw float8_e4m3fn [N, K], ws fp32 [N]) with ws = absmax / 448."""
    K, N = w.shape
    _need(w, "w", torch.float32, (K, N))
    if qw is None:
        qw = torch.empty((N, K), dtype=E4M3, device=w.device)
    if ws is None:
        ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    _need(qw, "qw", E4M3, (N, K))
    _need(ws, "ws", torch.float32, (N,))
    _check(load().wql_per_channel_quant_fp8(_ptr(w), K, N, _ptr(qw), _ptr(ws), _stream(w.device)),
           "wql_per_channel_quant_fp8")
    return qw, ws


def w8a8_gemm_fp8(q: torch.Tensor, xs: torch.Tensor, qw: torch.Tensor, ws: torch.Tensor,
                  bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, acc_out: torch.Tensor | None = None) -> torch.Tensor:
    """y [M, N] fp16 = fp16(((acc * xs) * ws + bias) + residual), acc the fp32 sum of e4m3 products of
    q [M, K] and qw [N, K]; bias [N] and residual [M, N] fp16 optional; optional fp32 acc_out [M, N]."""
    M, K = q.shape
    N = qw.shape[0]
    _need(q, "q", E4M3, (M, K))
    _need(xs, "xs", torch.float32, (M,))
    _need(qw, "qw", E4M3, (N, K))
    _need(ws, "ws", torch.float32, (N,))
    if bias is not None:
        _need(bias, "bias", torch.float16, (N,))
    if residual is not None:
        _need(residual, "residual", torch.float16, (M, N))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=q.device)
    _need(out, "out", torch.float16, (M, N))
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.float32, (M, N))
    _check(load().wql_w8a8_gemm_fp8(_ptr(q), _ptr(xs), _ptr(qw), _ptr(ws), _ptr(bias), _ptr(residual), M, K, N,
                                    _ptr(out), _ptr(acc_out), _stream(q.device)), "wql_w8a8_gemm_fp8")
    return out


# ---- KV cache int8, groups of 128 channels ------------------------------------------------------

def kv_quant_i8(kv: torch.Tensor, q: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """kv [..., D] fp16 (D % 128 == 0) -> (q int8 [..., D], scales fp32 [..., D / 128]); s = absmax / 127."""
    D = kv.shape[-1]
    rows = kv.numel() // D if D else 0
    _need(kv, "kv", torch.float16, tuple(kv.shape))
    if q is None:
        q = torch.empty(kv.shape, dtype=torch.int8, device=kv.device)
    if scales is None:
        scales = torch.empty(tuple(kv.shape[:-1]) + (D // 128,), dtype=torch.float32, device=kv.device)
    _need(q, "q", torch.int8, tuple(kv.shape))
    _need(scales, "scales", torch.float32, tuple(kv.shape[:-1]) + (D // 128,))
    _check(load().wql_kv_quant_i8(_ptr(kv), rows, D, _ptr(q), _ptr(scales), _stream(kv.device)), "wql_kv_quant_i8")
    return q, scales


def kv_dequant_i8(q: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp16 [..., D] = fp16(q * the scale of the element's group of 128)."""
    D = q.shape[-1]
    rows = q.numel() // D if D else 0
    _need(q, "q", torch.int8, tuple(q.shape))
    _need(scales, "scales", torch.float32, tuple(q.shape[:-1]) + (D // 128,))
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    _need(out, "out", torch.float16, tuple(q.shape))
    _check(load().wql_kv_dequant_i8(_ptr(q), _ptr(scales), rows, D, _ptr(out), _stream(q.device)), "wql_kv_dequant_i8")
    return out


# ---- paged KV cache in 4 bits, and attention -----------------------------------------------------
#
# A decode step makes these calls once per layer on little data, so their checks are written to cost little: one test
# per tensor (_is), and the one that names what is wrong (_refuse) only when it fails.

def _is(t, dtype: torch.dtype, shape: tuple, index: int) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous())


def _refuse(t, name: str, dtype: torch.dtype, shape: tuple, index: int) -> None:
    _need(t, name, dtype, tuple(shape))
    raise ValueError(f"{name} is on {t.device}, expected device {index}")


def _stride_of(t, name: str, heads: int | None, dim: int | None, tokens: int | None, index: int | None) -> int:
    """Check an fp16 CUDA tensor [tokens, heads, D] whose rows [heads, D] are dense (a view of a fused projection's
    output); returns its token stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must have dtype {torch.float16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [tokens, heads, D], got {tuple(t.shape)}")
    T, H, D = t.shape
    if (heads is not None and H != heads) or (dim is not None and D != dim) or (tokens is not None and T != tokens):
        raise ValueError(f"{name} must have shape [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {'D' if dim is None else dim}], got {tuple(t.shape)}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected device {index}")
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name} must be dense within a token (strides [any, {D}, 1], got {(st, sh, sd)})")
    return st if T > 1 else H * D


def _cache_dims(cache: torch.Tensor):
    """(pages, heads, page size, D) of a 4-bit cache."""
    if not isinstance(cache, torch.Tensor):
        raise TypeError("cache must be a torch.Tensor")
    if cache.dim() != 4 or cache.shape[3] % 16 != 0:
        raise ValueError("cache must be [pages, heads, page_size / 16, 16 (D + 8)]; see kv_cache_i4")
    if not (cache.dtype == torch.uint8 and cache.is_cuda and cache.is_contiguous()):
        _need(cache, "cache", torch.uint8, tuple(cache.shape))
    pages, H, blocks, nbytes = cache.shape
    return pages, H, 16 * blocks, nbytes // 16 - 8


# the current stream's handle without a Stream object around it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(fn: str, index: int, *args) -> None:
    """Call fn(*args, stream) with device `index` current, on its current stream."""
    lib = _lib or load()
    if torch.cuda.current_device() == index:
        status = getattr(lib, fn)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = getattr(lib, fn)(*args, _raw_stream(index))
    if status != WQL_OK:
        _check(status, fn)


def kv_cache_i4(pages: int, heads: int, head_dim: int, page_size: int, device=None) -> torch.Tensor:
    """A zeroed 4-bit KV cache, uint8 [pages, heads, page_size / 16, 16 (head_dim + 8)]."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    if page_size < 16 or page_size % 16:
        raise ValueError("page_size must be a positive multiple of 16")
    return torch.zeros((pages, heads, page_size // 16, 16 * (head_dim + 8)), dtype=torch.uint8, device=device or "cuda")


def kv_plan_pages(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, page_size: int, tokens: int):
    """Block tables and slot maps on the GPU: gives every request the pages it lacks for its new tokens.

    ctx_lens, new_lens [B] int32 (tokens held, tokens added); block_table [B, width] int32, whose entries of new
    pages are written in place; free_pages [F] int32 with free_count [1] int32 of them free.  Returns (slots
    [tokens], cu_new [B + 1], kv_lens [B], free_count_out [1]), int32; slots behind the last new token and those of
    refused requests are -1, kv_lens of refused requests 0.  See wql_kv_plan_pages in include/wql.h."""
    i32, B, width, F = torch.int32, ctx_lens.shape[0], block_table.shape[-1], free_pages.shape[0]
    index = ctx_lens.get_device()
    if not (index >= 0 and _is(ctx_lens, i32, (B,), index) and _is(new_lens, i32, (B,), index)
            and _is(block_table, i32, (B, width), index) and _is(free_pages, i32, (F,), index)
            and _is(free_count, i32, (1,), index)):
        for t, name, shape in ((ctx_lens, "ctx_lens", (B,)), (new_lens, "new_lens", (B,)),
                               (block_table, "block_table", (B, width)), (free_pages, "free_pages", (F,)),
                               (free_count, "free_count", (1,))):
            if index < 0 or not _is(t, i32, shape, index):
                _refuse(t, name, i32, shape, index)
    # one allocation: slots first (its start is 16-byte aligned), then the small outputs
    out = torch.empty((tokens + 2 * B + 2,), dtype=i32, device=ctx_lens.device)
    slots, cu_new, kv_lens, left = torch.unsafe_split_with_sizes(out, (tokens, B + 1, B, 1))
    p = out.data_ptr()
    _run("wql_kv_plan_pages", index, ctx_lens.data_ptr(), new_lens.data_ptr(), B, page_size, free_pages.data_ptr(), F,
         free_count.data_ptr(), block_table.data_ptr(), width, tokens, p + 4 * tokens, p + 4 * (tokens + B + 1), p,
         p + 4 * (tokens + 2 * B + 1))
    return slots, cu_new, kv_lens, left


def kv_append_i4(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor) -> torch.Tensor:
    """Quantise rows k, v [T, heads, D] fp16 (views of a fused QKV output are taken as they are) into the 4-bit
    cache at slots [T] int32; negative slots are passed over.  Returns cache."""
    pages, H, ps, D = _cache_dims(cache)
    index = cache.get_device()
    ks = _stride_of(k, "k", H, D, None, index)
    T = k.shape[0]
    vs = _stride_of(v, "v", H, D, T, index)
    if not _is(slots, torch.int32, (T,), index):
        _refuse(slots, "slots", torch.int32, (T,), index)
    _run("wql_kv_append_i4", index, k.data_ptr(), v.data_ptr(), ks, vs, T, H, D, slots.data_ptr(), cache.data_ptr(), pages,
         ps)
    return cache


def kv_read_i4(cache: torch.Tensor, slots: torch.Tensor, k: torch.Tensor | None = None,
               v: torch.Tensor | None = None):
    """(k, v) [T, heads, D] fp16: the values of the 4-bit cache at slots [T] int32; zeros for negative slots."""
    pages, H, ps, D = _cache_dims(cache)
    dev, index, T, f16, shape = cache.device, cache.get_device(), slots.shape[0], torch.float16, (slots.shape[0], H, D)
    if not _is(slots, torch.int32, (T,), index):
        _refuse(slots, "slots", torch.int32, (T,), index)
    if k is None:
        k = torch.empty(shape, dtype=f16, device=dev)
    elif not _is(k, f16, shape, index):
        _refuse(k, "k", f16, shape, index)
    if v is None:
        v = torch.empty(shape, dtype=f16, device=dev)
    elif not _is(v, f16, shape, index):
        _refuse(v, "v", f16, shape, index)
    _run("wql_kv_read_i4", index, cache.data_ptr(), pages, ps, H, D, slots.data_ptr(), T, k.data_ptr(), v.data_ptr())
    return k, v


def attention_kv_i4_workspace_bytes(B: int, Lq: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load().wql_attention_kv_i4_workspace_bytes(B, Lq, Hq, Hkv, D))


def attention_kv_i4(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
                    scale: float | None = None, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the last tokens of each sequence over the paged 4-bit cache, grouped heads.

    q [B, Hq, D] (one token each) or [B, Lq, Hq, D] fp16, its tokens evenly strided; block_table [B, width] and
    kv_lens [B] int32, the queried tokens counted in.  Row r of Lq sees the tokens up to kv_lens - Lq + r; a row that
    sees none is zero.  scale defaults to D ** -0.5.  workspace: uint8, attention_kv_i4_workspace_bytes() of them,
    allocated here if not given.  Returns out, dense, of q's shape."""
    pages, Hkv, ps, D = _cache_dims(cache)
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be a tensor [B, Hq, D] or [B, Lq, Hq, D]")
    dev, index, shape = cache.device, cache.get_device(), q.shape
    B, Hq = shape[0], shape[-2]
    if len(shape) == 3:
        Lq, rows = 1, q
    else:
        Lq = shape[1]
        if B > 1 and Lq > 1 and q.stride(0) != Lq * q.stride(1):
            raise ValueError("the tokens of q must be evenly strided")
        rows = q[:, 0] if Lq == 1 else q.as_strided((B * Lq, Hq, shape[3]), q.stride()[1:])
    qs = _stride_of(rows, "q", None, D, None, index)
    width = block_table.shape[-1]
    if not _is(block_table, torch.int32, (B, width), index):
        _refuse(block_table, "block_table", torch.int32, (B, width), index)
    if not _is(kv_lens, torch.int32, (B,), index):
        _refuse(kv_lens, "kv_lens", torch.int32, (B,), index)
    if out is None:
        out = torch.empty(shape, dtype=torch.float16, device=dev)
    elif not _is(out, torch.float16, shape, index):
        _refuse(out, "out", torch.float16, shape, index)
    if workspace is None:
        with torch.cuda.device(dev):
            n = attention_kv_i4_workspace_bytes(B, Lq, Hq, Hkv, D)
        workspace = torch.empty((n,), dtype=torch.uint8, device=dev)
    elif not _is(workspace, torch.uint8, (workspace.numel(),), index):
        _refuse(workspace, "workspace", torch.uint8, (workspace.numel(),), index)
    _run("wql_attention_kv_i4", index, q.data_ptr(), qs, B, Lq, Hq, Hkv, D, cache.data_ptr(), pages, ps,
         block_table.data_ptr(), width, kv_lens.data_ptr(), D ** -0.5 if scale is None else scale, out.data_ptr(),
         workspace.data_ptr(), workspace.numel())
    return out


def attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     scale: float | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention over packed prompts, grouped heads: q [T, Hq, D], k and v [T, Hkv, D] fp16 (views of a fused
    QKV output are taken as they are), cu_seqlens [B + 1] int32.  scale defaults to D ** -0.5.  Returns out
    [T, Hq, D], dense; rows of no sequence are left as they were (undefined when out is not given)."""
    qs = _stride_of(q, "q", None, None, None, None)
    dev, index, shape = q.device, q.get_device(), q.shape
    T, Hq, D = shape
    ks = _stride_of(k, "k", None, D, T, index)
    Hkv = k.shape[1]
    vs = _stride_of(v, "v", Hkv, D, T, index)
    B = cu_seqlens.shape[0] - 1
    if not _is(cu_seqlens, torch.int32, (B + 1,), index):
        _refuse(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), index)
    if out is None:
        out = torch.empty(shape, dtype=torch.float16, device=dev)
    elif not _is(out, torch.float16, shape, index):
        _refuse(out, "out", torch.float16, shape, index)
    _run("wql_attention_prompt", index, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, Hq, Hkv, D,
         cu_seqlens.data_ptr(), B, D ** -0.5 if scale is None else scale, out.data_ptr())
    return out
