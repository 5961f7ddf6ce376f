"""Python binding of libdmpq, the gfx950 hot path of 6Bit-Diffusion's dynamic
mixed-precision quantized linear layer.

Argument marshalling only: each function passes torch tensors' device
pointers, sizes and the current HIP stream to the C entry point of the same
name (``dmpq_<name>``) and raises :class:`DmpqError` on a non-OK status.  All
arithmetic runs in the library's HIP kernels; there is no fallback.  Output
tensors are allocated by the caller, as the C ABI requires.
"""
from __future__ import annotations

import ctypes as C
import functools
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdmpq.so")

OK = 0
ROUTE_NVFP4, ROUTE_INT8, ROUTE_BF16 = 0, 1, 2
OUT_F32, OUT_BF16, OUT_I32 = 0, 1, 2
NO_HADAMARD, AMAX_GIVEN = 1, 2
EPI_GELU, EPI_NVFP4_AMAX = 1, 2
CODEC_E4M3, CODEC_E2M1 = 0, 1
W8_FROM_NVFP4, W8_DIRECT = 0, 1
TDC_SKIP, TDC_REFRESH = 0, 1
FP4_BF16_DEQUANT = 0
FP4_SCALED_MFMA = 1
OP_GAMMA, OP_QUANT_NVFP4, OP_TDC, OP_PREP_WEIGHT, OP_OUTLIER, OP_GEMM_AMAX, OP_GEMM = 0, 1, 2, 3, 4, 5, 6
OP_GEMM_W4 = 7
OP_GRAD_NORM = 8
ACT_NONE, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
ROPE_PAIRS, ROPE_HALVES = 0, 1

EXPORTS = ("dmpq_last_error", "dmpq_version", "dmpq_workspace_bytes", "dmpq_gamma_sums",
           "dmpq_gate_and_route", "dmpq_hadamard_quant_int8", "dmpq_hadamard_quant_nvfp4",
           "dmpq_qgemm_int8", "dmpq_qgemm_nvfp4", "dmpq_tdc_init", "dmpq_tdc_decide",
           "dmpq_tdc_step", "dmpq_tdc_commit", "dmpq_prep_weight", "dmpq_weight_int8_from_nvfp4",
           "dmpq_outlier_count", "dmpq_pdr_decide", "dmpq_gemm_bf16", "dmpq_qgemm_int8_ex",
           "dmpq_qgemm_nvfp4_ex", "dmpq_gemm_bf16_ex", "dmpq_selftest_codec",
           "dmpq_hadamard_quant_nvfp4_noalloc", "dmpq_qgemm_int8_from_nvfp4",
           "dmpq_hadamard_quant_int8_w8", "dmpq_lora_shrink", "dmpq_lora_forward",
           "dmpq_gemm_bf16_lora", "dmpq_qgemm_int8_lora", "dmpq_qgemm_nvfp4_lora",
           "dmpq_lora_backward_bytes", "dmpq_lora_backward", "dmpq_adamw_table_bytes",
           "dmpq_adamw_table", "dmpq_grad_norm", "dmpq_adamw_step", "dmpq_gemm_bf16_linear",
           "dmpq_qgemm_int8_linear", "dmpq_qgemm_nvfp4_linear", "dmpq_linear_backward_bytes",
           "dmpq_linear_epilogue_backward", "dmpq_rope_table", "dmpq_qk_norm_rope",
           "dmpq_qk_backward_bytes", "dmpq_qk_norm_rope_backward")


class DmpqError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn} -> status {status}: {msg}")
        self.status = status


class TdcState(C.Structure):
    """Mirror of dmpq_tdc_state."""
    _fields_ = [("n_refresh", C.c_int64), ("d", C.c_double), ("acc", C.c_double),
                ("delta_valid", C.c_int32), ("gamma_valid", C.c_int32), ("gamma", C.c_double)]


class AdamwTensor(C.Structure):
    """Mirror of dmpq_adamw_tensor."""
    _fields_ = [("p", C.c_void_p), ("g", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("ms", C.c_void_p), ("vs", C.c_void_p), ("copy", C.c_void_p), ("n", C.c_int64)]


class QkHeadsStruct(C.Structure):
    """Mirror of dmpq_qk_heads."""
    _fields_ = [("n_q", C.c_int32), ("n_k", C.c_int32), ("dim", C.c_int32), ("norm", C.c_int32),
                ("layout", C.c_int32), ("w_dtype", C.c_int32), ("rope_pairs", C.c_int32), ("eps", C.c_double),
                ("wq", C.c_void_p), ("bq", C.c_void_p), ("wk", C.c_void_p), ("bk", C.c_void_p),
                ("table", C.c_void_p)]


class LoraTermStruct(C.Structure):
    """Mirror of dmpq_lora_term."""
    _fields_ = [("t", C.c_void_p), ("b", C.c_void_p), ("rank", C.c_void_p), ("scale", C.c_void_p),
                ("seg_start", C.c_void_p), ("seg_adapter", C.c_void_p), ("R", C.c_int64), ("S", C.c_int64),
                ("n_adapters", C.c_int64)]


class LinearEpilogueStruct(C.Structure):
    """Mirror of dmpq_linear_epilogue."""
    _fields_ = [("bias", C.c_void_p), ("gate", C.c_void_p), ("residual", C.c_void_p), ("gate_start", C.c_void_p),
                ("pre", C.c_void_p), ("gate_rows", C.c_int64), ("bias_dtype", C.c_int32), ("gate_dtype", C.c_int32),
                ("act", C.c_int32), ("flags", C.c_int32), ("heads", C.POINTER(QkHeadsStruct)),
                ("lora", C.POINTER(LoraTermStruct))]


class TdcParams(C.Structure):
    """Mirror of dmpq_tdc_params."""
    _fields_ = [("eps_sim", C.c_double), ("delta_acc", C.c_double)]


_lib = None


def lib():
    """Load libdmpq.so (built in-tree by dynamic_mixed_precision_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run python -m "
                              "dynamic_mixed_precision_amd.build (needs hipcc)")
        _lib = _declare(C.CDLL(LIB_PATH))
    return _lib


def _declare(L):
    vp, i64, i32, f64 = C.c_void_p, C.c_int64, C.c_int, C.c_double
    pd = C.POINTER(C.c_double)
    sig = {
        "dmpq_last_error": (C.c_char_p, []),
        "dmpq_version": (C.c_char_p, []),
        "dmpq_workspace_bytes": (C.c_size_t, [i32, i64, i64]),
        "dmpq_gamma_sums": (i32, [vp, vp, vp, i64, vp, vp, C.c_size_t]),
        "dmpq_gate_and_route": (i32, [vp, i32, vp, vp, f64, vp, vp, vp]),
        "dmpq_hadamard_quant_int8": (i32, [vp, vp, i64, i64, i32, vp, vp]),
        "dmpq_hadamard_quant_nvfp4": (i32, [vp, vp, i64, i64, i32, vp, vp, vp, vp, C.c_size_t]),
        "dmpq_qgemm_int8": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]),
        "dmpq_qgemm_nvfp4": (i32, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32]),
        "dmpq_tdc_init": (i32, [C.POINTER(TdcState)]),
        "dmpq_tdc_decide": (i32, [C.POINTER(TdcState), C.POINTER(TdcParams), C.POINTER(C.c_int)]),
        "dmpq_tdc_step": (i32, [vp, i32, vp, vp, vp, i64, i32, vp, vp, C.c_size_t]),
        "dmpq_tdc_commit": (i32, [C.POINTER(TdcState), i32, pd]),
        "dmpq_prep_weight": (i32, [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, vp, C.c_size_t]),
        "dmpq_weight_int8_from_nvfp4": (i32, [vp, vp, vp, vp, i64, i64, vp, vp]),
        "dmpq_hadamard_quant_int8_w8": (i32, [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp, i64, vp, vp]),
        "dmpq_outlier_count": (i32, [vp, vp, i64, i64, f64, vp, vp, C.c_size_t]),
        "dmpq_pdr_decide": (i32, [f64, i64, f64, C.POINTER(C.c_int)]),
        "dmpq_gemm_bf16": (i32, [vp, vp, vp, i64, i64, i64, i32, vp]),
        "dmpq_qgemm_int8_ex": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, vp, C.c_size_t]),
        "dmpq_qgemm_nvfp4_ex": (i32, [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, vp,
                                      C.c_size_t]),
        "dmpq_gemm_bf16_ex": (i32, [vp, vp, vp, i64, i64, i64, i32, vp, i32, vp, C.c_size_t]),
        "dmpq_selftest_codec": (i32, [vp, i32, C.c_uint32, C.c_uint32, vp]),
        "dmpq_hadamard_quant_nvfp4_noalloc": (i32, [vp, vp, i64, i64, i32, vp, vp, vp]),
        "dmpq_qgemm_int8_from_nvfp4": (i32, [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, vp,
                                             C.c_size_t]),
        "dmpq_lora_shrink": (i32, [vp] * 6 + [i64] * 5 + [vp]),
        "dmpq_lora_forward": (i32, [vp] * 9 + [i64] * 6 + [i32, vp, vp]),
        "dmpq_gemm_bf16_lora": (i32, [vp] * 9 + [i64] * 6 + [i32, vp, i32, vp, C.c_size_t]),
        "dmpq_qgemm_int8_lora": (i32, [vp] * 11 + [i64] * 6 + [i32, vp, i32, vp, C.c_size_t]),
        "dmpq_qgemm_nvfp4_lora": (i32, [vp] * 13 + [i64] * 6 + [i32, vp, i32, vp, C.c_size_t]),
        "dmpq_lora_backward_bytes": (C.c_size_t, [i64] * 6),
        "dmpq_lora_backward": (i32, [vp] * 11 + [i64] * 6 + [vp, vp, vp, vp, C.c_size_t]),
        "dmpq_adamw_table_bytes": (C.c_size_t, [C.POINTER(AdamwTensor), i64]),
        "dmpq_adamw_table": (i32, [C.POINTER(AdamwTensor), i64, i32, i32, i32, vp, C.c_size_t,
                                   C.POINTER(C.c_int64)]),
        "dmpq_grad_norm": (i32, [vp, vp, i64, i64, i32, vp, vp, C.c_size_t]),
        "dmpq_adamw_step": (i32, [vp, vp, i64, i64, i32, i32, i32, f64, f64, f64, f64, f64, i64, vp, f64]),
        "dmpq_gemm_bf16_linear": (i32, [vp] * 3 + [i64] * 3 + [i32, vp, vp, vp, C.c_size_t]),
        "dmpq_qgemm_int8_linear": (i32, [vp] * 5 + [i64] * 3 + [i32, vp, vp, vp, C.c_size_t]),
        "dmpq_qgemm_nvfp4_linear": (i32, [vp] * 7 + [i64] * 3 + [i32, vp, vp, vp, C.c_size_t]),
        "dmpq_linear_backward_bytes": (C.c_size_t, [i64] * 3),
        "dmpq_linear_epilogue_backward": (i32, [vp, vp, vp, i64, i64, i32, i32, vp, i32, vp, i64] + [vp] * 4 +
                                          [C.c_size_t]),
        "dmpq_rope_table": (i32, [vp, vp, i32, vp, i64, i32, vp, vp]),
        "dmpq_qk_norm_rope": (i32, [vp, vp, i64, vp, i64, i64, i32, vp, vp, i64, vp, i64]),
        "dmpq_qk_backward_bytes": (C.c_size_t, [i32]),
        "dmpq_qk_norm_rope_backward": (i32, [vp] + [vp, i64] * 4 + [i64, i32, vp] + [vp, i64] * 2 + [vp] * 5 +
                                       [C.c_size_t]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def _check(status: int, fn: str) -> None:
    if status != OK:
        raise DmpqError(status, fn, lib().dmpq_last_error().decode())


_torch_c = None


def _stream(stream=None) -> int:
    """The stream's handle; None: the current stream of the current device (by
    torch's raw query: building a Stream object takes longer than a launch)."""
    global _torch_c
    if stream is not None:
        return stream.cuda_stream
    if _torch_c is None:
        import torch
        torch.cuda.current_stream()  # initializes CUDA, or says why it cannot
        _torch_c = torch._C
    return _torch_c._cuda_getCurrentRawStream(_torch_c._cuda_getDevice())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdmpq device arguments must be GPU tensors")
    if not t.is_contiguous():
        raise ValueError("libdmpq tensors must be contiguous")
    return t.data_ptr()


_OUT_BYTES = {OUT_F32: 4, OUT_BF16: 2, OUT_I32: 4}


def _need(t, name: str, nbytes: int, esize: int | None = None) -> None:
    """The C entry points take bare device pointers, so the sizes they will
    read and write are checked here: raise ValueError unless tensor ``t`` holds
    at least ``nbytes`` bytes (and, with ``esize``, has elements of that size)."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if esize is not None and t.element_size() != esize:
        raise ValueError(f"{name} has {t.element_size()}-byte elements, needs {esize}-byte ones")
    have = t.nbytes
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes, needs {nbytes}")


def _need_out(y, M: int, N: int, out_dtype: int) -> None:
    if out_dtype in _OUT_BYTES:  # an unknown type is the library's error to report
        _need(y, "y", M * N * _OUT_BYTES[out_dtype], _OUT_BYTES[out_dtype])


def _need_nvfp4(codes, scales, g, rows: int, K: int, what: str) -> None:
    """An NVFP4 operand of `rows` x K: K/2 code bytes and K/16 scale bytes per
    row, one fp32 tensor scale."""
    _need(codes, f"{what} codes", rows * K // 2, 1)
    _need(scales, f"{what} scales", rows * K // 16, 1)
    _need(g, f"{what} tensor scale", 4, 4)


def _need_k(w, K: int, what: str) -> None:
    if len(w.shape) != 2 or w.shape[1] != K:
        raise ValueError(f"{what} has shape {tuple(w.shape)}, needs {K} per row")


def last_error() -> str:
    return lib().dmpq_last_error().decode()


def version() -> str:
    return lib().dmpq_version().decode()


def workspace_bytes(op: int, M: int = 0, K: int = 0) -> int:
    return int(lib().dmpq_workspace_bytes(op, M, K))


def new_workspace(op: int, device="cuda", M: int = 0, K: int = 0):
    """Zero-filled workspace tensor for ``op`` (sizes M, K for OP_GEMM_AMAX)."""
    import torch
    return torch.zeros(workspace_bytes(op, M, K), dtype=torch.uint8, device=device)


def gamma_sums(x_in, x_out, sums, ws, stream=None) -> None:
    n = x_in.numel()
    _need(x_in, "x_in", 2 * n, 2)
    _need(x_out, "x_out", 2 * n, 2)
    _need(sums, "sums", 16, 8)
    _check(lib().dmpq_gamma_sums(_stream(stream), _ptr(x_in), _ptr(x_out), x_in.numel(),
                                 _ptr(sums), _ptr(ws), ws.numel()), "dmpq_gamma_sums")


def gate_and_route(sums2, alpha, beta, tau: float):
    """Host router.  sums2: 2 floats or None (Gamma missing).
    Returns (gamma, errors[n_lin], routes[n_lin]).  Runs between the step's
    device->host copy and its first launch, so it passes raw addresses (a
    ctypes pointer cast costs tens of microseconds)."""
    a = np.ascontiguousarray(alpha, np.float64)
    b = np.ascontiguousarray(beta, np.float64)
    n = len(a)
    s = None if sums2 is None else np.ascontiguousarray(sums2, np.float64)
    out = np.empty(1 + n, np.float64)  # gamma, then the errors
    r = np.empty(n, np.uint8)
    _check(lib().dmpq_gate_and_route(
        None if s is None else s.ctypes.data, n, a.ctypes.data, b.ctypes.data, tau,
        out.ctypes.data, out.ctypes.data + 8, r.ctypes.data), "dmpq_gate_and_route")
    return float(out[0]), out[1:], r


def hadamard_quant_int8(x, q, s_row, flags: int = 0, stream=None) -> None:
    M, K = x.shape
    _need(x, "x", 2 * M * K, 2)
    _need(q, "q", M * K, 1)
    _need(s_row, "s_row", 4 * M, 4)
    _check(lib().dmpq_hadamard_quant_int8(_stream(stream), _ptr(x), M, K, flags, _ptr(q),
                                          _ptr(s_row)), "dmpq_hadamard_quant_int8")


def hadamard_quant_nvfp4(x, codes, scales, g, ws, flags: int = 0, stream=None) -> None:
    M, K = x.shape
    _need(x, "x", 2 * M * K, 2)
    _need_nvfp4(codes, scales, g, M, K, "output")
    _check(lib().dmpq_hadamard_quant_nvfp4(_stream(stream), _ptr(x), M, K, flags, _ptr(codes),
                                           _ptr(scales), _ptr(g), _ptr(ws), ws.numel()),
           "dmpq_hadamard_quant_nvfp4")


def hadamard_quant_nvfp4_noalloc(x, codes, scales, g, flags: int = 0, stream=None) -> None:
    """hadamard_quant_nvfp4 without a workspace (the library's static scratch)."""
    M, K = x.shape
    _need(x, "x", 2 * M * K, 2)
    _need_nvfp4(codes, scales, g, M, K, "output")
    _check(lib().dmpq_hadamard_quant_nvfp4_noalloc(_stream(stream), _ptr(x), M, K, flags,
                                                   _ptr(codes), _ptr(scales), _ptr(g)),
           "dmpq_hadamard_quant_nvfp4_noalloc")


def _need_int8_gemm(qa, sa, qw, sw, y, out_dtype):
    M, K = qa.shape
    N = qw.shape[0]
    _need(qa, "qa", M * K, 1)
    _need(sa, "sa", 4 * M, 4)
    _need_k(qw, K, "qw")
    _need(qw, "qw", N * K, 1)
    _need(sw, "sw", 4 * N, 4)
    _need_out(y, M, N, out_dtype)
    return M, N, K


def _need_nvfp4_gemm(ca, sa, ga, cw, sw, gw, y, out_dtype):
    M, K = ca.shape[0], 2 * ca.shape[1]
    N = cw.shape[0]
    _need_nvfp4(ca, sa, ga, M, K, "activation")
    _need_k(cw, K // 2, "cw")
    _need_nvfp4(cw, sw, gw, N, K, "weight")
    _need_out(y, M, N, out_dtype)
    return M, N, K


def _need_bf16_gemm(x, w, y, out_dtype):
    M, K = x.shape
    N = w.shape[0]
    _need(x, "x", 2 * M * K, 2)
    _need_k(w, K, "w")
    _need(w, "w", 2 * N * K, 2)
    _need_out(y, M, N, out_dtype)
    return M, N, K


def qgemm_int8(qa, sa, qw, sw, y, out_dtype: int = OUT_F32, stream=None) -> None:
    M, N, K = _need_int8_gemm(qa, sa, qw, sw, y, out_dtype)
    _check(lib().dmpq_qgemm_int8(_stream(stream), _ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), M, N, K,
                                 out_dtype, _ptr(y)), "dmpq_qgemm_int8")


def qgemm_nvfp4(ca, sa, ga, cw, sw, gw, y, out_dtype: int = OUT_F32,
                variant: int = FP4_BF16_DEQUANT, stream=None) -> None:
    M, N, K = _need_nvfp4_gemm(ca, sa, ga, cw, sw, gw, y, out_dtype)
    _check(lib().dmpq_qgemm_nvfp4(_stream(stream), _ptr(ca), _ptr(sa), _ptr(ga), _ptr(cw),
                                  _ptr(sw), _ptr(gw), M, N, K, out_dtype, _ptr(y), variant),
           "dmpq_qgemm_nvfp4")


def tdc_init() -> TdcState:
    st = TdcState()
    _check(lib().dmpq_tdc_init(C.byref(st)), "dmpq_tdc_init")
    return st


def tdc_decide(st: TdcState, eps_sim: float, delta_acc: float) -> bool:
    p = TdcParams(eps_sim, delta_acc)
    out = C.c_int(0)
    _check(lib().dmpq_tdc_decide(C.byref(st), C.byref(p), C.byref(out)), "dmpq_tdc_decide")
    return bool(out.value)


def tdc_step(mode: int, x_in, x_out, delta, delta_valid: bool, sums=None, ws=None,
             stream=None) -> None:
    n = x_in.numel()
    for t, name in ((x_in, "x_in"), (x_out, "x_out"), (delta, "delta")):
        _need(t, name, 2 * n, 2)
    if mode == TDC_REFRESH:
        _need(sums, "sums", 32, 8)
    _check(lib().dmpq_tdc_step(_stream(stream), mode, _ptr(x_in), _ptr(x_out), _ptr(delta),
                               x_in.numel(), int(delta_valid), _ptr(sums), _ptr(ws),
                               0 if ws is None else ws.numel()), "dmpq_tdc_step")


def tdc_commit(st: TdcState, mode: int, sums4=None) -> None:
    s = None if sums4 is None else np.ascontiguousarray(sums4, np.float64)
    _check(lib().dmpq_tdc_commit(C.byref(st), mode,
                                 None if s is None else s.ctypes.data_as(C.POINTER(C.c_double))),
           "dmpq_tdc_commit")


def prep_weight(w, cw, sw, gw, qw, sw_row, ws, int8_mode: int = W8_FROM_NVFP4,
                stream=None) -> None:
    N, K = w.shape
    _need(w, "w", 2 * N * K, 2)
    _need_nvfp4(cw, sw, gw, N, K, "weight")
    _need(qw, "qw", N * K, 1)
    _need(sw_row, "sw_row", 4 * N, 4)
    _check(lib().dmpq_prep_weight(_stream(stream), _ptr(w), N, K, int8_mode, _ptr(cw), _ptr(sw),
                                  _ptr(gw), _ptr(qw), _ptr(sw_row), _ptr(ws), ws.numel()),
           "dmpq_prep_weight")


def weight_int8_from_nvfp4(cw, sw, gw, qw, sw_row, stream=None) -> None:
    """INT8 weight (qw, sw_row) from the NVFP4 weight (cw, sw, gw)."""
    N, K = cw.shape[0], 2 * cw.shape[1]
    _need_nvfp4(cw, sw, gw, N, K, "weight")
    _need(qw, "qw", N * K, 1)
    _need(sw_row, "sw_row", 4 * N, 4)
    _check(lib().dmpq_weight_int8_from_nvfp4(_stream(stream), _ptr(cw), _ptr(sw), _ptr(gw), N, K,
                                             _ptr(qw), _ptr(sw_row)), "dmpq_weight_int8_from_nvfp4")


def hadamard_quant_int8_w8(x, q, s_row, cw, sw, gw, qw, sw_row, flags: int = 0, stream=None) -> None:
    """hadamard_quant_int8(x, q, s_row) and weight_int8_from_nvfp4(cw, sw, gw,
    qw, sw_row) in one launch (x and the weight share K)."""
    M, K = x.shape
    N = cw.shape[0]
    _need(x, "x", 2 * M * K, 2)
    _need(q, "q", M * K, 1)
    _need(s_row, "s_row", 4 * M, 4)
    _need_k(cw, K // 2, "cw")
    _need_nvfp4(cw, sw, gw, N, K, "weight")
    _need(qw, "qw", N * K, 1)
    _need(sw_row, "sw_row", 4 * N, 4)
    _check(lib().dmpq_hadamard_quant_int8_w8(_stream(stream), _ptr(x), M, K, flags, _ptr(q), _ptr(s_row),
                                             _ptr(cw), _ptr(sw), _ptr(gw), N, _ptr(qw), _ptr(sw_row)),
           "dmpq_hadamard_quant_int8_w8")


def qgemm_int8_from_nvfp4(qa, sa, cw, sw, gw, y, ws, epilogue: int = 0, out_dtype: int = OUT_BF16,
                          stream=None) -> None:
    """INT8 linear against the NVFP4 weight (cw, sw, gw), converted inside the
    GEMM; ws: an OP_GEMM_W4 workspace for (M, N)."""
    M, K = qa.shape
    N = cw.shape[0]
    _need(qa, "qa", M * K, 1)
    _need(sa, "sa", 4 * M, 4)
    _need_k(cw, K // 2, "cw")
    _need_nvfp4(cw, sw, gw, N, K, "weight")
    _need_out(y, M, N, out_dtype)
    _check(lib().dmpq_qgemm_int8_from_nvfp4(_stream(stream), _ptr(qa), _ptr(sa), _ptr(cw), _ptr(sw),
                                            _ptr(gw), M, N, K, out_dtype, _ptr(y), epilogue, *_ws(ws)),
           "dmpq_qgemm_int8_from_nvfp4")


def outlier_count(x, kappa: float, count, ws, stream=None) -> None:
    """PDR outlier count of x [M x K] bf16 (as int16 bits) into count (fp64[1])."""
    M, K = x.shape
    _need(x, "x", 2 * M * K, 2)
    _need(count, "count", 8, 8)
    _check(lib().dmpq_outlier_count(_stream(stream), _ptr(x), M, K, float(kappa), _ptr(count),
                                    _ptr(ws), ws.numel()), "dmpq_outlier_count")


def pdr_decide(count: float, n: int, rho: float) -> bool:
    force = C.c_int(0)
    _check(lib().dmpq_pdr_decide(float(count), int(n), float(rho), C.byref(force)), "dmpq_pdr_decide")
    return bool(force.value)


def gemm_bf16(x, w, y, out_dtype: int = OUT_F32, stream=None) -> None:
    """Full-precision linear y = x w^T over bf16 operands (fp32 accumulation)."""
    M, N, K = _need_bf16_gemm(x, w, y, out_dtype)
    _check(lib().dmpq_gemm_bf16(_stream(stream), _ptr(x), _ptr(w), M, N, K, out_dtype, _ptr(y)),
           "dmpq_gemm_bf16")


def _ws(ws):
    return (None, 0) if ws is None else (_ptr(ws), ws.numel())


def qgemm_int8_ex(qa, sa, qw, sw, y, epilogue: int = 0, ws=None, out_dtype: int = OUT_BF16,
                  stream=None) -> None:
    """qgemm_int8 with a producer epilogue (EPI_GELU, EPI_NVFP4_AMAX); with an
    OP_GEMM workspace the last partial wave of tiles is split along K."""
    M, N, K = _need_int8_gemm(qa, sa, qw, sw, y, out_dtype)
    _check(lib().dmpq_qgemm_int8_ex(_stream(stream), _ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), M, N,
                                    K, out_dtype, _ptr(y), epilogue, *_ws(ws)),
           "dmpq_qgemm_int8_ex")


def qgemm_nvfp4_ex(ca, sa, ga, cw, sw, gw, y, epilogue: int = 0, ws=None, out_dtype: int = OUT_BF16,
                   stream=None) -> None:
    """qgemm_nvfp4 (BF16-dequant variant) with a producer epilogue and the
    optional tail split."""
    M, N, K = _need_nvfp4_gemm(ca, sa, ga, cw, sw, gw, y, out_dtype)
    _check(lib().dmpq_qgemm_nvfp4_ex(_stream(stream), _ptr(ca), _ptr(sa), _ptr(ga), _ptr(cw),
                                     _ptr(sw), _ptr(gw), M, N, K, out_dtype, _ptr(y), epilogue,
                                     *_ws(ws)),
           "dmpq_qgemm_nvfp4_ex")


def gemm_bf16_ex(x, w, y, epilogue: int = 0, ws=None, out_dtype: int = OUT_BF16,
                 stream=None) -> None:
    """gemm_bf16 with a producer epilogue and the optional tail split."""
    M, N, K = _need_bf16_gemm(x, w, y, out_dtype)
    _check(lib().dmpq_gemm_bf16_ex(_stream(stream), _ptr(x), _ptr(w), M, N, K, out_dtype, _ptr(y),
                                   epilogue, *_ws(ws)),
           "dmpq_gemm_bf16_ex")


def selftest_codec(codec: int, lo: int, hi: int, stats, stream=None) -> None:
    """Per-code (lowest, highest, count) of the fp32 patterns [lo, hi) through
    a device converter (CODEC_E4M3 or CODEC_E2M1); stats: uint32/int32 tensor
    of 3 words per code (128 codes for E4M3, 16 for E2M1)."""
    if codec in (CODEC_E4M3, CODEC_E2M1):  # an unknown codec is the library's error to report
        _need(stats, "stats", 12 * (128 if codec == CODEC_E4M3 else 16), 4)
    _check(lib().dmpq_selftest_codec(_stream(stream), codec, lo, hi, _ptr(stats)),
           "dmpq_selftest_codec")


# ---- low-rank adapters beside a linear ----------------------------------------

_types = None


def _load_types():
    """Per kind of operand the tensor types that hold it: bf16 also as its bits,
    8-bit codes also as bytes."""
    global _types
    import torch
    _types = {"fp32": frozenset((torch.float32,)), "fp64": frozenset((torch.float64,)), "int32": frozenset((torch.int32,)),
              "bf16": frozenset((torch.bfloat16, torch.int16, torch.uint16)),
              "E4M3": frozenset((torch.float8_e4m3fn, torch.uint8, torch.int8))}
    return _types


def _need_type(t, name: str, nbytes: int, kind: str) -> None:
    """As _need, and by type instead of element size: fp16 has bf16's size, and
    fp32 has int32's."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype not in (_types or _load_types())[kind]:
        raise ValueError(f"{name} is {t.dtype}, needs {kind}")
    have = t.nbytes
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes, needs {nbytes}")


def _need_lora_out(y, name: str, M: int, N: int, out_dtype: int) -> None:
    if out_dtype == OUT_BF16:
        _need_type(y, name, 2 * M * N, "bf16")
    elif out_dtype == OUT_F32:  # any other type is the library's error to report
        _need_type(y, name, 4 * M * N, "fp32")

def _need_lora(x_rows: int, a, b, rank, scale, seg_start, seg_adapter, t, K=None, N=None):
    """The pool and batch that every adapter call shares; returns (R, S, n)."""
    n, R = _pool_shape(a if a is not None else b, a is not None)
    if a is not None:
        if a.shape != (n, R, K):
            raise ValueError(f"a has shape {tuple(a.shape)}, needs {(n, R, K)}")
        _need_type(a, "a", 2 * n * R * K, "bf16")
    if b is not None:
        if b.shape != (n, N, R):
            raise ValueError(f"b has shape {tuple(b.shape)}, needs {(n, N, R)}")
        _need_type(b, "b", 2 * n * N * R, "bf16")
    _need_type(rank, "rank", 4 * n, "int32")
    if scale is not None:
        _need_type(scale, "scale", 4 * n, "fp32")
    S = seg_start.numel() - 1
    if S < 0:
        raise ValueError("seg_start needs at least one entry")
    _need_type(seg_start, "seg_start", 4 * (S + 1), "int32")
    _need_type(seg_adapter, "seg_adapter", 4 * S, "int32")
    _need_type(t, "t", 4 * x_rows * R, "fp32")
    return R, S, n


def _pool_shape(pool, is_a: bool):
    shape = pool.shape
    if len(shape) != 3:
        raise ValueError(f"the adapter pool has shape {tuple(shape)}, needs 3 dimensions")
    return shape[0], shape[1 if is_a else 2]


def new_lora_workspace(M: int, N: int, K: int, R: int, S: int, n_adapters: int, device="cuda"):
    """Workspace tensor for lora_backward."""
    import torch
    return torch.empty(int(lib().dmpq_lora_backward_bytes(M, N, K, R, S, n_adapters)), dtype=torch.uint8,
                       device=device)


def lora_shrink(x, a, rank, seg_start, seg_adapter, t, stream=None) -> None:
    """t [M, R] fp32 = x a^T, each row through the adapter of its request."""
    M, K = x.shape
    _need_type(x, "x", 2 * M * K, "bf16")
    R, S, n = _need_lora(M, a, None, rank, None, seg_start, seg_adapter, t, K=K)
    _check(lib().dmpq_lora_shrink(_stream(stream), _ptr(x), _ptr(a), _ptr(rank), _ptr(seg_start),
                                  _ptr(seg_adapter), M, K, R, S, n, _ptr(t)), "dmpq_lora_shrink")


def lora_forward(x, base, a, b, rank, scale, seg_start, seg_adapter, t, y, out_dtype: int = OUT_BF16,
                 stream=None) -> None:
    """t as lora_shrink, and y = base + scale * t b^T (base may be y, or None for zeros)."""
    M, K = x.shape
    N = b.shape[1]
    _need_type(x, "x", 2 * M * K, "bf16")
    R, S, n = _need_lora(M, a, b, rank, scale, seg_start, seg_adapter, t, K=K, N=N)
    _need_lora_out(y, "y", M, N, out_dtype)
    if base is not None:
        _need_lora_out(base, "base", M, N, out_dtype)
    _check(lib().dmpq_lora_forward(_stream(stream), _ptr(x), _ptr(base), _ptr(a), _ptr(b), _ptr(rank),
                                   _ptr(scale), _ptr(seg_start), _ptr(seg_adapter), M, N, K, R, S, n,
                                   out_dtype, _ptr(t), _ptr(y)), "dmpq_lora_forward")


def gemm_bf16_lora(x, w, t, b, rank, scale, seg_start, seg_adapter, y, epilogue: int = 0, ws=None,
                   out_dtype: int = OUT_BF16, stream=None) -> None:
    """gemm_bf16_ex with the adapters' scale * t b^T added in its epilogue."""
    M, N, K = _need_bf16_gemm(x, w, y, out_dtype)
    _need_type(x, "x", 0, "bf16")
    _need_type(w, "w", 0, "bf16")
    _need_lora_out(y, "y", M, N, out_dtype)
    R, S, n = _need_lora(M, None, b, rank, scale, seg_start, seg_adapter, t, N=N)
    _check(lib().dmpq_gemm_bf16_lora(_stream(stream), _ptr(x), _ptr(w), _ptr(t), _ptr(b), _ptr(rank),
                                     _ptr(scale), _ptr(seg_start), _ptr(seg_adapter), M, N, K, R, S, n,
                                     out_dtype, _ptr(y), epilogue, *_ws(ws)), "dmpq_gemm_bf16_lora")


def qgemm_int8_lora(qa, sa, qw, sw, t, b, rank, scale, seg_start, seg_adapter, y, epilogue: int = 0,
                    ws=None, out_dtype: int = OUT_BF16, stream=None) -> None:
    """qgemm_int8_ex with the adapters' scale * t b^T added in its epilogue."""
    M, N, K = _need_int8_gemm(qa, sa, qw, sw, y, out_dtype)
    _need_lora_out(y, "y", M, N, out_dtype)
    R, S, n = _need_lora(M, None, b, rank, scale, seg_start, seg_adapter, t, N=N)
    _check(lib().dmpq_qgemm_int8_lora(_stream(stream), _ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), _ptr(t),
                                      _ptr(b), _ptr(rank), _ptr(scale), _ptr(seg_start), _ptr(seg_adapter),
                                      M, N, K, R, S, n, out_dtype, _ptr(y), epilogue, *_ws(ws)),
           "dmpq_qgemm_int8_lora")


def qgemm_nvfp4_lora(ca, sa, ga, cw, sw, gw, t, b, rank, scale, seg_start, seg_adapter, y,
                     epilogue: int = 0, ws=None, out_dtype: int = OUT_BF16, stream=None) -> None:
    """qgemm_nvfp4_ex with the adapters' scale * t b^T added in its epilogue."""
    M, N, K = _need_nvfp4_gemm(ca, sa, ga, cw, sw, gw, y, out_dtype)
    _need_lora_out(y, "y", M, N, out_dtype)
    R, S, n = _need_lora(M, None, b, rank, scale, seg_start, seg_adapter, t, N=N)
    _check(lib().dmpq_qgemm_nvfp4_lora(_stream(stream), _ptr(ca), _ptr(sa), _ptr(ga), _ptr(cw), _ptr(sw),
                                       _ptr(gw), _ptr(t), _ptr(b), _ptr(rank), _ptr(scale),
                                       _ptr(seg_start), _ptr(seg_adapter), M, N, K, R, S, n, out_dtype,
                                       _ptr(y), epilogue, *_ws(ws)), "dmpq_qgemm_nvfp4_lora")


def lora_backward(dy, x, t, a, b, rank, scale, seg_start, seg_adapter, dx_base, dx, da, db, ws,
                  stream=None) -> None:
    """dx = dx_base + scale dy b a, da [n, R, K] and db [n, N, R] fp32 (dx_base
    may be dx, or None for zeros; dx None: not computed)."""
    M, K = x.shape
    N = b.shape[1]
    _need_type(x, "x", 2 * M * K, "bf16")
    _need_type(dy, "dy", 2 * M * N, "bf16")
    R, S, n = _need_lora(M, a, b, rank, scale, seg_start, seg_adapter, t, K=K, N=N)
    for g, name in ((dx_base, "dx_base"), (dx, "dx")):
        if g is not None:
            _need_type(g, name, 2 * M * K, "bf16")
    _need_type(da, "da", 4 * n * R * K, "fp32")
    _need_type(db, "db", 4 * n * N * R, "fp32")
    _check(lib().dmpq_lora_backward(_stream(stream), _ptr(dy), _ptr(x), _ptr(t), _ptr(a), _ptr(b),
                                    _ptr(rank), _ptr(scale), _ptr(seg_start), _ptr(seg_adapter),
                                    _ptr(dx_base), M, N, K, R, S, n, _ptr(dx), _ptr(da), _ptr(db),
                                    *_ws(ws)), "dmpq_lora_backward")


# ---- AdamW over many tensors ----------------------------------------------------

class AdamwTable:
    """The places of the tensors that one adamw_step call updates.  Holds the
    tensors themselves, whatever becomes of the lists they came in: their memory
    must not move while the table is used."""

    def __init__(self, table, n: int, chunks: int, p_dtype: int, g_dtype: int, bits: int, keep):
        self.table, self.n, self.chunks = table, n, chunks
        self.p_dtype, self.g_dtype, self.bits = p_dtype, g_dtype, bits
        self._keep = keep


def adamw_table(params, grads, m, v, m_scales=None, v_scales=None, copies=None) -> AdamwTable:
    """Table of the given lists of tensors, one entry each: params and grads
    fp32 or bf16 (one type per list), states m and v fp32, or 8-bit codes with
    m_scales and v_scales (fp32, one per 256 values); copies: bf16 copies of
    the new params, or None."""
    import torch
    k = len(params)
    eight = m_scales is not None
    lists = [params, grads, m, v, m_scales if eight else [None] * k, v_scales if eight else [None] * k,
             copies if copies is not None else [None] * k]
    if any(x is None or len(x) != k for x in lists):
        raise ValueError("adamw_table needs lists of the same length")
    p_dtype, g_dtype = _one_type(params, "params"), _one_type(grads, "grads")
    rows = (AdamwTensor * max(1, k))()
    for i, (p, g, mi, vi, ms, vs, c) in enumerate(zip(*lists)):
        n = p.numel()
        blocks = (n + 255) // 256
        _need(g, "grad", n * g.element_size())
        for s, name in ((mi, "m"), (vi, "v")):
            _need_type(s, name, n * (1 if eight else 4), "E4M3" if eight else "fp32")
        if eight:
            _need_type(ms, "m_scales", 4 * blocks, "fp32")
            _need_type(vs, "v_scales", 4 * blocks, "fp32")
        if c is not None:
            _need_type(c, "copy", 2 * n, "bf16")
        for f, q in (("p", p), ("g", g), ("m", mi), ("v", vi), ("ms", ms), ("vs", vs), ("copy", c)):
            setattr(rows[i], f, _ptr(q))
        rows[i].n = n
    nbytes = int(lib().dmpq_adamw_table_bytes(rows, k))
    host = torch.empty(max(nbytes, 16), dtype=torch.uint8)
    chunks = C.c_int64(0)
    bits = 8 if eight else 32
    _check(lib().dmpq_adamw_table(rows, k, p_dtype, g_dtype, bits, host.data_ptr(), nbytes,
                                  C.byref(chunks)), "dmpq_adamw_table")
    device = params[0].device if k else "cuda"
    return AdamwTable(host.to(device), k, chunks.value, p_dtype, g_dtype, bits, [tuple(x) for x in lists])


def _one_type(ts, name: str) -> int:
    kinds = {t.dtype for t in ts}
    for out, kind in ((OUT_F32, "fp32"), (OUT_BF16, "bf16")):
        if kinds <= (_types or _load_types())[kind]:
            return out
    raise ValueError(f"{name} must all be fp32 or all bf16")


def grad_norm(table: AdamwTable, norm, ws, stream=None) -> None:
    """norm (fp64[1]) = the L2 norm of all gradients of the table."""
    _need(norm, "norm", 8, 8)
    _check(lib().dmpq_grad_norm(_stream(stream), _ptr(table.table), table.n, table.chunks, table.g_dtype,
                                _ptr(norm), *_ws(ws)), "dmpq_grad_norm")


def adamw_step(table: AdamwTable, lr: float, beta1: float = 0.9, beta2: float = 0.999,
               eps: float = 1e-8, weight_decay: float = 0.01, step: int = 1, norm=None,
               max_norm: float = 0.0, stream=None) -> None:
    """One AdamW step of every tensor of the table, in place.  norm: the
    gradients' norm from grad_norm, for clipping to max_norm (> 0) and for
    leaving out a step whose norm is not finite."""
    if norm is not None:
        _need(norm, "norm", 8, 8)
    _check(lib().dmpq_adamw_step(_stream(stream), _ptr(table.table), table.n, table.chunks, table.p_dtype,
                                 table.g_dtype, table.bits, lr, beta1, beta2, eps, weight_decay, int(step),
                                 _ptr(norm), max_norm), "dmpq_adamw_step")


# ---- the whole linear -----------------------------------------------------------

def _float_type(t, name: str) -> int:
    """OUT_F32 or OUT_BF16 of an fp32 or bf16 tensor."""
    kinds = _types or _load_types()
    if t.dtype in kinds["fp32"]:
        return OUT_F32
    if t.dtype in kinds["bf16"]:
        return OUT_BF16
    raise ValueError(f"{name} is {t.dtype}, needs fp32 or bf16")


_KIND = {OUT_F32: ("fp32", 4), OUT_BF16: ("bf16", 2)}


class QkHeads:
    """The heads of q and k (qk_heads).  Holds its tensors."""

    def __init__(self, struct, n_q: int, n_k: int, dim: int, norm: int, table, keep):
        self.struct, self.n_q, self.n_k, self.dim, self.norm, self.table = struct, n_q, n_k, dim, norm, table
        self._keep = keep


def qk_heads(n_q: int, n_k: int, dim: int, norm: int = NORM_NONE, eps: float = 1e-6, wq=None, bq=None, wk=None,
             bk=None, table=None, layout: int = ROPE_PAIRS) -> QkHeads:
    """n_q heads of q and n_k of k of `dim` values: their norm with weights w and
    b [dim] (fp32 or bf16, one type; None: 1 and 0) and, with the `table`
    [rows, pairs, 2] of rope_table, the rotation.  The object can be kept: it
    holds the tensors, which must not move."""
    keep = (wq, bq, wk, bk, table)
    kinds = set()
    for w, name in ((wq, "wq"), (bq, "bq"), (wk, "wk"), (bk, "bk")):
        if w is not None:
            kinds.add(_float_type(w, name))
            _need(w, name, dim * w.element_size())
    if len(kinds) > 1:
        raise ValueError("wq, bq, wk and bk must all be fp32 or all bf16")
    pairs = 0
    if table is not None:
        if table.dim() != 3 or table.shape[2] != 2:
            raise ValueError(f"table has shape {tuple(table.shape)}, needs (rows, pairs, 2)")
        _need_type(table, "table", 0, "fp32")
        pairs = table.shape[1]
    st = QkHeadsStruct(n_q, n_k, dim, norm, layout, kinds.pop() if kinds else OUT_F32, pairs, eps, _ptr(wq),
                       _ptr(bq), _ptr(wk), _ptr(bk), _ptr(table))
    return QkHeads(st, n_q, n_k, dim, norm, table, keep)


def _need_table(heads: QkHeads, M: int) -> None:
    if heads.table is not None and heads.table.shape[0] < M:
        raise ValueError(f"table has {heads.table.shape[0]} rows, needs {M}")


class LinearEpilogue:
    """What follows the product of a *_linear GEMM (linear_epilogue).  Holds its
    tensors."""

    def __init__(self, struct, bias, gate, gate_start, residual, pre, heads, adapters, keep):
        self.struct, self.bias, self.gate, self.gate_start = struct, bias, gate, gate_start
        self.residual, self.pre, self.heads, self.adapters = residual, pre, heads, adapters
        self._keep = keep
        self._checked = None


def linear_epilogue(bias=None, act: int = ACT_NONE, gate=None, gate_start=None, residual=None, pre=None, heads=None,
                    adapters=None, amax: bool = False) -> LinearEpilogue:
    """y = residual + gate[request of the row] * act(x w^T + adapters + bias).

    bias [N] and gate [S, N]: fp32 or bf16; gate_start int32 [S + 1]: the rows'
    requests (None: the gate's one row is for all; S = 0: no row has one);
    residual and pre [M, N] of y's type, pre receiving the value before heads and
    act; heads: a QkHeads, for a QKV linear; adapters: (t, b, rank, scale, seg_start, seg_adapter) as
    the *_lora GEMMs take them; amax: leave the NVFP4 amax of y in the workspace
    (EPI_NVFP4_AMAX).  The object can be kept for further calls of the same
    shapes: it holds the tensors, which must not move."""
    rows = 0
    bias_type = OUT_F32 if bias is None else _float_type(bias, "bias")
    gate_type = OUT_F32 if gate is None else _float_type(gate, "gate")
    if gate is not None:
        if gate.dim() != 2:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, needs (requests, N)")
        rows = _gate_rows(gate, gate_start)
    elif gate_start is not None:
        raise ValueError("gate is missing")
    lora = None
    if adapters is not None:
        t, b, rank, scale, seg_start, seg_adapter = adapters
        R, S, n = _need_lora(0, None, b, rank, scale, seg_start, seg_adapter, t, N=_pool_n(b))
        lora = LoraTermStruct(_ptr(t), _ptr(b), _ptr(rank), _ptr(scale), _ptr(seg_start), _ptr(seg_adapter), R, S, n)
    st = LinearEpilogueStruct(
        _ptr(bias), _ptr(gate), _ptr(residual), _ptr(gate_start), _ptr(pre), rows, bias_type, gate_type, act,
        EPI_NVFP4_AMAX if amax else 0, None if heads is None else C.pointer(heads.struct),
        None if lora is None else C.pointer(lora))
    return LinearEpilogue(st, bias, gate, gate_start, residual, pre, heads, adapters, lora)


def _gate_rows(gate, gate_start) -> int:
    rows = gate.shape[0]
    if gate_start is not None:
        _need_type(gate_start, "gate_start", 4 * (rows + 1), "int32")
    elif rows == 0:  # an empty tensor has no address: the library would see no gate
        raise ValueError("a gate of 0 rows needs gate_start")
    return rows


def _pool_n(b) -> int:
    if b.dim() != 3:
        raise ValueError(f"the adapter pool has shape {tuple(b.shape)}, needs 3 dimensions")
    return b.shape[1]


def _need_linear(epi: LinearEpilogue, y, M: int, N: int, out_dtype: int):
    _need_lora_out(y, "y", M, N, out_dtype)
    if epi._checked != (M, N, out_dtype):  # an epilogue that is kept is looked over once per shape
        if epi.bias is not None:
            _need(epi.bias, "bias", N * epi.bias.element_size())
        if epi.gate is not None and epi.gate.shape[1] != N:
            raise ValueError(f"gate has shape {tuple(epi.gate.shape)}, needs {N} columns")
        for t, name in ((epi.residual, "residual"), (epi.pre, "pre")):
            if t is not None:
                _need_lora_out(t, name, M, N, out_dtype)
        if epi.heads is not None:
            _need_table(epi.heads, M)
        if epi.adapters is not None:
            t, b, rank, scale, seg_start, seg_adapter = epi.adapters
            _need_lora(M, None, b, rank, scale, seg_start, seg_adapter, t, N=N)
        epi._checked = (M, N, out_dtype)
    return C.addressof(epi.struct)


def gemm_bf16_linear(x, w, y, epilogue: LinearEpilogue, ws=None, out_dtype: int = OUT_BF16, stream=None) -> None:
    """The BF16 linear x w^T with the whole epilogue; ws: an OP_GEMM workspace
    (None: no tail split; needed for amax)."""
    M, N, K = _need_bf16_gemm(x, w, y, out_dtype)
    _need_type(x, "x", 0, "bf16")
    _need_type(w, "w", 0, "bf16")
    e = _need_linear(epilogue, y, M, N, out_dtype)
    _check(lib().dmpq_gemm_bf16_linear(_stream(stream), _ptr(x), _ptr(w), M, N, K, out_dtype, _ptr(y), e, *_ws(ws)),
           "dmpq_gemm_bf16_linear")


def qgemm_int8_linear(qa, sa, qw, sw, y, epilogue: LinearEpilogue, ws=None, out_dtype: int = OUT_BF16,
                      stream=None) -> None:
    """The INT8 linear with the whole epilogue."""
    M, N, K = _need_int8_gemm(qa, sa, qw, sw, y, out_dtype)
    e = _need_linear(epilogue, y, M, N, out_dtype)
    _check(lib().dmpq_qgemm_int8_linear(_stream(stream), _ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), M, N, K, out_dtype,
                                        _ptr(y), e, *_ws(ws)), "dmpq_qgemm_int8_linear")


def qgemm_nvfp4_linear(ca, sa, ga, cw, sw, gw, y, epilogue: LinearEpilogue, ws=None, out_dtype: int = OUT_BF16,
                       stream=None) -> None:
    """The NVFP4 linear with the whole epilogue."""
    M, N, K = _need_nvfp4_gemm(ca, sa, ga, cw, sw, gw, y, out_dtype)
    e = _need_linear(epilogue, y, M, N, out_dtype)
    _check(lib().dmpq_qgemm_nvfp4_linear(_stream(stream), _ptr(ca), _ptr(sa), _ptr(ga), _ptr(cw), _ptr(sw), _ptr(gw),
                                         M, N, K, out_dtype, _ptr(y), e, *_ws(ws)), "dmpq_qgemm_nvfp4_linear")


def new_linear_backward_workspace(M: int, N: int, gate_rows: int = 0, device="cuda"):
    """Workspace tensor for linear_epilogue_backward."""
    import torch
    return torch.empty(int(lib().dmpq_linear_backward_bytes(M, N, gate_rows)), dtype=torch.uint8, device=device)


def linear_epilogue_backward(dy, pre, du, ws=None, act: int = ACT_NONE, gate=None, gate_start=None, dgate=None,
                             dbias=None, stream=None) -> None:
    """Gradients of y = residual + gate * act(pre) from dy [M, N]: du of pre
    (may be dy or pre, or None), dgate [S, N] and dbias [N] fp32 (None: not
    computed).  pre may be None where act is ACT_NONE and dgate None."""
    M, N = dy.shape
    dtype = _float_type(dy, "dy")
    kind, size = _KIND[dtype]
    for t, name in ((pre, "pre"), (du, "du")):
        if t is not None:
            _need_type(t, name, size * M * N, kind)
    rows = 0
    if gate is not None:
        if gate.dim() != 2 or gate.shape[1] != N:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, needs (requests, {N})")
        rows = _gate_rows(gate, gate_start)
        if dgate is not None:
            _need_type(dgate, "dgate", 4 * rows * N, "fp32")
    elif gate_start is not None or dgate is not None:
        raise ValueError("gate is missing")
    if dbias is not None:
        _need_type(dbias, "dbias", 4 * N, "fp32")
    _check(lib().dmpq_linear_epilogue_backward(
        _stream(stream), _ptr(dy), _ptr(pre), M, N, dtype, act, _ptr(gate),
        0 if gate is None else _float_type(gate, "gate"), _ptr(gate_start), rows, _ptr(du), _ptr(dgate), _ptr(dbias),
        *_ws(ws)), "dmpq_linear_epilogue_backward")


# ---- the heads of q and k ---------------------------------------------------------

@functools.lru_cache(64)
def _int32s(values: tuple):
    return (C.c_int32 * len(values))(*values)


def rope_table(pos, freqs, axis_pairs, table, stream=None) -> None:
    """table [M, P, 2] fp32 = (cos, sin) of pos[m, axis] * freqs[p]: pos [M, axes]
    int32 or fp32, freqs [P] fp64 (radians per position), axis_pairs: how many of
    the P pairs turn with each axis, in their order."""
    if pos.dim() != 2 or pos.shape[1] != len(axis_pairs):
        raise ValueError(f"pos has shape {tuple(pos.shape)}, needs (rows, {len(axis_pairs)})")
    M, P = pos.shape[0], sum(axis_pairs)
    kinds = _types or _load_types()
    kind = OUT_F32 if pos.dtype in kinds["fp32"] else OUT_I32 if pos.dtype in kinds["int32"] else None
    if kind is None:
        raise ValueError(f"pos is {pos.dtype}, needs int32 or fp32")
    if freqs.dtype not in kinds["fp64"]:
        raise ValueError(f"freqs is {freqs.dtype}, needs fp64")
    _need(freqs, "freqs", 8 * P)
    _need_type(table, "table", 8 * M * P, "fp32")
    pairs = _int32s(tuple(axis_pairs))
    _check(lib().dmpq_rope_table(_stream(stream), _ptr(pos), kind, _ptr(freqs), M, len(axis_pairs), pairs,
                                 _ptr(table)), "dmpq_rope_table")


def _rows(t, name: str, M: int, n: int, dim: int, kind: str):
    """(pointer, row stride) of [M, n, dim] heads whose rows may lie apart."""
    if t is None:
        if n * M > 0:
            raise ValueError(f"{name} is missing")
        return None, n * dim
    if t.shape != (M, n, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {(M, n, dim)}")
    if t.dtype not in (_types or _load_types())[kind]:
        raise ValueError(f"{name} is {t.dtype}, needs {kind}")
    if not t.is_cuda:
        raise ValueError("libdmpq device arguments must be GPU tensors")
    st = t.stride()
    if (dim > 1 and st[2] != 1) or (n > 1 and st[1] != dim):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return (t.data_ptr() if M and n else None), (st[0] if M > 1 else n * dim)


def _qk_shape(q, k, heads: QkHeads):
    some = q if q is not None else k
    if some is None:
        raise ValueError("q and k are missing")
    M = some.shape[0]
    _need_table(heads, M)
    dtype = _float_type(some, "q")
    return M, dtype, _KIND[dtype][0]


def qk_norm_rope(q, k, heads: QkHeads, q_out, k_out, stream=None) -> None:
    """q_out, k_out = the heads of q [M, n_q, dim] and k [M, n_k, dim] normed and
    rotated (fp32 or bf16; may be q and k).  Rows may lie apart: q and k can be
    views into the rows of QKV.  q and q_out (k and k_out) are None for 0 heads."""
    M, dtype, kind = _qk_shape(q, k, heads)
    args = []
    for t, name, n in ((q, "q", heads.n_q), (k, "k", heads.n_k), (q_out, "q_out", heads.n_q),
                       (k_out, "k_out", heads.n_k)):
        args.append(_rows(t, name, M, n, heads.dim, kind))
    (pq, lq), (pk, lk), (po, lo), (pko, lko) = args
    _check(lib().dmpq_qk_norm_rope(_stream(stream), pq, lq, pk, lk, M, dtype, C.addressof(heads.struct), po, lo, pko,
                                   lko), "dmpq_qk_norm_rope")


def new_qk_backward_workspace(M: int, heads: QkHeads, device="cuda"):
    """Workspace tensor for qk_norm_rope_backward (the same for every M)."""
    import torch
    return torch.empty(int(lib().dmpq_qk_backward_bytes(heads.dim)), dtype=torch.uint8, device=device)


def qk_norm_rope_backward(dq, dk, q, k, heads: QkHeads, dxq, dxk, dwq=None, dbq=None, dwk=None, dbk=None, ws=None,
                          stream=None) -> None:
    """Gradients of qk_norm_rope: dxq, dxk of its inputs q and k from dq, dk of its
    outputs (may be the same), and dw*, db* [dim] fp32 (None: not computed).
    Without a norm q and k may be None."""
    M, dtype, kind = _qk_shape(dq, dk, heads)
    args = []
    for t, name, n in ((dq, "dq", heads.n_q), (dk, "dk", heads.n_k), (q, "q", heads.n_q), (k, "k", heads.n_k),
                       (dxq, "dxq", heads.n_q), (dxk, "dxk", heads.n_k)):
        if t is None and heads.norm == NORM_NONE and name in ("q", "k"):
            args += [None, n * heads.dim]
        else:
            args += _rows(t, name, M, n, heads.dim, kind)
    for t, name in ((dwq, "dwq"), (dbq, "dbq"), (dwk, "dwk"), (dbk, "dbk")):
        if t is not None:
            _need_type(t, name, 4 * heads.dim, "fp32")
    _check(lib().dmpq_qk_norm_rope_backward(
        _stream(stream), *args[:8], M, dtype, C.addressof(heads.struct), *args[8:], _ptr(dwq), _ptr(dbq), _ptr(dwk),
        _ptr(dbk), *_ws(ws)), "dmpq_qk_norm_rope_backward")
