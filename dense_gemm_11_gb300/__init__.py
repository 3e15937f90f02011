"""Python binding of libgemm11.so, the GB300 (sm_103a) dense GEMM library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/gemm11.h``.  There is no
fallback: if the shared library is missing, every call raises.

    gemm_f32(A, B, C, alpha=1.0, beta=0.0)            C = alpha*A@B + beta*C (fp32)
    gemm_f32_3xtf32(A, B, C, alpha=1.0, beta=0.0)     the same on the tensor cores (3 TF32 products)
    gemm_f16_f32acc_epilogue(A, B, C, alpha=1.0, beta=0.0, bias=None, act=0)
                                                      C = act(alpha*A@B + beta*C + bias)
    gemm_bf16_f32acc_epilogue(...)                    the same with bf16 A and B
    gemm_tc(A, B, C, ...)                             the same for fp16/bf16 A, B and fp32/fp16/bf16 C
    gemm_tc_batched(A, B, C, ..., b_trans=False)      a strided batch of those (3-D tensors), op(B) = B or B^T
    fp8_quantize(X, Q, S, layout="rows")              X held in 8 bits with an FP32 scale for each block of 128
    gemm_fp8(A, SA, B, SB, C, ..., b_trans=True)      the product of two matrices held that way
    moe_few_tokens(X, router, gate, up, down, Y, k)   a mixture-of-experts layer for a few tokens, one launch
    moe_dispatch(ids, X, Xs, offsets, rows)           the tokens' rows of such a layer, sorted by expert
    moe_combine(Ys, rows, Y, weights=None)            the experts' rows back to their tokens
    moe_combine_grad(dY, Ys, rows, weights, dYs, dw)  and the gradient of that
    gemm_grouped(A, B, C, offsets, ...)               every expert's rows times its matrix
    gemm_grouped_wgrad(A, B, C, offsets, ...)         the gradient of every expert's matrix
    fp8_gated_act(G, U, H, GQ, GS, UQ, US)            act(g) u, and g and u kept in 8 bits
    fp8_gated_act_grad(dH, GQ, GS, UQ, US, dG, dU)    its backward pass from these

Tensors are torch CUDA tensors on the current device; A and B may be 2-D
views with a leading dimension larger than their width (unit column stride).
Calls are asynchronous on the current torch stream (or ``stream=``).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from .build import DEBUG_LIB_PATH, LIB_PATH, build  # noqa: F401  (build() is part of the public API)

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = -1
GEMM_ERR_UNSUPPORTED = -2
GEMM_ERR_CUDA = -3
GEMM_ERR_TIMEOUT = -4
GEMM_ERR_SCRATCH_LIMIT = -5
GEMM_ERR_DEBUG_CHECK = -6
GEMM_ACT_NONE = 0
GEMM_ACT_GELU = 1
GEMM_ACT_RELU = 2
GEMM_ACT_GELU_TANH = 3
GEMM_ACT_SILU = 4
GEMM_DTYPE_F32 = 0
GEMM_DTYPE_F16 = 1
GEMM_DTYPE_BF16 = 2
GEMM_DTYPE_E4M3 = 3
GEMM_DTYPE_E5M2 = 4
GEMM_FP8_ROWS = 0
GEMM_FP8_COLS = 1
GEMM_FP8_BLOCKS = 2
GEMM_PATH_F32 = 0
GEMM_PATH_TC = 1


class TuneEntry(ctypes.Structure):
    """One row of the tuning table (gemm_tune_entry in include/gemm11.h)."""
    _fields_ = [("path", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("variant", ctypes.c_int), ("bn", ctypes.c_int), ("splits", ctypes.c_int)]

    def as_dict(self):
        return {f: int(getattr(self, f)) for f, _ in self._fields_}

EXPORTED_SYMBOLS = ("gemm_f32", "gemm_f32_3xtf32", "gemm_f16_f32acc_epilogue", "gemm_bf16_f32acc_epilogue",
                    "gemm_tc_f32acc_epilogue", "gemm_tc_strided_batched", "gemm_f16_f32acc_epilogue_noalloc",
                    "gemm_fp8_quantize_block128", "gemm_fp8_block128", "gemm_moe_few_tokens",
                    "gemm_moe_dispatch", "gemm_moe_combine", "gemm_moe_combine_grad", "gemm_grouped_f32acc",
                    "gemm_grouped_wgrad_f32acc", "gemm_fp8_gated_act", "gemm_fp8_gated_act_grad", "gemm_call_words",
                    "gemm_tune_set", "gemm_tune_get",
                    "gemm_status_string", "gemm_last_cuda_error", "gemm_check", "gemm_watchdog_selftest",
                    "gemm_last_plan", "gemm_last_launch_count", "gemm_tc_rate_probe",
                    "gemm_pipeline_stall_selftest", "gemm_fma_rate_probe", "gemm_tma_read_probe",
                    "gemm_debug_build")

_lock = threading.Lock()
_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = status_string(status) if _lib is not None else str(status)
        if status == GEMM_ERR_CUDA and _lib is not None:
            msg += f" (cudaError {_lib.gemm_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


def library_path() -> str:
    """The library this process uses: the debug build (libgemm11_debug.so)
    when the environment variable GEMM11_DEBUG is 1, else libgemm11.so."""
    return DEBUG_LIB_PATH if os.environ.get("GEMM11_DEBUG", "0") == "1" else LIB_PATH


def lib():
    """The loaded library (ctypes): libgemm11.so, or libgemm11_debug.so with
    GEMM11_DEBUG=1.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{os.path.basename(path)} is not built ({path}); call "
                                   "dense_gemm_11_gb300.build()")
            L = ctypes.CDLL(path)
            c_int, c_float, c_void_p = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
            L.gemm_f32.restype = c_int
            L.gemm_f32.argtypes = [c_int, c_int, c_int, c_float, c_void_p, c_int, c_void_p, c_int, c_float,
                                   c_void_p, c_int, c_void_p]
            L.gemm_f32_3xtf32.restype = c_int
            L.gemm_f32_3xtf32.argtypes = L.gemm_f32.argtypes
            L.gemm_f16_f32acc_epilogue.restype = c_int
            L.gemm_f16_f32acc_epilogue.argtypes = [c_int, c_int, c_int, c_float, c_void_p, c_void_p, c_float,
                                                   c_void_p, c_void_p, c_int, c_void_p]
            L.gemm_bf16_f32acc_epilogue.restype = c_int
            L.gemm_bf16_f32acc_epilogue.argtypes = L.gemm_f16_f32acc_epilogue.argtypes
            L.gemm_tc_f32acc_epilogue.restype = c_int
            L.gemm_tc_f32acc_epilogue.argtypes = [c_int, c_int, c_int, c_float, c_void_p, c_void_p, c_int,
                                                  c_float, c_void_p, c_int, c_void_p, c_int, c_void_p]
            c_ll = ctypes.c_longlong
            L.gemm_tc_strided_batched.restype = c_int
            L.gemm_tc_strided_batched.argtypes = [c_int, c_int, c_int, c_int, c_float, c_void_p, c_ll, c_void_p,
                                                  c_ll, c_int, c_int, c_float, c_void_p, c_ll, c_int, c_void_p,
                                                  c_int, c_void_p]
            L.gemm_f16_f32acc_epilogue_noalloc.restype = c_int
            L.gemm_f16_f32acc_epilogue_noalloc.argtypes = L.gemm_f16_f32acc_epilogue.argtypes
            L.gemm_fp8_quantize_block128.restype = c_int
            L.gemm_fp8_quantize_block128.argtypes = [c_int, c_int, c_void_p, c_int, c_ll, c_void_p, c_int, c_ll,
                                                     c_void_p, c_ll, c_int, c_void_p]
            L.gemm_fp8_block128.restype = c_int
            L.gemm_fp8_block128.argtypes = [c_int, c_int, c_int, c_float, c_void_p, c_int, c_ll, c_void_p, c_ll,
                                            c_void_p, c_int, c_ll, c_void_p, c_ll, c_int, c_int, c_float, c_void_p,
                                            c_int, c_ll, c_void_p, c_int, c_void_p]
            L.gemm_moe_few_tokens.restype = c_int
            L.gemm_moe_few_tokens.argtypes = [c_int, c_int, c_int, c_int, c_int, c_void_p, c_int, c_ll, c_void_p, c_int,
                                              c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_int,
                                              c_int, c_void_p, c_int, c_ll, c_void_p, c_void_p, c_void_p]
            L.gemm_moe_dispatch.restype = c_int
            L.gemm_moe_dispatch.argtypes = [c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_int, c_ll, c_void_p, c_ll, c_void_p,
                                            c_void_p, c_void_p]
            L.gemm_moe_combine.restype = c_int
            L.gemm_moe_combine.argtypes = [c_int, c_int, c_int, c_int, c_void_p, c_int, c_ll, c_void_p, c_void_p, c_void_p, c_ll,
                                           c_void_p]
            L.gemm_moe_combine_grad.restype = c_int
            L.gemm_moe_combine_grad.argtypes = [c_int, c_int, c_int, c_int, c_void_p, c_int, c_ll, c_void_p, c_ll, c_void_p,
                                                c_void_p, c_void_p, c_ll, c_void_p, c_void_p]
            L.gemm_grouped_f32acc.restype = c_int
            L.gemm_grouped_f32acc.argtypes = [c_int, c_int, c_int, c_int, c_float, c_void_p, c_ll, c_void_p, c_ll, c_ll, c_int,
                                              c_int, c_float, c_void_p, c_int, c_ll, c_void_p, c_void_p]
            L.gemm_grouped_wgrad_f32acc.restype = c_int
            L.gemm_grouped_wgrad_f32acc.argtypes = [c_int, c_int, c_int, c_int, c_float, c_void_p, c_ll, c_void_p, c_ll, c_int,
                                                    c_float, c_void_p, c_int, c_ll, c_ll, c_void_p, c_void_p]
            L.gemm_fp8_gated_act.restype = c_int
            L.gemm_fp8_gated_act.argtypes = [c_int, c_int, c_void_p, c_ll, c_void_p, c_ll, c_int, c_void_p, c_ll, c_void_p, c_ll,
                                             c_void_p, c_ll, c_void_p, c_ll, c_void_p, c_ll, c_int, c_int, c_void_p]
            L.gemm_fp8_gated_act_grad.restype = c_int
            L.gemm_fp8_gated_act_grad.argtypes = [c_int, c_int, c_void_p, c_ll, c_int, c_void_p, c_ll, c_void_p, c_ll, c_void_p,
                                                  c_ll, c_void_p, c_ll, c_int, c_void_p, c_ll, c_void_p, c_ll, c_void_p, c_ll,
                                                  c_int, c_void_p]
            L.gemm_call_words.restype = c_int
            L.gemm_call_words.argtypes = [c_int, ctypes.c_char_p, c_int]
            L.gemm_tune_set.restype = c_int
            L.gemm_tune_set.argtypes = [ctypes.POINTER(TuneEntry), c_int]
            L.gemm_tune_get.restype = c_int
            L.gemm_tune_get.argtypes = [ctypes.POINTER(TuneEntry), c_int]
            L.gemm_status_string.restype = ctypes.c_char_p
            L.gemm_status_string.argtypes = [c_int]
            L.gemm_last_cuda_error.restype = c_int
            L.gemm_last_cuda_error.argtypes = []
            L.gemm_check.restype = c_int
            L.gemm_check.argtypes = [c_void_p]
            L.gemm_watchdog_selftest.restype = c_int
            L.gemm_watchdog_selftest.argtypes = [c_int, c_void_p]
            L.gemm_last_plan.restype = ctypes.c_char_p
            L.gemm_last_plan.argtypes = []
            L.gemm_last_launch_count.restype = c_int
            L.gemm_last_launch_count.argtypes = []
            L.gemm_pipeline_stall_selftest.restype = c_int
            L.gemm_pipeline_stall_selftest.argtypes = [c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_int,
                                                       c_void_p]
            L.gemm_debug_build.restype = c_int
            L.gemm_debug_build.argtypes = []
            L.gemm_fma_rate_probe.restype = c_int
            L.gemm_fma_rate_probe.argtypes = [c_int, c_int, ctypes.POINTER(ctypes.c_double), c_void_p]
            L.gemm_tc_rate_probe.restype = c_int
            L.gemm_tc_rate_probe.argtypes = [c_int, ctypes.POINTER(ctypes.c_double), c_void_p]
            L.gemm_tma_read_probe.restype = c_int
            L.gemm_tma_read_probe.argtypes = [c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(ctypes.c_double),
                                              ctypes.POINTER(ctypes.c_double), c_void_p]
            _lib = L
    return _lib


def debug_build() -> bool:
    """True when the loaded library is the GEMM11_DEBUG build."""
    return bool(lib().gemm_debug_build())


def status_string(status: int) -> str:
    return lib().gemm_status_string(int(status)).decode()


def last_plan() -> str:
    return lib().gemm_last_plan().decode()


def last_launch_count() -> int:
    return int(lib().gemm_last_launch_count())


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _mat(t, name, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs unit column stride")
    # a single row has no row stride of its own: report the tensor's when it is
    # a valid one (a view keeps its parent's, which may be 16-byte aligned)
    if t.shape[0] > 1 or t.stride(0) >= t.shape[1]:
        _check_rows(name, *t.shape, t.stride(0))
        return t.data_ptr(), max(t.stride(0), 1)
    return t.data_ptr(), max(t.shape[1], 1)


def _check_rows(name, rows, cols, ld):
    """Rows that share memory (an expanded tensor) have no leading dimension."""
    if rows > 1 and 0 < cols > ld:
        raise ValueError(f"{name} needs a row stride of at least its width, got {ld} for {rows} x {cols} (an expanded tensor?)")


def gemm_f32_raw(M, N, K, alpha, A_ptr, lda, B_ptr, ldb, beta, C_ptr, ldc, stream_ptr=0) -> int:
    """Direct C-ABI call with integer device pointers; returns the status code."""
    return lib().gemm_f32(int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr), int(lda),
                          ctypes.c_void_p(B_ptr), int(ldb), float(beta), ctypes.c_void_p(C_ptr), int(ldc),
                          ctypes.c_void_p(stream_ptr))


def gemm_f16_raw(M, N, K, alpha, A_ptr, B_ptr, beta, C_ptr, bias_ptr=0, act=0, stream_ptr=0) -> int:
    """Direct C-ABI call with integer device pointers; returns the status code."""
    return lib().gemm_f16_f32acc_epilogue(int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr),
                                          ctypes.c_void_p(B_ptr), float(beta), ctypes.c_void_p(C_ptr),
                                          ctypes.c_void_p(bias_ptr or None), int(act), ctypes.c_void_p(stream_ptr))


def gemm_bf16_raw(M, N, K, alpha, A_ptr, B_ptr, beta, C_ptr, bias_ptr=0, act=0, stream_ptr=0) -> int:
    """Direct C-ABI call of the BF16-input entry point; returns the status code."""
    return lib().gemm_bf16_f32acc_epilogue(int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr),
                                           ctypes.c_void_p(B_ptr), float(beta), ctypes.c_void_p(C_ptr),
                                           ctypes.c_void_p(bias_ptr or None), int(act), ctypes.c_void_p(stream_ptr))


def gemm_tc_raw(M, N, K, alpha, A_ptr, B_ptr, ab_type, beta, C_ptr, c_type, bias_ptr=0, act=0,
                stream_ptr=0) -> int:
    """Direct C-ABI call of the general tensor-core entry point; returns the status code."""
    return lib().gemm_tc_f32acc_epilogue(int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr),
                                         ctypes.c_void_p(B_ptr), int(ab_type), float(beta), ctypes.c_void_p(C_ptr),
                                         int(c_type), ctypes.c_void_p(bias_ptr or None), int(act),
                                         ctypes.c_void_p(stream_ptr))


def gemm_tc_batched_raw(batch, M, N, K, alpha, A_ptr, stride_a, B_ptr, stride_b, ab_type, b_trans, beta, C_ptr,
                        stride_c, c_type, bias_ptr=0, act=0, stream_ptr=0) -> int:
    """Direct C-ABI call of the strided-batched entry point; returns the status code."""
    return lib().gemm_tc_strided_batched(int(batch), int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr),
                                         int(stride_a), ctypes.c_void_p(B_ptr), int(stride_b), int(ab_type),
                                         int(b_trans), float(beta), ctypes.c_void_p(C_ptr), int(stride_c),
                                         int(c_type), ctypes.c_void_p(bias_ptr or None), int(act),
                                         ctypes.c_void_p(stream_ptr))


def gemm_f16_noalloc_raw(M, N, K, alpha, A_ptr, B_ptr, beta, C_ptr, bias_ptr=0, act=0, stream_ptr=0) -> int:
    """C-ABI call of the no-allocation variant (M <= 64); returns the status code.

    For callers that cannot let the library allocate device memory: the
    split-K scratch is a fixed array inside the library.  Calls that overlap
    on the GPU share that array and race; issue them on one stream.
    """
    return lib().gemm_f16_f32acc_epilogue_noalloc(int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr),
                                                  ctypes.c_void_p(B_ptr), float(beta), ctypes.c_void_p(C_ptr),
                                                  ctypes.c_void_p(bias_ptr or None), int(act),
                                                  ctypes.c_void_p(stream_ptr))


def gemm_f32_3xtf32_raw(M, N, K, alpha, A_ptr, lda, B_ptr, ldb, beta, C_ptr, ldc, stream_ptr=0) -> int:
    """Direct C-ABI call of the 3xTF32 FP32 GEMM; returns the status code."""
    return lib().gemm_f32_3xtf32(int(M), int(N), int(K), float(alpha), ctypes.c_void_p(A_ptr), int(lda),
                                 ctypes.c_void_p(B_ptr), int(ldb), float(beta), ctypes.c_void_p(C_ptr), int(ldc),
                                 ctypes.c_void_p(stream_ptr))


def gemm_f32_3xtf32(A, B, C, alpha: float = 1.0, beta: float = 0.0, *, stream=None) -> None:
    """C = alpha * A @ B + beta * C, FP32 operands, on the tensor cores (3 TF32 products)."""
    _gemm_f32_like("gemm_f32_3xtf32", A, B, C, alpha, beta, stream)


def gemm_f32(A, B, C, alpha: float = 1.0, beta: float = 0.0, *, stream=None) -> None:
    """C = alpha * A @ B + beta * C in true FP32 (CUDA-core FFMA)."""
    _gemm_f32_like("gemm_f32", A, B, C, alpha, beta, stream)


def _gemm_f32_like(fn_name, A, B, C, alpha, beta, stream) -> None:
    import torch
    a_ptr, lda = _mat(A, "A", torch.float32)
    b_ptr, ldb = _mat(B, "B", torch.float32)
    c_ptr, ldc = _mat(C, "C", torch.float32)
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    st = getattr(lib(), fn_name)(M, N, K, float(alpha), ctypes.c_void_p(a_ptr), lda, ctypes.c_void_p(b_ptr), ldb,
                                 float(beta), ctypes.c_void_p(c_ptr), ldc, _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, fn_name)


def _gemm_16bit(fn_name, in_dtype, A, B, C, alpha, beta, bias, act, stream) -> None:
    import torch
    for name, t, dt in (("A", A, in_dtype), ("B", B, in_dtype), ("C", C, torch.float32)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dt or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D CUDA {dt} tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (leading dimension = width)")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    bias_ptr = None
    if bias is not None:
        if not bias.is_cuda or bias.dtype != torch.float32 or bias.numel() != N or not bias.is_contiguous():
            raise TypeError("bias must be a contiguous CUDA float32 tensor of length N")
        bias_ptr = bias.data_ptr()
    st = getattr(lib(), fn_name)(M, N, K, float(alpha), ctypes.c_void_p(A.data_ptr()),
                                 ctypes.c_void_p(B.data_ptr()), float(beta), ctypes.c_void_p(C.data_ptr()),
                                 ctypes.c_void_p(bias_ptr), int(act), _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, fn_name)


def gemm_f16_f32acc_epilogue(A, B, C, alpha: float = 1.0, beta: float = 0.0, bias=None, act: int = 0, *,
                             stream=None) -> None:
    """C = act(alpha * A @ B + beta * C + bias): fp16 A, B; fp32 accumulate, bias and C."""
    import torch
    _gemm_16bit("gemm_f16_f32acc_epilogue", torch.float16, A, B, C, alpha, beta, bias, act, stream)


def gemm_bf16_f32acc_epilogue(A, B, C, alpha: float = 1.0, beta: float = 0.0, bias=None, act: int = 0, *,
                              stream=None) -> None:
    """C = act(alpha * A @ B + beta * C + bias): bf16 A, B; fp32 accumulate, bias and C."""
    import torch
    _gemm_16bit("gemm_bf16_f32acc_epilogue", torch.bfloat16, A, B, C, alpha, beta, bias, act, stream)


def gemm_tc(A, B, C, alpha: float = 1.0, beta: float = 0.0, bias=None, act: int = 0, *, stream=None) -> None:
    """C = act(alpha * A @ B + beta * C + bias) on the tensor cores, FP32 accumulate.

    A and B: both fp16 or both bf16.  C: fp32, fp16 or bf16 (a 16-bit C is the
    FP32 epilogue value rounded once to nearest even).  bias: fp32 or None.
    """
    import torch
    types = {torch.float32: GEMM_DTYPE_F32, torch.float16: GEMM_DTYPE_F16, torch.bfloat16: GEMM_DTYPE_BF16}
    for name, t in (("A", A), ("B", B), ("C", C)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.dtype not in types:
            raise TypeError(f"{name} must be a 2-D CUDA float32/float16/bfloat16 tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (leading dimension = width)")
    if A.dtype != B.dtype or A.dtype == torch.float32:
        raise TypeError("A and B must both be float16 or both bfloat16")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    bias_ptr = 0
    if bias is not None:
        if not bias.is_cuda or bias.dtype != torch.float32 or bias.numel() != N or not bias.is_contiguous():
            raise TypeError("bias must be a contiguous CUDA float32 tensor of length N")
        bias_ptr = bias.data_ptr()
    st = lib().gemm_tc_f32acc_epilogue(M, N, K, float(alpha), ctypes.c_void_p(A.data_ptr()),
                                       ctypes.c_void_p(B.data_ptr()), types[A.dtype], float(beta),
                                       ctypes.c_void_p(C.data_ptr()), types[C.dtype],
                                       ctypes.c_void_p(bias_ptr or None), int(act), _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_tc_f32acc_epilogue")


def _batched_operand(t, name, rows, cols):
    """(pointer, batch stride in elements, batch) of a 2-D (shared) or 3-D operand
    whose matrices are row-major with unit column stride and row stride = cols."""
    if t.dim() == 2:
        if tuple(t.shape) != (rows, cols) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {rows} x {cols} matrix")
        return t.data_ptr(), 0, None
    if t.dim() != 3 or tuple(t.shape[1:]) != (rows, cols) or t.stride(2) != 1 or t.stride(1) != cols:
        raise ValueError(f"{name} must be (batch, {rows}, {cols}) with row-major matrices, got "
                         f"shape {tuple(t.shape)} strides {t.stride()}")
    return t.data_ptr(), t.stride(0), t.shape[0]


def gemm_tc_batched(A, B, C, alpha: float = 1.0, beta: float = 0.0, bias=None, act: int = 0, *,
                    b_trans: bool = False, stream=None) -> None:
    """C[z] = act(alpha * A[z] @ op(B[z]) + beta * C[z] + bias) for every z, one launch.

    C: (batch, M, N) fp32/fp16/bf16.  A: (batch, M, K) or a shared (M, K).
    B: (batch, K, N), or (batch, N, K) with b_trans=True (op(B) = B^T, e.g. the
    keys of Q K^T); a 2-D B is shared by the batch.  A 3-D operand may have
    batch stride 0 (torch.expand).  A and B both fp16 or both bf16.
    """
    import torch
    types = {torch.float32: GEMM_DTYPE_F32, torch.float16: GEMM_DTYPE_F16, torch.bfloat16: GEMM_DTYPE_BF16}
    for name, t in (("A", A), ("B", B), ("C", C)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in types:
            raise TypeError(f"{name} must be a CUDA float32/float16/bfloat16 tensor")
    if A.dtype != B.dtype or A.dtype == torch.float32:
        raise TypeError("A and B must both be float16 or both bfloat16")
    if C.dim() != 3:
        raise ValueError("C must be (batch, M, N)")
    batch, M, N = C.shape
    K = A.shape[-1]
    c_ptr, sc, _ = _batched_operand(C, "C", M, N)
    a_ptr, sa, ba = _batched_operand(A, "A", M, K)
    b_ptr, sb, bb = _batched_operand(B, "B", N if b_trans else K, K if b_trans else N)
    for nb, name in ((ba, "A"), (bb, "B")):
        if nb is not None and nb != batch:
            raise ValueError(f"{name} has batch {nb}, C has {batch}")
    if batch > 1 and sc < M * N:
        raise ValueError("C's matrices overlap (batch stride < M * N)")
    bias_ptr = 0
    if bias is not None:
        if not bias.is_cuda or bias.dtype != torch.float32 or bias.numel() != N or not bias.is_contiguous():
            raise TypeError("bias must be a contiguous CUDA float32 tensor of length N")
        bias_ptr = bias.data_ptr()
    st = lib().gemm_tc_strided_batched(batch, M, N, K, float(alpha), ctypes.c_void_p(a_ptr), sa,
                                       ctypes.c_void_p(b_ptr), sb, types[A.dtype], 1 if b_trans else 0, float(beta),
                                       ctypes.c_void_p(c_ptr), sc if batch > 1 else M * N, types[C.dtype],
                                       ctypes.c_void_p(bias_ptr or None), int(act), _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_tc_strided_batched")


_FP8_LAYOUTS = {"rows": GEMM_FP8_ROWS, "cols": GEMM_FP8_COLS, "blocks": GEMM_FP8_BLOCKS}
_TYPE_NAMES = ("float32", "float16", "bfloat16", "float8_e4m3fn", "float8_e5m2")
_F32 = (GEMM_DTYPE_F32,)
_HALFS = (GEMM_DTYPE_F16, GEMM_DTYPE_BF16)
_FLOATS = (GEMM_DTYPE_F32, GEMM_DTYPE_F16, GEMM_DTYPE_BF16)
_FP8S = (GEMM_DTYPE_E4M3, GEMM_DTYPE_E5M2)
_codes = {}  # torch dtype -> gemm_dtype code
_plain_types = {}  # name -> torch dtype
_raw_stream = _device_now = None


def _load_codes():
    """Fill the type tables and look up how to get the current stream and device; torch is imported on first use."""
    global _raw_stream, _device_now
    import torch
    _device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _plain_types.update(int32=torch.int32, float32=torch.float32)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
    _codes.update({getattr(torch, name): code for code, name in enumerate(_TYPE_NAMES)})


def _typed_mat(t, name, allowed):
    """(pointer, row stride, rows, cols, type code) of a 2-D CUDA tensor with unit
    column stride and one of the types `allowed`.  The calls below are short on
    the GPU: the checks take one pass over the tensor's properties."""
    if not _codes:
        _load_codes()
    code = _codes.get(getattr(t, "dtype", None), -1)
    if code not in allowed or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of type {'/'.join(_TYPE_NAMES[c] for c in allowed)}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    ld, step = stride
    if step != 1 and cols > 1:
        raise ValueError(f"{name} needs unit column stride")
    if ld < cols:  # a single row has no row stride of its own
        _check_rows(name, rows, cols, ld)
        ld = cols
    return t.data_ptr(), ld or 1, rows, cols, code


def _stream_ptr(stream, t):
    """The raw handle of `stream`, or of the current stream of t's device."""
    return stream.cuda_stream if stream is not None else _raw_stream(t.get_device())


def _fp8_shapes(rows, cols, layout):
    """Shapes of Q and S of a rows x cols matrix."""
    if layout not in _FP8_LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(_FP8_LAYOUTS)}, got {layout!r}")
    if layout == "rows":
        return (rows, cols), (-(-cols // 128), rows)
    if layout == "cols":
        return (cols, rows), (-(-rows // 128), cols)
    return (rows, cols), (-(-rows // 128), -(-cols // 128))


def fp8_empty(rows: int, cols: int, layout: str = "rows", dtype=None, device="cuda"):
    """Uninitialised (Q, S) for fp8_quantize of a rows x cols matrix, with row
    strides that gemm_fp8 takes (Q: a multiple of 16, S: a multiple of 4)."""
    import torch
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    (qr, qc), (sr, sc) = _fp8_shapes(rows, cols, layout)
    Q = torch.empty(qr, (qc + 15) // 16 * 16, dtype=dtype, device=device)[:, :qc]
    S = torch.empty(sr, (sc + 3) // 4 * 4, dtype=torch.float32, device=device)[:, :sc]
    return Q, S


def fp8_quantize(X, Q, S, layout: str = "rows", *, stream=None) -> None:
    """X (rows x cols; fp32, fp16 or bf16) to 8 bits with one FP32 scale for each block of 128.

    layout "rows":   blocks of 128 along a row; Q is rows x cols, S is (ceil(cols/128), rows).
    layout "cols":   blocks of 128 along a column; Q is the transpose, cols x rows, S is (ceil(rows/128), cols).
    layout "blocks": blocks of 128 x 128; Q is rows x cols, S is (ceil(rows/128), ceil(cols/128)).
    Q is float8_e4m3fn or float8_e5m2.  fp8_empty() makes a fitting pair.
    """
    x_ptr, ldx, rows, cols, x_type = _typed_mat(X, "X", _FLOATS)
    q_ptr, ldq, q_rows, q_cols, q_type = _typed_mat(Q, "Q", _FP8S)
    s_ptr, lds, s_rows, s_cols, _ = _typed_mat(S, "S", _F32)
    if ((q_rows, q_cols), (s_rows, s_cols)) != _fp8_shapes(rows, cols, layout):
        raise ValueError(f"shape mismatch X{tuple(X.shape)} Q{tuple(Q.shape)} S{tuple(S.shape)} for layout {layout!r}")
    st = lib().gemm_fp8_quantize_block128(rows, cols, x_ptr, x_type, ldx, q_ptr, q_type, ldq, s_ptr, lds,
                                          _FP8_LAYOUTS[layout], _stream_ptr(stream, X))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp8_quantize_block128")


def gemm_fp8(A, SA, B, SB, C, alpha: float = 1.0, beta: float = 0.0, bias=None, act: int = 0, *,
             b_trans: bool = True, b_scales: str = "blocks", stream=None) -> None:
    """C = act(alpha * A @ op(B) + beta * C + bias) of matrices held in 8 bits (see fp8_quantize).

    A: (M, K) with SA in layout "rows".  C: (M, N) fp32, fp16 or bf16; bias: fp32 or None.
    b_trans=True:  B is (N, K), op(B) = B^T, with scales in layout b_scales, "blocks" or "rows".
    b_trans=False: B is (K, N), op(B) = B, with scales in layout "blocks".
    So y = x W^T takes x in "rows" and W in "blocks"; dx = dy W takes dy in "rows" and the same
    W with b_trans=False; dW = dy^T x takes both quantized with layout "cols" and b_scales="rows".
    """
    a_ptr, lda, M, K, a_type = _typed_mat(A, "A", _FP8S)
    b_ptr, ldb, b_rows, b_cols, b_type = _typed_mat(B, "B", _FP8S)
    c_ptr, ldc, c_rows, N, c_type = _typed_mat(C, "C", _FLOATS)
    sa_ptr, ldsa, sa_rows, sa_cols, _ = _typed_mat(SA, "SA", _F32)
    sb_ptr, ldsb, sb_rows, sb_cols, _ = _typed_mat(SB, "SB", _F32)
    if c_rows != M or (b_rows, b_cols) != ((N, K) if b_trans else (K, N)):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    if b_scales != "blocks" and (b_scales != "rows" or not b_trans):
        raise ValueError(f"b_scales must be 'blocks', or 'rows' with b_trans=True, got {b_scales!r}")
    if sa_rows != -(-K // 128) or sa_cols != M or (sb_rows, sb_cols) != _fp8_shapes(b_rows, b_cols, b_scales)[1]:
        raise ValueError(f"scales do not fit: SA{tuple(SA.shape)} SB{tuple(SB.shape)} for A{tuple(A.shape)} B{tuple(B.shape)}")
    st = lib().gemm_fp8_block128(M, N, K, alpha, a_ptr, a_type, lda, sa_ptr, ldsa, b_ptr, b_type, ldb, sb_ptr, ldsb,
                                 1 if b_trans else 0, _FP8_LAYOUTS[b_scales], beta, c_ptr, c_type, ldc,
                                 None if bias is None else _vector(bias, "bias", N), act, _stream_ptr(stream, A))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp8_block128")


def moe_few_tokens(X, router, gate, up, down, Y, top_k: int, *, scales=None, act: int = GEMM_ACT_SILU,
                   renormalize: bool = True, ids=None, weights=None, stream=None) -> None:
    """Y = sum_j w_j down[e_j] @ (act(gate[e_j] @ x) * (up[e_j] @ x)) for every row x of X, in one launch.

    X: (T, H) fp16 or bf16.  router: (E, H), X's type or fp32.  gate, up: (E, I, H), down: (E, H, I), contiguous,
    X's type, or float8_e4m3fn with scales = (s_gate, s_up, s_down), one fp32 scale for each 128 x 128 block
    ((E, ceil(I/128), ceil(H/128)) and (E, ceil(H/128), ceil(I/128)); fp8_quantize with layout "blocks", expert by
    expert).  up=None: no gating, h = act(gate @ x).  Y: (T, H) fp32, fp16 or bf16.
    The e_j are the top_k largest logits of router @ x (ties: the lower index); w_j their softmax probabilities,
    divided by their sum with renormalize=True.  ids (int32) and weights (fp32), both (T, top_k) and contiguous,
    receive them if given.  Limits: T <= 128, E <= 512, top_k <= 16, T * top_k <= 1024, H and I multiples of 16, H <= 32768,
    T * top_k * I < 2^31.
    """
    x_ptr, ldx, T, H, x_type = _typed_mat(X, "X", _HALFS)
    y_ptr, ldy, y_rows, y_cols, y_type = _typed_mat(Y, "Y", _FLOATS)
    r_ptr, ldr, E, r_cols, r_type = _typed_mat(router, "router", _FLOATS)
    if y_rows != T or y_cols != H or r_cols != H or (E > 1 and ldr != H):
        raise ValueError(f"shape mismatch X{tuple(X.shape)} router{tuple(router.shape)} Y{tuple(Y.shape)} (router contiguous)")
    if r_type != x_type and r_type != GEMM_DTYPE_F32:
        raise TypeError("router must have X's type or be float32")
    shape = getattr(gate, "shape", ())
    I = shape[1] if len(shape) == 3 else -1
    w_type = _codes.get(getattr(gate, "dtype", None), -1)
    if w_type != x_type and w_type != GEMM_DTYPE_E4M3:
        raise TypeError("gate, up and down must have X's type or be float8_e4m3fn")
    g_ptr = _expert_tensor(gate, "gate", gate.dtype, E, I, H)
    u_ptr = None if up is None else _expert_tensor(up, "up", gate.dtype, E, I, H)
    d_ptr = _expert_tensor(down, "down", gate.dtype, E, H, I)
    sg_ptr = su_ptr = sd_ptr = None
    if w_type == GEMM_DTYPE_E4M3:
        if scales is None or len(scales) != 3:
            raise ValueError("8-bit weights need scales = (s_gate, s_up, s_down)")
        import torch
        hb, ib = -(-H // 128), -(-I // 128)
        sg_ptr = _expert_tensor(scales[0], "scales[0]", torch.float32, E, ib, hb)
        su_ptr = None if up is None else _expert_tensor(scales[1], "scales[1]", torch.float32, E, ib, hb)
        sd_ptr = _expert_tensor(scales[2], "scales[2]", torch.float32, E, hb, ib)
    elif scales is not None:
        raise ValueError("scales are for 8-bit weights only")
    st = lib().gemm_moe_few_tokens(T, E, top_k, H, I, x_ptr, x_type, ldx, r_ptr, r_type, g_ptr, u_ptr, d_ptr, w_type, sg_ptr,
                                   su_ptr, sd_ptr, act, 1 if renormalize else 0, y_ptr, y_type, ldy,
                                   None if ids is None else _choice(ids, "ids", "int32", T, top_k),
                                   None if weights is None else _choice(weights, "weights", "float32", T, top_k),
                                   _stream_ptr(stream, X))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_moe_few_tokens")


def _expert_tensor(t, name, dtype, E, rows, cols):
    if getattr(t, "dtype", None) != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.shape != (E, rows, cols) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and {(E, rows, cols)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _choice(t, name, dtype, T, k):
    import torch
    if getattr(t, "dtype", None) != getattr(torch, dtype) or not t.is_cuda or t.shape != (T, k) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {(T, k)}")
    return t.data_ptr()


def _vector(t, name, n):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA float32 tensor of length {n}")
    return t.data_ptr()


# The calls below are short on the GPU, and most of a call is what the host does:
# each tensor is looked at once, and the arguments go over as an array of words.
_pack13, _pack12, _pack15, _pack20, _pack22 = (struct.Struct(f"={n}q").pack for n in (13, 12, 15, 20, 22))
_pack_grouped, _pack_wgrad = struct.Struct("=4qd7qd5q").pack, struct.Struct("=4qd5qd6q").pack


def _placed(t, name, allowed):
    """(pointer, row stride, rows, cols, type code, device) of a 2-D CUDA tensor, as _typed_mat takes it."""
    try:
        code, device = _codes[t.dtype], t.get_device()
        rows, cols = t.shape
        ld, step = t.stride()
        if code in allowed and step == 1 and ld >= cols > 0 <= device:
            return t.data_ptr(), ld, rows, cols, code, device
    except Exception:  # noqa: S110 (no tensor, another type or shape: named below)
        pass
    if not _codes:
        _load_codes()
    code = _codes.get(getattr(t, "dtype", None), -1)
    if code not in allowed or (device := t.get_device()) < 0:
        raise TypeError(f"{name} must be a CUDA tensor of type {'/'.join(_TYPE_NAMES[c] for c in allowed)}")
    if len(t.shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} needs unit column stride")
    if ld < cols:  # a single row has no row stride of its own
        _check_rows(name, rows, cols, ld)
        ld = cols
    return t.data_ptr(), ld or 1, rows, cols, code, device


def _packed(t, name, dtype_name, shape):
    """(pointer, device) of a contiguous CUDA tensor of this type and shape."""
    if not _codes:
        _load_codes()
    if getattr(t, "dtype", None) is not _plain_types[dtype_name] or (device := t.get_device()) < 0:
        raise TypeError(f"{name} must be a CUDA {dtype_name} tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr(), device


def _slots(t, name):
    """(pointer, T, top_k, device) of a contiguous (T, top_k) int32 tensor."""
    shape = getattr(t, "shape", ())
    ptr, device = _packed(t, name, "int32", shape)
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be (T, top_k) with top_k >= 1, got {tuple(shape)}")
    return ptr, shape[0], shape[1], device


def _offsets(t):
    """(pointer, E, device) of the offsets of E experts' rows."""
    shape = getattr(t, "shape", ())
    ptr, device = _packed(t, "offsets", "int32", shape)
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError(f"offsets must be (E + 1,), got {tuple(shape)}")
    return ptr, shape[0] - 1, device


def _expert_mats(t, name, allowed):
    """(pointer, row stride, matrix stride, E, rows, cols, type code, device) of a 3-D CUDA tensor of row-major matrices."""
    if not _codes:
        _load_codes()
    code = _codes.get(getattr(t, "dtype", None), -1)
    if code not in allowed or (device := t.get_device()) < 0:
        raise TypeError(f"{name} must be a CUDA tensor of type {'/'.join(_TYPE_NAMES[c] for c in allowed)}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D")
    E, rows, cols = shape
    step, ld, one = stride
    if one != 1 and cols > 1:
        raise ValueError(f"{name} needs unit column stride")
    if ld < cols:
        _check_rows(name, rows, cols, ld)
        ld = cols
    size = (rows - 1) * ld + cols
    if E > 1 and rows > 0 and cols > 0 and step < size:
        raise ValueError(f"{name} needs matrices that share no memory, got stride {step} for {rows} x {cols} (an expanded tensor?)")
    return t.data_ptr(), ld or 1, max(step, 1), E, rows, cols, code, device


def _elsewhere(*devices):
    raise ValueError(f"every tensor must be on the current device, cuda:{_device_now()}; got them on {devices}")


def moe_dispatch(ids, X, Xs, offsets, rows, *, stream=None) -> None:
    """The choice of a router sorted by expert, and the tokens' rows copied into that order.

    ids: (T, top_k) int32, the experts of every token (moe_few_tokens writes them, any router may); an id outside
    0 .. E - 1 chooses none.  offsets: (E + 1,) int32, receives where each expert's rows start.  rows: (T, top_k) int32,
    receives the row of every slot (-1: none); slots of one expert keep their order.
    X: (T, H) fp32, fp16 or bf16; Xs: the same type and width, at least T * top_k rows, receives Xs[rows[t, j]] = X[t]
    (rows from offsets[E] on stay as they are).  X=None and Xs=None: the order alone.
    Limits: E <= 4096, top_k <= 128, T * top_k <= 2^31 - 32768.
    """
    ids_ptr, T, k, here = _slots(ids, "ids")
    off_ptr, E, off_on = _offsets(offsets)
    rows_ptr, rows_on = _packed(rows, "rows", "int32", (T, k))
    x_on = xs_on = here
    x_ptr = xs_ptr = 0
    H, x_type, ldx, ldxs = 0, GEMM_DTYPE_F32, 1, 1
    if X is not None or Xs is not None:
        x_ptr, ldx, x_rows, H, x_type, x_on = _placed(X, "X", _FLOATS)
        xs_ptr, ldxs, xs_rows, xs_cols, xs_type, xs_on = _placed(Xs, "Xs", _FLOATS)
        if xs_type != x_type:
            raise TypeError("X and Xs must have one type")
        if x_rows != T or xs_cols != H or xs_rows < T * k:
            raise ValueError(f"shape mismatch ids{(T, k)} X{tuple(X.shape)} Xs{tuple(Xs.shape)} (at least T * top_k rows)")
    if not here == off_on == rows_on == x_on == xs_on == _device_now():
        _elsewhere(here, off_on, rows_on, x_on, xs_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack13(T, E, k, H, ids_ptr, x_ptr, x_type, ldx, xs_ptr, ldxs, off_ptr, rows_ptr, on)
    st = (_lib or lib()).gemm_call_words(0, words, 13)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_moe_dispatch")


def moe_combine(Ys, rows, Y, weights=None, *, stream=None) -> None:
    """Y[t] = sum_j weights[t, j] * Ys[rows[t, j]], added in fp32 in the order of the slots.

    Ys: (R, H), Y: (T, H), both fp32, fp16 or bf16.  rows: (T, top_k) int32 (moe_dispatch); a slot without a row adds
    nothing.  weights: (T, top_k) fp32, or None: ones, which also makes this the gradient of moe_dispatch's copy.
    """
    ys_ptr, ldys, R, H, y_type, ys_on = _placed(Ys, "Ys", _FLOATS)
    y_ptr, ldy, T, y_cols, code, here = _placed(Y, "Y", _FLOATS)
    rows_ptr, r_T, k, rows_on = _slots(rows, "rows")
    if code != y_type:
        raise TypeError("Ys and Y must have one type")
    if r_T != T or y_cols != H:
        raise ValueError(f"shape mismatch Ys{tuple(Ys.shape)} rows{tuple(rows.shape)} Y{tuple(Y.shape)}")
    w_ptr, w_on = (0, here) if weights is None else _packed(weights, "weights", "float32", (T, k))
    if not here == ys_on == rows_on == w_on == _device_now():
        _elsewhere(here, ys_on, rows_on, w_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack12(T, k, H, R, ys_ptr, y_type, ldys, rows_ptr, w_ptr, y_ptr, ldy, on)
    st = (_lib or lib()).gemm_call_words(1, words, 12)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_moe_combine")


def moe_combine_grad(dY, Ys, rows, weights, dYs, dweights, *, stream=None) -> None:
    """The gradient of moe_combine: dYs[rows[t, j]] = weights[t, j] * dY[t], dweights[t, j] = <dY[t], Ys[rows[t, j]]>.

    dY: (T, H), Ys and dYs: (R, H), one type; rows: (T, top_k) int32; weights and dweights: (T, top_k) fp32.  A slot
    without a row gets dweights 0; rows of dYs that no slot names stay as they are.
    """
    dy_ptr, lddy, T, H, code, here = _placed(dY, "dY", _FLOATS)
    ys_ptr, ldys, R, ys_cols, ys_type, ys_on = _placed(Ys, "Ys", _FLOATS)
    dys_ptr, lddys, dys_rows, dys_cols, dys_type, dys_on = _placed(dYs, "dYs", _FLOATS)
    rows_ptr, r_T, k, rows_on = _slots(rows, "rows")
    if ys_type != code or dys_type != code:
        raise TypeError("dY, Ys and dYs must have one type")
    if r_T != T or ys_cols != H or (dys_rows, dys_cols) != (R, H):
        raise ValueError(f"shape mismatch dY{tuple(dY.shape)} Ys{tuple(Ys.shape)} rows{tuple(rows.shape)} dYs{tuple(dYs.shape)}")
    w_ptr, w_on = _packed(weights, "weights", "float32", (T, k))
    dw_ptr, dw_on = _packed(dweights, "dweights", "float32", (T, k))
    if not here == ys_on == dys_on == rows_on == w_on == dw_on == _device_now():
        _elsewhere(here, ys_on, dys_on, rows_on, w_on, dw_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack15(T, k, H, R, dy_ptr, code, lddy, ys_ptr, ldys, rows_ptr, w_ptr, dys_ptr, lddys, dw_ptr, on)
    st = (_lib or lib()).gemm_call_words(2, words, 15)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_moe_combine_grad")


def gemm_grouped(A, B, C, offsets, alpha: float = 1.0, beta: float = 0.0, *, b_trans: bool = True, stream=None) -> None:
    """C[r] = alpha * A[r] @ op(B[e]) + beta * C[r] for the rows offsets[e] <= r < offsets[e + 1] of every expert e.

    A: (R, K), C: (R, N).  B: (E, N, K), op(B) = B^T, or (E, K, N) with b_trans=False.  A and B both fp16 or both bf16,
    C fp32, fp16 or bf16.  offsets: (E + 1,) int32 on the device, not descending, from 0 to R (moe_dispatch); rows of C
    that no expert has stay as they are.  A's and B's rows start on 16-byte boundaries (row strides multiples of 8).
    So y = x W^T of every expert takes W as it is, and dx = dy W the same W with b_trans=False.
    """
    a_ptr, lda, R, K, a_type, here = _placed(A, "A", _HALFS)
    b_ptr, ldb, stride_b, E, b_rows, b_cols, b_type, b_on = _expert_mats(B, "B", _HALFS)
    c_ptr, ldc, c_rows, N, c_type, c_on = _placed(C, "C", _FLOATS)
    off_ptr, off_E, off_on = _offsets(offsets)
    if a_type != b_type:
        raise TypeError("A and B must both be float16 or both bfloat16")
    if c_rows != R or off_E != E or (b_rows, b_cols) != ((N, K) if b_trans else (K, N)):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)} offsets{tuple(offsets.shape)}")
    if not here == b_on == c_on == off_on == _device_now():
        _elsewhere(here, b_on, c_on, off_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack_grouped(E, R, N, K, alpha, a_ptr, lda, b_ptr, ldb, stride_b, a_type, 1 if b_trans else 0, beta, c_ptr, c_type,
                          ldc, off_ptr, on)
    st = (_lib or lib()).gemm_call_words(3, words, 18)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_grouped_f32acc")


def gemm_grouped_wgrad(A, B, C, offsets, alpha: float = 1.0, beta: float = 0.0, *, stream=None) -> None:
    """C[e] = alpha * A[rows of e]^T @ B[rows of e] + beta * C[e] for every expert e (rows offsets[e] .. offsets[e + 1] - 1).

    A: (R, M), B: (R, N), both fp16 or both bf16; C: (E, M, N) fp32, fp16 or bf16.  An expert without rows gets
    beta * C[e].  So dW = dy^T x of every expert takes dy as A and x as B.  offsets and alignment as for gemm_grouped.
    """
    a_ptr, lda, R, M, a_type, here = _placed(A, "A", _HALFS)
    b_ptr, ldb, b_rows, N, b_type, b_on = _placed(B, "B", _HALFS)
    c_ptr, ldc, stride_c, E, c_rows, c_cols, c_type, c_on = _expert_mats(C, "C", _FLOATS)
    off_ptr, off_E, off_on = _offsets(offsets)
    if a_type != b_type:
        raise TypeError("A and B must both be float16 or both bfloat16")
    if b_rows != R or off_E != E or (c_rows, c_cols) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)} offsets{tuple(offsets.shape)}")
    if not here == b_on == c_on == off_on == _device_now():
        _elsewhere(here, b_on, c_on, off_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack_wgrad(E, R, M, N, alpha, a_ptr, lda, b_ptr, ldb, a_type, beta, c_ptr, c_type, ldc, stride_c, off_ptr, on)
    st = (_lib or lib()).gemm_call_words(4, words, 17)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_grouped_wgrad_f32acc")


def _kept(Q, S, q_name, s_name, rows, cols):
    """(pointer, row stride, type, device) of Q and (pointer, row stride, device) of S, a rows x cols matrix in 8 bits (layout "rows")."""
    q_ptr, ldq, q_rows, q_cols, code, q_on = _placed(Q, q_name, _FP8S)
    s_ptr, lds, s_rows, s_cols, _, s_on = _placed(S, s_name, _F32)
    if q_rows != rows or q_cols != cols or s_rows != (cols + 127) // 128 or s_cols != rows:
        raise ValueError(f"{q_name}{tuple(Q.shape)} and {s_name}{tuple(S.shape)} do not hold {rows} x {cols} in layout 'rows'")
    return q_ptr, ldq, code, q_on, s_ptr, lds, s_on


def _same(t, name, rows, cols, code):
    """(pointer, row stride, device) of a rows x cols matrix of type `code`."""
    ptr, ld, r, c, _, device = _placed(t, name, (code,))
    if r != rows or c != cols:
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(t.shape)}")
    return ptr, ld, device


def fp8_gated_act(G, U, H, GQ, GS, UQ=None, US=None, act: int = GEMM_ACT_SILU, *, stream=None) -> None:
    """H = act(G) * U, and G and U kept in 8 bits for fp8_gated_act_grad.

    G, U, H: (rows, cols), one type, fp32, fp16 or bf16.  GQ, GS and UQ, US receive what fp8_quantize makes of G and U
    with layout "rows" (fp8_empty() makes fitting pairs).  U=None (and UQ=US=None): H = act(G).  act: any GEMM_ACT_*.
    An infinity makes the scale of its block of 128 infinite; what the backward pass computes from that block is NaN.
    """
    g_ptr, ldg, rows, cols, code, here = _placed(G, "G", _FLOATS)
    h_ptr, ldh, h_on = _same(H, "H", rows, cols, code)
    gq_ptr, ldgq, q_type, gq_on, gs_ptr, ldgs, gs_on = _kept(GQ, GS, "GQ", "GS", rows, cols)
    u_ptr = uq_ptr = us_ptr = 0
    ldu = lduq = ldus = 1
    u_on = uq_on = us_on = here
    if U is not None:
        u_ptr, ldu, u_on = _same(U, "U", rows, cols, code)
        uq_ptr, lduq, uq_type, uq_on, us_ptr, ldus, us_on = _kept(UQ, US, "UQ", "US", rows, cols)
        if uq_type != q_type:
            raise TypeError("GQ and UQ must have one type")
    elif UQ is not None or US is not None:
        raise ValueError("UQ and US are for a gate: without U they must be None")
    if not here == h_on == gq_on == gs_on == u_on == uq_on == us_on == _device_now():
        _elsewhere(here, h_on, gq_on, gs_on, u_on, uq_on, us_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack20(rows, cols, g_ptr, ldg, u_ptr, ldu, code, h_ptr, ldh, gq_ptr, ldgq, gs_ptr, ldgs, uq_ptr, lduq, us_ptr, ldus,
                    q_type, act, on)
    st = (_lib or lib()).gemm_call_words(5, words, 20)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp8_gated_act")


def fp8_gated_act_grad(dH, GQ, GS, UQ, US, dG, dU, H=None, act: int = GEMM_ACT_SILU, *, stream=None) -> None:
    """The backward pass of fp8_gated_act from its 8-bit copies g' = GQ * GS and u' = UQ * US.

    dG = dH * u' * act'(g'), dU = dH * act(g'), and, with H given, H = act(g') * u' again (for the gradient of the
    weights that H is multiplied by).  dH, dG, dU, H: (rows, cols), one type, fp32, fp16 or bf16.
    Without a gate UQ, US and dU are None, and u' is 1.
    """
    dh_ptr, lddh, rows, cols, code, here = _placed(dH, "dH", _FLOATS)
    gq_ptr, ldgq, q_type, gq_on, gs_ptr, ldgs, gs_on = _kept(GQ, GS, "GQ", "GS", rows, cols)
    dg_ptr, lddg, dg_on = _same(dG, "dG", rows, cols, code)
    uq_ptr = us_ptr = du_ptr = h_ptr = 0
    lduq = ldus = lddu = ldh = 1
    uq_on = us_on = du_on = h_on = here
    if UQ is not None:
        uq_ptr, lduq, uq_type, uq_on, us_ptr, ldus, us_on = _kept(UQ, US, "UQ", "US", rows, cols)
        if uq_type != q_type:
            raise TypeError("GQ and UQ must have one type")
        du_ptr, lddu, du_on = _same(dU, "dU", rows, cols, code)
    elif US is not None or dU is not None:
        raise ValueError("US and dU are for a gate: without UQ they must be None")
    if H is not None:
        h_ptr, ldh, h_on = _same(H, "H", rows, cols, code)
    if not here == gq_on == gs_on == dg_on == uq_on == us_on == du_on == h_on == _device_now():
        _elsewhere(here, gq_on, gs_on, dg_on, uq_on, us_on, du_on, h_on)
    on = _raw_stream(here) if stream is None else stream.cuda_stream
    words = _pack22(rows, cols, dh_ptr, lddh, code, gq_ptr, ldgq, gs_ptr, ldgs, uq_ptr, lduq, us_ptr, ldus, q_type, dg_ptr, lddg,
                    du_ptr, lddu, h_ptr, ldh, act, on)
    st = (_lib or lib()).gemm_call_words(6, words, 22)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fp8_gated_act_grad")


def tune_set(entries) -> None:
    """Install a tuning table: an iterable of dicts (or TuneEntry) with keys
    path, M, N, K, variant, bn, splits.  An empty iterable clears the table."""
    rows = [e if isinstance(e, TuneEntry) else TuneEntry(**{k: int(e.get(k, 0)) for k, _ in TuneEntry._fields_})
            for e in entries]
    arr = (TuneEntry * max(1, len(rows)))(*rows)
    st = lib().gemm_tune_set(arr, len(rows))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_tune_set")


def tune_get() -> list:
    """The installed tuning table as a list of dicts."""
    n = lib().gemm_tune_get(None, 0)
    arr = (TuneEntry * max(1, n))()
    n = lib().gemm_tune_get(arr, n)
    return [arr[i].as_dict() for i in range(n)]


def default_tuning_path() -> str:
    """The tuning table shipped for GB300 (written by ``autotune`` on one)."""
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "tuning", "gb300.json")


def load_tuning(path: str) -> int:
    """Install the table stored by ``autotune`` in a JSON file; returns the entry count."""
    import json
    with open(path) as f:
        doc = json.load(f)
    tune_set(doc["entries"])
    return len(doc["entries"])


def watchdog_selftest(wait_ms: int = 20, stream=None) -> int:
    """Enqueue the watchdog probe (a wait that must time out after wait_ms); returns the status."""
    return int(lib().gemm_watchdog_selftest(int(wait_ms), _stream_handle(stream)))


def pipeline_stall_selftest_raw(M, N, K, A_ptr, B_ptr, C_ptr, wait_ms=5, stream_ptr=0) -> int:
    """Enqueue the single-CTA tensor-core GEMM with its TMA producer switched off
    and every wait limited to wait_ms (the waits must run out); returns the status."""
    return int(lib().gemm_pipeline_stall_selftest(int(M), int(N), int(K), ctypes.c_void_p(A_ptr),
                                                  ctypes.c_void_p(B_ptr), ctypes.c_void_p(C_ptr), int(wait_ms),
                                                  ctypes.c_void_p(stream_ptr)))


def fma_rate_probe(packed: bool = True, iters: int = 4096, stream=None) -> float:
    """FP32 FMAs per clock per SM of an 8 x 8 outer product in registers,
    measured with the packed two-wide FMA form gemm_f32 uses (packed=True)
    or with scalar FMAs."""
    out = ctypes.c_double(0.0)
    st = lib().gemm_fma_rate_probe(1 if packed else 0, int(iters), ctypes.byref(out), _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_fma_rate_probe")
    return float(out.value)


def tma_read_probe(clusters: int, multicast: bool = False, stages: int = 4, kblocks: int = 512,
                   region_mb: int = 24, stream=None) -> dict:
    """Bytes per SM clock that each CTA receives through TMA (median over the
    CTAs) and the total GB/s, for `clusters` clusters of 2 CTAs streaming
    `kblocks` 32 KB stages (the 64-wide k block of a 256-row panel of a
    K-major FP16 operand with 4096-element rows, two 128-row boxes) from a
    `region_mb` MB region (24 MB stays in L2), each CTA loading its own copy
    or (multicast=True) one box per CTA multicast to both."""
    per_sm, total = ctypes.c_double(0.0), ctypes.c_double(0.0)
    st = lib().gemm_tma_read_probe(int(clusters), 1 if multicast else 0, int(stages), int(kblocks), int(region_mb),
                                   ctypes.byref(per_sm), ctypes.byref(total), _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_tma_read_probe")
    return {"bytes_per_clock_per_sm": float(per_sm.value), "total_gbs": float(total.value)}


def tma_read_probe_raw(clusters, multicast, stages, kblocks, region_mb, per_sm_ptr, total_ptr, stream_ptr=0) -> int:
    """Direct C-ABI call of gemm_tma_read_probe (pointers: addresses of doubles, or 0)."""
    dp = ctypes.POINTER(ctypes.c_double)
    return int(lib().gemm_tma_read_probe(int(clusters), int(multicast), int(stages), int(kblocks), int(region_mb),
                                         ctypes.cast(per_sm_ptr, dp), ctypes.cast(total_ptr, dp),
                                         ctypes.c_void_p(stream_ptr)))


def fma_rate_probe_raw(packed, iters, out_ptr, stream_ptr=0) -> int:
    """Direct C-ABI call of gemm_fma_rate_probe (out_ptr: address of a double, or 0)."""
    return int(lib().gemm_fma_rate_probe(int(packed), int(iters), ctypes.cast(out_ptr, ctypes.POINTER(ctypes.c_double)),
                                         ctypes.c_void_p(stream_ptr)))


def tc_rate_probe(iters: int = 4096, stream=None) -> float:
    """The tensor core's dense FP16/BF16 rate per SM in FLOP per clock,
    measured by timing back-to-back MMAs on every SM (median over the SMs)."""
    out = ctypes.c_double(0.0)
    st = lib().gemm_tc_rate_probe(int(iters), ctypes.byref(out), _stream_handle(stream))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_tc_rate_probe")
    return float(out.value)


def check(stream=None) -> int:
    """Synchronise the stream and return the watchdog status (GEMM_OK or GEMM_ERR_TIMEOUT)."""
    return int(lib().gemm_check(_stream_handle(stream)))
