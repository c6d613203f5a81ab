"""ctypes binding of libdense_gemm_row.so (include/dense_gemm_row.h).

Argument marshalling only: every step of the computation runs in the CUDA
library. Importing this module loads the library and raises ImportError when
it has not been built; there is no fallback.

Two layers:

* ``gemm_f32 / gemm_bf16 / gemm_f16 / gemm_s8(M, N, K, alpha, A, lda, B, ldb,
  beta, C, ldc, stream=None)`` mirror the C entry points. A, B and C are raw
  device addresses (int) or tensors (their ``data_ptr()`` is passed). ``stream``
  is a raw ``cudaStream_t`` (int), a ``torch.cuda.Stream``, or None for torch's
  current stream. A non-zero status raises :class:`GemmError`.
* ``gemm(A, B, C, alpha, beta)`` takes 2-D CUDA tensors with unit column stride
  (row stride = leading dimension), picks the entry point from A's dtype and
  runs on torch's current stream.

The extended entry points (strided-batched GEMM with transposed operands) have
the same two layers: ``gemm_f32_ex / gemm_bf16_ex / gemm_f16_ex / gemm_s8_ex(
opA, opB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
strideC, batch, stream=None)`` (opX: OP_N or OP_T) and ``gemm_batched(A, B, C,
alpha, beta, trans_a=False, trans_b=False)`` for 3-D tensors (a 2-D operand,
or one expanded along the batch with stride 0, is shared by every entry).

The linear-layer operators have one function each for CUDA tensors:
``gemm_epilogue`` (a product with bias, activation and residual in its
epilogue), ``gemm_dact`` and ``act_grad`` (the gradient at the pre-activation),
``gemm_gated`` (two projections and their gated product), ``gemm_gated_dact``,
``quantise_blocks`` (8-bit operands with a scale for each block of 128),
``rms_norm``, ``layer_norm`` and their gradients ``rms_norm_grad`` and
``layer_norm_grad``. The dtypes pick the C entry point. They
check shapes, dtypes, strides and devices before the call and write into the
tensors they are given.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdense_gemm_row.so")

STATUS = {
    0: "GEMM_OK",
    1: "GEMM_ERR_INVALID_VALUE",
    2: "GEMM_ERR_UNSUPPORTED_LAYOUT",
    3: "GEMM_ERR_LAUNCH",
    4: "GEMM_ERR_DEVICE",
    5: "GEMM_ERR_TIMEOUT",
    6: "GEMM_ERR_TOO_LARGE",
}

# Every function include/dense_gemm_row.h declares.
EXPORTED = ("gemm_f32", "gemm_bf16", "gemm_f16", "gemm_s8", "gemm_u8", "gemm_f16_f16",
            "gemm_bf16_bf16", "gemm_tf32", "gemm_f64", "gemm_f32_ex", "gemm_bf16_ex",
            "gemm_f16_ex", "gemm_s8_ex", "gemm_s8_noalloc", "gemm_status_string",
            "gemm_check_device_error", "gemm_selftest_wait_timeout", "gemm_last_launch_error",
            "gemm_peak_ffma", "gemm_peak_tc_f16", "gemm_pool_usage", "gemm_version",
            "gemm_bf16_epi", "gemm_f16_epi", "gemm_e4m3_bf16_epi", "gemm_e4m3_f16_epi",
            "gemm_bf16_dact", "gemm_f16_dact", "gemm_act_grad_bf16", "gemm_act_grad_f16",
            "gemm_rms_norm_bf16", "gemm_rms_norm_f16", "gemm_rms_norm_bf16_e4m3",
            "gemm_rms_norm_f16_e4m3", "gemm_rms_norm_grad_bf16", "gemm_rms_norm_grad_f16",
            "gemm_bf16_gated", "gemm_f16_gated", "gemm_bf16_gated_dact", "gemm_f16_gated_dact",
            "gemm_e4m3_bf16_gated", "gemm_e4m3_f16_gated", "gemm_e4m3_block_bf16_epi",
            "gemm_e4m3_block_f16_epi", "gemm_quantise_bf16_e4m3", "gemm_quantise_f16_e4m3",
            "gemm_layer_norm_bf16", "gemm_layer_norm_f16", "gemm_layer_norm_grad_bf16",
            "gemm_layer_norm_grad_f16")

OP_N, OP_T = 0, 1  # gemm_op_t


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = int(status)
        msg = f"{where}: {STATUS.get(self.status, self.status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m dense_gemm_row_gb300.build` "
            "(or __graft_entry__.build()). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    f32, i32 = ctypes.c_float, ctypes.c_int32
    for name in ("gemm_f32", "gemm_bf16", "gemm_f16", "gemm_f16_f16", "gemm_bf16_bf16",
                 "gemm_tf32"):
        fn = getattr(lib, name)
        fn.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        fn.restype = ctypes.c_int
    f64 = ctypes.c_double
    lib.gemm_f64.argtypes = [i64, i64, i64, f64, vp, i64, vp, i64, f64, vp, i64, vp]
    lib.gemm_f64.restype = ctypes.c_int
    for name in ("gemm_s8", "gemm_s8_noalloc", "gemm_u8"):
        fn = getattr(lib, name)
        fn.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp]
        fn.restype = ctypes.c_int
    op = ctypes.c_int
    for name, sc in (("gemm_f32_ex", f32), ("gemm_bf16_ex", f32), ("gemm_f16_ex", f32),
                     ("gemm_s8_ex", i32)):
        fn = getattr(lib, name)
        fn.argtypes = [op, op, i64, i64, i64, sc, vp, i64, i64, vp, i64, i64, sc, vp, i64, i64,
                       i64, vp]
        fn.restype = ctypes.c_int
    lib.gemm_status_string.argtypes = [ctypes.c_int]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_check_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.gemm_check_device_error.restype = ctypes.c_int
    lib.gemm_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
    lib.gemm_selftest_wait_timeout.restype = ctypes.c_int
    lib.gemm_last_launch_error.argtypes = []
    lib.gemm_last_launch_error.restype = ctypes.c_char_p
    lib.gemm_peak_ffma.argtypes = [i32, vp, ctypes.POINTER(f64), vp]
    lib.gemm_peak_ffma.restype = ctypes.c_int
    lib.gemm_peak_tc_f16.argtypes = [i32, ctypes.POINTER(f64), vp]
    lib.gemm_peak_tc_f16.restype = ctypes.c_int
    lib.gemm_version.argtypes = []
    lib.gemm_version.restype = ctypes.c_int
    lib.gemm_pool_usage.argtypes = [ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.c_int]
    lib.gemm_pool_usage.restype = ctypes.c_int
    for fmt in ("bf16", "f16"):
        layer = {
            f"gemm_{fmt}_epi": [op, op, i64, i64, i64, f32, vp, i64, vp, i64, op, vp, vp, i64,
                                vp, i64, vp, i64, vp],
            f"gemm_e4m3_{fmt}_epi": [i64, i64, i64, f32, vp, i64, vp, vp, i64, vp, op, vp, vp,
                                     i64, vp, i64, vp, i64, vp],
            f"gemm_{fmt}_dact": [op, op, i64, i64, i64, f32, vp, i64, vp, i64, op, vp, i64, vp,
                                 i64, vp, vp],
            f"gemm_act_grad_{fmt}": [i64, i64, op, vp, i64, vp, i64, vp, i64, vp, vp],
            f"gemm_rms_norm_{fmt}": [i64, i64, f32, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp,
                                     vp],
            f"gemm_rms_norm_{fmt}_e4m3": [i64, i64, f32, vp, i64, vp, i64, vp, vp, i64, vp, i64,
                                          vp, vp, vp],
            f"gemm_rms_norm_grad_{fmt}": [i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64,
                                          vp, vp],
            f"gemm_{fmt}_gated": [op, op, i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, op, vp,
                                  vp, vp, i64, vp, i64, vp, i64, vp],
            f"gemm_e4m3_{fmt}_gated": [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, i64, vp,
                                       i64, vp, i64, op, vp, vp, vp, i64, vp, i64, vp, i64, vp],
            f"gemm_e4m3_block_{fmt}_epi": [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, i64,
                                           op, vp, vp, i64, vp, i64, vp, i64, vp],
            f"gemm_quantise_{fmt}_e4m3": [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp],
            f"gemm_{fmt}_gated_dact": [op, op, i64, i64, i64, f32, vp, i64, vp, i64, op, vp, i64,
                                       vp, i64, vp, i64, vp, i64, vp, vp, vp],
            f"gemm_layer_norm_{fmt}": [i64, i64, f32, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64,
                                       vp, vp, vp],
            f"gemm_layer_norm_grad_{fmt}": [i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp,
                                            i64, vp, vp, vp],
        }
        for name, argtypes in layer.items():
            fn = getattr(lib, name)
            fn.argtypes = argtypes
            fn.restype = ctypes.c_int
    return lib


lib = _load()


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(s) -> int | None:
    if s is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != 0:
        detail = lib.gemm_last_launch_error().decode() if status == 3 else ""
        raise GemmError(status, where, detail)


def gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_f32(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                        _stream(stream)), "gemm_f32")


def gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_bf16(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                         _stream(stream)), "gemm_bf16")


def gemm_f16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_f16(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                        _stream(stream)), "gemm_f16")


def gemm_s8(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_s8(M, N, K, int(alpha), _addr(A), lda, _addr(B), ldb, int(beta), _addr(C),
                       ldc, _stream(stream)), "gemm_s8")


def gemm_u8(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_u8(M, N, K, int(alpha), _addr(A), lda, _addr(B), ldb, int(beta), _addr(C),
                       ldc, _stream(stream)), "gemm_u8")


def gemm_f16_f16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_f16_f16(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                            _stream(stream)), "gemm_f16_f16")


def gemm_bf16_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_bf16_bf16(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                              _stream(stream)), "gemm_bf16_bf16")


def gemm_tf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_tf32(M, N, K, alpha, _addr(A), lda, _addr(B), ldb, beta, _addr(C), ldc,
                         _stream(stream)), "gemm_tf32")


def gemm_f64(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    _check(lib.gemm_f64(M, N, K, float(alpha), _addr(A), lda, _addr(B), ldb, float(beta),
                        _addr(C), ldc, _stream(stream)), "gemm_f64")


def gemm_s8_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None):
    """gemm_s8 on the library's fixed scratch array: allocates no device memory.
    Problems needing more than 64 MiB of widened operands raise GemmError
    (GEMM_ERR_TOO_LARGE); calls that overlap on the GPU race on the array."""
    _check(lib.gemm_s8_noalloc(M, N, K, int(alpha), _addr(A), lda, _addr(B), ldb, int(beta),
                               _addr(C), ldc, _stream(stream)), "gemm_s8_noalloc")


def _ex(name, cast):
    def call(opA, opB, M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc, strideC,
             batch, stream=None):
        _check(getattr(lib, name)(int(opA), int(opB), M, N, K, cast(alpha), _addr(A), lda,
                                  strideA, _addr(B), ldb, strideB, cast(beta), _addr(C), ldc,
                                  strideC, batch, _stream(stream)), name)
    call.__name__ = name
    call.__doc__ = (f"{name}: strided-batched C_b = alpha*op(A_b)*op(B_b) + beta*C_b "
                    "(include/dense_gemm_row.h).")
    return call


gemm_f32_ex = _ex("gemm_f32_ex", float)
gemm_bf16_ex = _ex("gemm_bf16_ex", float)
gemm_f16_ex = _ex("gemm_f16_ex", float)
gemm_s8_ex = _ex("gemm_s8_ex", int)


def peak_ffma(iters, sink, stream=None) -> float:
    """Enqueue the packed-FP32-FMA peak microbenchmark; returns its flop count."""
    f = ctypes.c_double(0.0)
    _check(lib.gemm_peak_ffma(int(iters), _addr(sink), ctypes.byref(f), _stream(stream)),
           "gemm_peak_ffma")
    return f.value


def peak_tc_f16(iters, stream=None) -> float:
    """Enqueue the tcgen05 kind::f16 peak microbenchmark; returns its flop count."""
    f = ctypes.c_double(0.0)
    _check(lib.gemm_peak_tc_f16(int(iters), ctypes.byref(f), _stream(stream)), "gemm_peak_tc_f16")
    return f.value


def pool_usage(reset_high: bool = False) -> tuple[int, int]:
    """(high-water mark of bytes in use, bytes reserved) of the library's memory
    pool on the current device; reset_high clears the mark after reading."""
    used = ctypes.c_int64(0)
    reserved = ctypes.c_int64(0)
    _check(lib.gemm_pool_usage(ctypes.byref(used), ctypes.byref(reserved), int(reset_high)),
           "gemm_pool_usage")
    return used.value, reserved.value


def check_device_error() -> int:
    """Reads and clears the device error word; raises GemmError(GEMM_ERR_TIMEOUT)
    if a kernel gave up a bounded wait. Returns the raw word otherwise (0)."""
    w = ctypes.c_uint32(0)
    st = lib.gemm_check_device_error(ctypes.byref(w))
    if st != 0:
        raise GemmError(st, f"device error word 0x{w.value:08x}")
    return int(w.value)


def _ld(t, name) -> int:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[0] > 0 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs unit column stride (row-major)")
    return max(int(t.stride(0)), int(t.shape[1]), 1)


def gemm(A, B, C, alpha=1.0, beta=0.0, stream=None, tf32=False):
    """C = alpha*A*B + beta*C for 2-D CUDA tensors; the dtypes select the entry
    point: float32 -> gemm_f32 (gemm_tf32 with tf32=True), float64 -> gemm_f64,
    bfloat16 / float16 with a float32 C -> gemm_bf16 / gemm_f16, with a C of the
    inputs' dtype -> gemm_bf16_bf16 / gemm_f16_f16, int8 -> gemm_s8 and uint8
    -> gemm_u8 (C int32)."""
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError("gemm: shapes do not chain (A: MxK, B: KxN, C: MxN)")
    if A.dtype != B.dtype:
        raise TypeError("gemm: A and B must share a dtype")
    fns = {torch.float32: (gemm_tf32 if tf32 else gemm_f32, torch.float32),
           torch.float64: (gemm_f64, torch.float64),
           torch.bfloat16: (gemm_bf16, torch.float32), torch.float16: (gemm_f16, torch.float32),
           torch.int8: (gemm_s8, torch.int32), torch.uint8: (gemm_u8, torch.int32)}
    if A.dtype not in fns:
        raise TypeError(f"gemm: unsupported dtype {A.dtype}")
    fn, c_dtype = fns[A.dtype]
    if A.dtype in (torch.bfloat16, torch.float16) and C.dtype == A.dtype:
        fn, c_dtype = (gemm_bf16_bf16 if A.dtype == torch.bfloat16 else gemm_f16_f16), A.dtype
    if C.dtype != c_dtype:
        raise TypeError(f"gemm: C must be {c_dtype} for {A.dtype} inputs")
    fn(M, N, K, alpha, A, _ld(A, "A"), B, _ld(B, "B"), beta, C, _ld(C, "C"), stream)
    return C


def _mat(t, name):
    """(matrix stride, row stride) of a 2-D or 3-D operand with unit column
    stride; a 2-D operand is one matrix shared by every batch entry."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be 2-D or 3-D")
    rows, cols = t.shape[-2], t.shape[-1]
    if rows > 0 and cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} needs unit column stride (row-major)")
    ld = max(int(t.stride(-2)), int(cols), 1)
    mstride = int(t.stride(0)) if t.dim() == 3 and t.shape[0] > 1 else 0
    return mstride, ld


def gemm_batched(A, B, C, alpha=1.0, beta=0.0, trans_a=False, trans_b=False, stream=None):
    """C[b] = alpha * op(A[b]) * op(B[b]) + beta * C[b] for CUDA tensors.

    C is (batch, M, N). A is (batch, M, K), or (batch, K, M) with trans_a; B is
    (batch, K, N), or (batch, N, K) with trans_b. A 2-D A or B (or one expanded
    along the batch, stride 0) is shared by every entry. Rows must have unit
    column stride; row and matrix strides are passed through. dtypes as gemm()."""
    import torch
    if C.dim() != 3:
        raise ValueError("gemm_batched: C must be 3-D (batch, M, N)")
    batch, M, N = C.shape
    K = A.shape[-2] if trans_a else A.shape[-1]
    a_rows = A.shape[-1] if trans_a else A.shape[-2]
    b_k = B.shape[-1] if trans_b else B.shape[-2]
    b_n = B.shape[-2] if trans_b else B.shape[-1]
    if a_rows != M or b_k != K or b_n != N:
        raise ValueError("gemm_batched: shapes do not chain")
    for t, name in ((A, "A"), (B, "B")):
        if t.dim() == 3 and t.shape[0] not in (1, batch):
            raise ValueError(f"gemm_batched: {name} has {t.shape[0]} matrices, C {batch}")
    if A.dtype != B.dtype:
        raise TypeError("gemm_batched: A and B must share a dtype")
    fns = {torch.float32: (gemm_f32_ex, torch.float32),
           torch.bfloat16: (gemm_bf16_ex, torch.float32),
           torch.float16: (gemm_f16_ex, torch.float32), torch.int8: (gemm_s8_ex, torch.int32)}
    if A.dtype not in fns:
        raise TypeError(f"gemm_batched: unsupported dtype {A.dtype}")
    fn, c_dtype = fns[A.dtype]
    if C.dtype != c_dtype:
        raise TypeError(f"gemm_batched: C must be {c_dtype} for {A.dtype} inputs")
    sa, lda = _mat(A, "A")
    sb, ldb = _mat(B, "B")
    sc, ldc = _mat(C, "C")
    fn(OP_T if trans_a else OP_N, OP_T if trans_b else OP_N, M, N, K, alpha, A, lda, sa, B, ldb,
       sb, beta, C, ldc, sc, batch, stream)
    return C


# ------------------------------------------------------ linear-layer operators

_layers = None


def _load_layers():
    """The marshalling module of the linear-layer operators, bound to the library.
    Loaded by the first call: it links against torch, which the raw entry points
    above do not need."""
    global _layers
    import importlib
    if not os.path.exists(os.path.join(_PKG, "_layers.so")):
        raise ImportError(
            "dense_gemm_row_gb300/_layers.so is missing: build it with "
            "`python -m dense_gemm_row_gb300.build` (or __graft_entry__.build()).")
    import torch  # noqa: F401  (the module links against torch's libraries)
    mod = importlib.import_module("dense_gemm_row_gb300._layers")
    for name in EXPORTED:
        if any(part in name for part in ("_epi", "gated", "quantise", "dact", "act_grad", "_norm")):
            mod.bind(name, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
    _layers = mod
    return mod


def gemm_epilogue(A, B, D, *, alpha=1.0, bias=None, act=None, residual=None, preact=None,
                  trans_a=False, trans_b=False, scale_a=None, scale_b=None, stream=None):
    """D = act(Z) + residual with Z = alpha * op(A) * op(B) + bias; returns D.

    A is M x K (K x M with trans_a), B is K x N (N x K with trans_b), D M x N.
    bfloat16 or float16 A, B: everything else has their dtype. float8_e4m3fn A
    and B (trans_b only: B stored N x K): D is bfloat16 or float16 and the
    product of row i and column j is scaled by scale_a[i] * scale_b[j] (float32
    vectors, either may be None), or, block by block of 128 along K, by
    scale_a[i, k // 128] * scale_b[j // 128, k // 128] (float32 matrices, as
    quantise_blocks writes them with rows=1 for A and rows=128 for B). bias (N values), residual (M x N, may be D
    itself) and act ("relu", "gelu", "gelu_tanh", "silu" or None) may be left
    out; preact (M x N), when given, receives Z for gemm_dact or act_grad.
    A and B start on 16-byte boundaries with row strides in whole 16-byte units."""
    st = (_layers or _load_layers()).gemm_epilogue(A, B, D, alpha, bias, act, residual, preact,
                                                   trans_a, trans_b, scale_a, scale_b, stream)
    if st:
        _check(st, "gemm_epilogue")
    return D


def gemm_dact(A, B, Z, dZ, *, act=None, alpha=1.0, dbias=None, trans_a=False, trans_b=False,
              stream=None):
    """dZ = (alpha * op(A) * op(B)) .* act'(Z), dbias = column sums of dZ; returns dZ.

    The product that carries a gradient back (A the output gradient of the next
    layer, B its weights) with the activation's derivative at the stored
    pre-activation Z (M x N; None without an activation) in its epilogue. dbias
    (N values of the same dtype) may be None. dZ may be Z itself."""
    st = (_layers or _load_layers()).gemm_dact(A, B, Z, dZ, act, alpha, dbias, trans_a, trans_b,
                                               stream)
    if st:
        _check(st, "gemm_dact")
    return dZ


def act_grad(dD, Z, dZ, *, act=None, dbias=None, stream=None):
    """dZ = dD .* act'(Z), dbias = column sums of dZ; returns dZ.

    gemm_dact for an output gradient that is already in memory. Without an
    activation Z may be None, and dZ too when only dbias is wanted. dZ may be
    dD or Z itself."""
    st = (_layers or _load_layers()).act_grad(dD, Z, dZ, act, dbias, stream)
    if st:
        _check(st, "act_grad")
    return dZ


def rms_norm(X, Y, *, weight=None, residual=None, h=None, scale=None, rstd=None, eps=1e-6,
             stream=None):
    """Y = H / rms(H) * weight per row with H = X + residual; returns Y.

    X is rows x cols, bfloat16 or float16; weight (cols values), residual and h
    (which receives H) have its dtype. Y has it too, or is float8_e4m3fn with
    one scale per row written to scale (float32, required then): Y stands for
    Y * scale[:, None], which gemm_epilogue takes as A and scale_a. rstd
    (float32, rows values), when given, receives 1 / rms for rms_norm_grad."""
    st = (_layers or _load_layers()).rms_norm(X, Y, weight, residual, h, scale, rstd, eps, stream)
    if st:
        _check(st, "rms_norm")
    return Y


def rms_norm_grad(dY, H, rstd, dX, *, weight=None, dh=None, dweight=None, stream=None):
    """The gradient of rms_norm: dX (of X and of the residual alike), plus dh,
    the gradient that reaches H past the norm; dweight (cols values) receives
    the weight's gradient. H and rstd are those of the forward call. dX may be
    dY or dh itself. Returns dX."""
    st = (_layers or _load_layers()).rms_norm_grad(dY, H, rstd, dX, weight, dh, dweight, stream)
    if st:
        _check(st, "rms_norm_grad")
    return dX


def gemm_gated(A, Bg, Bu, D, *, act="silu", alpha=1.0, bias_gate=None, bias_up=None, gate=None,
               up=None, trans_a=False, trans_b=False, scale_a=None, scale_gate=None, scale_up=None,
               stream=None):
    """D = act(G) * U with G = alpha * op(A) * op(Bg) + bias_gate and
    U = alpha * op(A) * op(Bu) + bias_up, in one kernel; returns D.

    A is M x K (K x M with trans_a), Bg and Bu are K x N (N x K with trans_b), D
    M x N; all are bfloat16 or float16. bias_gate and bias_up (N values each) may be
    None; gate and up (M x N), when given, receive G and U for gemm_gated_dact; they
    and D are distinct. Bg and Bu may be parts of one matrix. float8_e4m3fn A, Bg and
    Bu (trans_b only) come with scales per block of 128: scale_a, scale_gate and
    scale_up as gemm_epilogue's float32 matrices. Layouts as gemm_epilogue."""
    st = (_layers or _load_layers()).gemm_gated(A, Bg, Bu, D, act, alpha, bias_gate, bias_up,
                                                gate, up, trans_a, trans_b, scale_a, scale_gate,
                                                scale_up, stream)
    if st:
        _check(st, "gemm_gated")
    return D


def quantise_blocks(X, Y, scale, *, rows=1, stream=None):
    """Y = X / scale in float8_e4m3fn with scale = max |X| / 448 over each block of
    `rows` (1 or 128) x 128 values; returns Y.

    X is bfloat16 or float16; scale is float32, ceil(M / rows) x ceil(N / 128) for an
    M x N X. rows=1 makes an A and scale_a for gemm_epilogue or gemm_gated, rows=128 a
    B and its scales; a product wants Y's rows in whole 16-byte units."""
    st = (_layers or _load_layers()).quantise_blocks(X, Y, scale, rows, stream)
    if st:
        _check(st, "quantise_blocks")
    return Y


def gemm_gated_dact(A, B, G, U, dG, dU, *, act="silu", alpha=1.0, dbias_gate=None, dbias_up=None,
                    trans_a=False, trans_b=False, stream=None):
    """The gradient of gemm_gated at its projections, from the product
    dD = alpha * op(A) * op(B) that carries it back (A the next layer's output
    gradient, B its weights): dG = dD * U * act'(G), dU = dD * act(G), and their
    column sums dbias_gate and dbias_up (N values each, either may be None). G and U
    are what gemm_gated stored; dG may be G itself, dU U. Returns (dG, dU)."""
    st = (_layers or _load_layers()).gemm_gated_dact(A, B, G, U, dG, dU, act, alpha, dbias_gate,
                                                     dbias_up, trans_a, trans_b, stream)
    if st:
        _check(st, "gemm_gated_dact")
    return dG, dU


def layer_norm(X, Y, *, weight=None, bias=None, residual=None, h=None, mean=None, rstd=None,
               eps=1e-5, stream=None):
    """Y = (H - mean) / sqrt(variance + eps) * weight + bias per row with
    H = X + residual; returns Y.

    X is rows x cols, bfloat16 or float16; everything else but the statistics has
    its dtype: weight and bias (cols values), residual, h (which receives H) and Y.
    mean and rstd (float32, rows values), when given, receive the row's mean and
    1 / sqrt(variance + eps) for layer_norm_grad."""
    st = (_layers or _load_layers()).layer_norm(X, Y, weight, bias, residual, h, mean, rstd, eps,
                                                stream)
    if st:
        _check(st, "layer_norm")
    return Y


def layer_norm_grad(dY, H, mean, rstd, dX, *, weight=None, dh=None, dweight=None, dbias=None,
                    stream=None):
    """The gradient of layer_norm: dX (of X and of the residual alike), plus dh,
    the gradient that reaches H past the norm; dweight and dbias (cols values)
    receive the parameters' gradients. H, mean and rstd are those of the forward
    call. dX may be dY or dh itself. Returns dX."""
    st = (_layers or _load_layers()).layer_norm_grad(dY, H, mean, rstd, dX, weight, dh, dweight,
                                                     dbias, stream)
    if st:
        _check(st, "layer_norm_grad")
    return dX
