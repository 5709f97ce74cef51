"""ctypes binding of libdgemm.so: the C entry points under the same names.

Argument marshalling only -- every step of the product runs in the library's
CUDA kernels.  Pointers are integers (device addresses), `stream` is a
cudaStream_t handle as an integer (0 = legacy default stream).  Each function
returns the library's status code; see include/dgemm.h for the semantics.
"""
import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdgemm.so")

# Status codes (dgemm_status_t in include/dgemm.h).
OK = 0
ERR_INVALID_VALUE = 1
ERR_NULL_POINTER = 2
ERR_ALIAS = 3
ERR_UNSUPPORTED = 4
ERR_CUDA = 5
ERR_ARCH = 6
ERR_MISALIGNED = 7
ERR_INVALID_POINTER = 8
ERR_WATCHDOG = 9
ERR_SCRATCH_LIMIT = 10
NOALLOC_SCRATCH_BYTES = 16 << 20

TC_TF32 = 0
TC_3XTF32 = 1

OP_N = 0
OP_T = 1
PATH_SIMT, PATH_TF32, PATH_3XTF32, PATH_BF16, PATH_FP16, PATH_F8_E4M3, PATH_F8_E5M2 = range(7)
F8_E4M3 = 0
F8_E5M2 = 1

# Element types and activations of the feed-forward operators.
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = range(3)
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)

EXPORTED = ("gemm_f32_simt", "gemm_f32_tc", "gemm_bf16_tc", "dgemm_status_string",
            "dgemm_last_cuda_error", "dgemm_watchdog_status", "dgemm_version",
            "dgemm_kernel_launches", "gemm_f32_tc_noalloc", "gemm_f16_tc", "dgemm_gemm_ex",
            "gemm_f8_tc", "dgemm_layer_norm", "dgemm_layer_norm_backward", "dgemm_linear",
            "dgemm_linear_backward", "dgemm_gated_ffn", "dgemm_gated_ffn_backward",
            "dgemm_quantize_int8", "dgemm_linear_int8_workspace", "dgemm_linear_int8",
            "dgemm_gated_ffn_int8_workspace", "dgemm_gated_ffn_int8",
            "dgemm_orthogonalize_workspace", "dgemm_orthogonalize")

_lib = None


class LibraryMissing(RuntimeError):
    pass


def load():
    """Load libdgemm.so (built by dense_gemm_f32_gb300.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise LibraryMissing(
            f"{LIB_PATH} is missing: build it first with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    i, p = ctypes.c_int, ctypes.c_void_p
    gemm_args = [i, i, i, p, i, p, i, p, i, p]
    lib.gemm_f32_simt.argtypes = gemm_args
    lib.gemm_f32_simt.restype = i
    lib.gemm_f32_tc.argtypes = [i] + gemm_args
    lib.gemm_f32_tc.restype = i
    lib.gemm_bf16_tc.argtypes = gemm_args
    lib.gemm_bf16_tc.restype = i
    lib.dgemm_status_string.argtypes = [i]
    lib.dgemm_status_string.restype = ctypes.c_char_p
    lib.dgemm_last_cuda_error.argtypes = []
    lib.dgemm_last_cuda_error.restype = ctypes.c_char_p
    lib.dgemm_watchdog_status.argtypes = [p, ctypes.POINTER(ctypes.c_int)]
    lib.dgemm_watchdog_status.restype = i
    lib.dgemm_version.argtypes = []
    lib.dgemm_version.restype = i
    lib.dgemm_kernel_launches.argtypes = []
    lib.dgemm_kernel_launches.restype = ctypes.c_ulonglong
    lib.gemm_f32_tc_noalloc.argtypes = [i] + gemm_args
    lib.gemm_f32_tc_noalloc.restype = i
    lib.gemm_f16_tc.argtypes = gemm_args
    lib.gemm_f16_tc.restype = i
    lib.dgemm_gemm_ex.argtypes = [i, i, i] + gemm_args
    lib.dgemm_gemm_ex.restype = i
    lib.gemm_f8_tc.argtypes = [i] + gemm_args
    lib.gemm_f8_tc.restype = i
    m = [p, i]  # a matrix and its leading dimension
    lib.dgemm_layer_norm.argtypes = [i, i, i, ctypes.c_float, *m, p, p, *m, p, p, p]
    lib.dgemm_layer_norm_backward.argtypes = [i, i, i, *m, *m, p, p, p, *m, *m, p, p, p]
    lib.dgemm_linear.argtypes = [i] * 6 + [*m, *m, p, *m, *m, *m, p]
    lib.dgemm_linear_backward.argtypes = [i] * 6 + m * 7 + [p, p]
    lib.dgemm_gated_ffn.argtypes = [i] * 6 + m * 9 + [p]
    lib.dgemm_gated_ffn_backward.argtypes = [i] * 6 + m * 14 + [p]
    lib.dgemm_quantize_int8.argtypes = [i] * 4 + [*m, *m, p, p]
    lib.dgemm_linear_int8.argtypes = [i] * 5 + [*m, p, *m, p, p, *m, *m, p, p]
    lib.dgemm_gated_ffn_int8.argtypes = [i] * 5 + m + [*m, p] * 3 + [*m, *m, p, p]
    for name in ("layer_norm", "layer_norm_backward", "linear", "linear_backward", "gated_ffn",
                 "gated_ffn_backward", "quantize_int8", "linear_int8", "gated_ffn_int8",
                 "orthogonalize"):
        getattr(lib, "dgemm_" + name).restype = i
    f = ctypes.c_float
    lib.dgemm_orthogonalize.argtypes = [i, i, i, ctypes.POINTER(f), f, f, f, i, i, *m, *m, *m, p, p]
    lib.dgemm_linear_int8_workspace.argtypes = lib.dgemm_orthogonalize_workspace.argtypes = [i] * 2
    lib.dgemm_gated_ffn_int8_workspace.argtypes = [i] * 3
    for name in ("linear_int8", "gated_ffn_int8", "orthogonalize"):
        getattr(lib, f"dgemm_{name}_workspace").restype = ctypes.c_size_t
    _lib = lib
    return lib


def gemm_f32_simt(M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    return load().gemm_f32_simt(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_tc(mode, M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    return load().gemm_f32_tc(mode, M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_tc_noalloc(mode, M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    """gemm_f32_tc without allocating: re-pitch scratch is the library's fixed
    16 MiB device array (see include/dgemm.h)."""
    return load().gemm_f32_tc_noalloc(mode, M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_tc(M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    return load().gemm_bf16_tc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f16_tc(M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    return load().gemm_f16_tc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f8_tc(fmt, M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    return load().gemm_f8_tc(fmt, M, N, K, A, lda, B, ldb, C, ldc, stream)


def dgemm_gemm_ex(path, op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, stream=0):
    return load().dgemm_gemm_ex(path, op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, stream)


def dgemm_layer_norm(dtype, rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream=0):
    return load().dgemm_layer_norm(dtype, rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean,
                                   rstd, stream)


def dgemm_layer_norm_backward(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr,
                              dX, lddx, dweight, dbias, stream=0):
    return load().dgemm_layer_norm_backward(dtype, rows, cols, dY, lddy, X, ldx, weight, mean,
                                            rstd, dR, lddr, dX, lddx, dweight, dbias, stream)


def dgemm_linear(dtype, activation, op_w, M, N, K, X, ldx, W, ldw, bias, R, ldr, D, ldd, Z, ldz,
                 stream=0):
    return load().dgemm_linear(dtype, activation, op_w, M, N, K, X, ldx, W, ldw, bias, R, ldr, D,
                               ldd, Z, ldz, stream)


def dgemm_linear_backward(dtype, activation, op_w, M, N, K, dD, lddd, X, ldx, W, ldw, Z, ldz, dZ,
                          lddz, dX, lddx, dW, lddw, dbias, stream=0):
    return load().dgemm_linear_backward(dtype, activation, op_w, M, N, K, dD, lddd, X, ldx, W, ldw,
                                        Z, ldz, dZ, lddz, dX, lddx, dW, lddw, dbias, stream)


def dgemm_gated_ffn(dtype, activation, op_w, M, D, F, X, ldx, Wg, ldwg, Wu, ldwu, Wd, ldwd, R, ldr,
                    H, ldh, G, ldg, U, ldu, Y, ldy, stream=0):
    return load().dgemm_gated_ffn(dtype, activation, op_w, M, D, F, X, ldx, Wg, ldwg, Wu, ldwu, Wd,
                                  ldwd, R, ldr, H, ldh, G, ldg, U, ldu, Y, ldy, stream)


def dgemm_gated_ffn_backward(dtype, activation, op_w, M, D, F, dY, lddy, X, ldx, Wg, ldwg, Wu,
                             ldwu, Wd, ldwd, G, ldg, U, ldu, H, ldh, dG, lddg, dU, lddu, dX, lddx,
                             dWg, lddwg, dWu, lddwu, dWd, lddwd, stream=0):
    return load().dgemm_gated_ffn_backward(dtype, activation, op_w, M, D, F, dY, lddy, X, ldx, Wg,
                                           ldwg, Wu, ldwu, Wd, ldwd, G, ldg, U, ldu, H, ldh, dG,
                                           lddg, dU, lddu, dX, lddx, dWg, lddwg, dWu, lddwu, dWd,
                                           lddwd, stream)


def dgemm_quantize_int8(dtype, op, rows, cols, X, ldx, Q, ldq, scale, stream=0):
    return load().dgemm_quantize_int8(dtype, op, rows, cols, X, ldx, Q, ldq, scale, stream)


def dgemm_linear_int8_workspace(M, K):
    """Bytes of `work` for dgemm_linear_int8."""
    return load().dgemm_linear_int8_workspace(M, K)


def dgemm_linear_int8(dtype, activation, M, N, K, X, ldx, x_scale, W, ldw, w_scale, bias, R, ldr,
                      D, ldd, work, stream=0):
    return load().dgemm_linear_int8(dtype, activation, M, N, K, X, ldx, x_scale, W, ldw, w_scale,
                                    bias, R, ldr, D, ldd, work, stream)


def dgemm_gated_ffn_int8_workspace(M, D, F):
    """Bytes of `work` for dgemm_gated_ffn_int8."""
    return load().dgemm_gated_ffn_int8_workspace(M, D, F)


def dgemm_gated_ffn_int8(dtype, activation, M, D, F, X, ldx, Wg, ldwg, g_scale, Wu, ldwu, u_scale,
                         Wd, ldwd, d_scale, R, ldr, Y, ldy, work, stream=0):
    return load().dgemm_gated_ffn_int8(dtype, activation, M, D, F, X, ldx, Wg, ldwg, g_scale, Wu,
                                       ldwu, u_scale, Wd, ldwd, d_scale, R, ldr, Y, ldy, work,
                                       stream)


def dgemm_orthogonalize_workspace(rows, cols):
    """Bytes of `work` for dgemm_orthogonalize."""
    return load().dgemm_orthogonalize_workspace(rows, cols)


def dgemm_orthogonalize(x_dtype, dtype, steps, coefficients, eps, scale, residual_scale, rows, cols,
                        X, ldx, R, ldr, D, ldd, work, stream=0):
    """coefficients: a sequence of 3 * steps numbers, or None."""
    if coefficients is not None:
        if len(coefficients) < 3 * steps:
            raise ValueError(f"{3 * steps} coefficients are needed, got {len(coefficients)}")
        coefficients = (ctypes.c_float * len(coefficients))(*coefficients)
    return load().dgemm_orthogonalize(x_dtype, dtype, steps, coefficients, eps, scale,
                                      residual_scale, rows, cols, X, ldx, R, ldr, D, ldd, work,
                                      stream)


def dgemm_status_string(status):
    return load().dgemm_status_string(status).decode()


def dgemm_last_cuda_error():
    return load().dgemm_last_cuda_error().decode()


def dgemm_watchdog_status(stream=0):
    """(status, site code)."""
    where = ctypes.c_int(0)
    st = load().dgemm_watchdog_status(stream, ctypes.byref(where))
    return st, where.value


def dgemm_version():
    return load().dgemm_version()


def dgemm_kernel_launches():
    return load().dgemm_kernel_launches()
