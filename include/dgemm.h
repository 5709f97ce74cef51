/*
 * dgemm.h -- C ABI of the GB300 (sm_103a) dense GEMM library.
 *
 * Every gemm_* entry point and dgemm_gemm_ex computes the plain row-major
 * matrix product (the feed-forward operators around it are described where
 * they are declared)
 *
 *     C[i*ldc + j] = sum_{k=0}^{K-1} A[i*lda + k] * B[k*ldb + j],  0 <= i < M, 0 <= j < N
 *
 * as defined in "第八课：GPU 如何完成矩阵乘法" (Lesson 8: how a GPU does matrix
 * multiplication), section 一 (C = A x B with A in R^{M x K}, B in R^{K x N},
 * C_{i,j} = sum_k A_{i,k} B_{k,j}); the same formula opens "SGEMM 优化旅程",
 * Level 1, and section 4.1 of "4. 矩阵乘法（GEMM）优化".  The pages use the
 * compact row-major addressing A[row*K + k], B[k*N + col], C[row*N + col]
 * (Lesson 8 section 四, section 二十八); these entry points take BLAS-style
 * leading dimensions lda >= K, ldb >= N, ldc >= N, counted in elements.
 *
 * Semantics shared by all entry points
 *   - C is OVERWRITTEN inside its M x N region (no alpha/beta: the pages store
 *     the finished sum, C[row*N + col] = sum).  Elements of C outside that
 *     region (the ldc - N gap at the end of each row) are never written.
 *   - K == 0: the empty sum; the M x N region of C is set to zero.
 *   - M == 0 or N == 0: nothing to do; DGEMM_OK with no launch (the pointers
 *     are not looked at).
 *   - Sizes are int, as in the pages' kernel signatures; all offsets are
 *     computed in 64-bit.
 *
 * Pointers and ownership
 *   - A, B and C are DEVICE pointers (cudaMalloc'd or managed memory) on the
 *     current CUDA device, owned by the caller.  Host pointers are rejected
 *     with DGEMM_ERR_INVALID_POINTER before anything is launched.
 *   - Only natural element alignment is required (4 bytes for fp32, 2 for
 *     bf16).  Any pointer or leading dimension, aligned to 16 bytes or not, is
 *     accepted; the library chooses the load path itself.
 *   - C must not overlap the bytes A or B span: DGEMM_ERR_ALIAS.
 *
 * Execution
 *   - Asynchronous on `stream` (0 = the legacy default stream): the call
 *     validates, enqueues and returns.  Work on the same stream is ordered.
 *   - A launch failure, or a sticky error left by earlier work, is returned as
 *     DGEMM_ERR_CUDA; dgemm_last_cuda_error() gives the CUDA message.
 *   - Deterministic: the same inputs give bitwise identical C on every call
 *     (no floating-point atomics; K-split partial tiles are added in a fixed
 *     order).
 *   - Thread-safe and re-entrant; the only mutable library state is a
 *     per-thread error string and a per-device watchdog word (see
 *     dgemm_watchdog_status).
 *   - Some paths use temporary device memory (re-pitched operands, the FP32
 *     SIMT path's K-split partials, the lo parts of 3xTF32 operands, 8-bit
 *     transposes): stream-ordered allocations on `stream`, freed on `stream`
 *     at the end of the call, from a memory pool the library creates per
 *     device.  Back-to-back calls reuse the pool's memory; at the next
 *     stream, event or device synchronisation the pool returns what it holds
 *     beyond 32 MiB to the system, so no more than 32 MiB stays reserved
 *     between calls.  DGEMM_POOL_KEEP_BYTES (read once, when the pool is
 *     created) sets another bound, e.g. 0 to keep nothing.
 */
#ifndef DGEMM_H
#define DGEMM_H

#include <stddef.h>              /* size_t */
#include <cuda_runtime_api.h>   /* cudaStream_t */

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes.  Every entry point returns one; only DGEMM_OK means the work
 * was enqueued. */
typedef enum {
    DGEMM_OK = 0,
    DGEMM_ERR_INVALID_VALUE = 1,   /* negative or too large size, leading dimension too small, bad eps */
    DGEMM_ERR_NULL_POINTER = 2,    /* NULL A, B or C (or a matrix that is not optional) with work to do */
    DGEMM_ERR_ALIAS = 3,           /* an output overlaps another argument        */
    DGEMM_ERR_UNSUPPORTED = 4,     /* unknown mode, element type or activation   */
    DGEMM_ERR_CUDA = 5,            /* CUDA runtime/driver error (see below)      */
    DGEMM_ERR_ARCH = 6,            /* current device is not compute capability 10.3 */
    DGEMM_ERR_MISALIGNED = 7,      /* pointer not aligned to its element size    */
    DGEMM_ERR_INVALID_POINTER = 8, /* A, B or C is not device-accessible memory  */
    DGEMM_ERR_WATCHDOG = 9,        /* a kernel gave up a bounded wait (see dgemm_watchdog_status) */
    DGEMM_ERR_SCRATCH_LIMIT = 10   /* gemm_f32_tc_noalloc: operands need more than its fixed scratch */
} dgemm_status_t;

/* Operand operations of dgemm_gemm_ex: op(X) = X or its transpose. */
typedef enum {
    DGEMM_OP_N = 0,  /* as stored */
    DGEMM_OP_T = 1   /* transposed */
} dgemm_op_t;

/* Arithmetic paths of dgemm_gemm_ex (element type of A and B in brackets). */
typedef enum {
    DGEMM_PATH_SIMT = 0,    /* FP32 FFMA on the CUDA cores       [fp32] */
    DGEMM_PATH_TF32 = 1,    /* tcgen05, TF32 operands            [fp32] */
    DGEMM_PATH_3XTF32 = 2,  /* tcgen05, split-precision 3xTF32   [fp32] */
    DGEMM_PATH_BF16 = 3,    /* tcgen05, BF16 operands            [bf16] */
    DGEMM_PATH_FP16 = 4,    /* tcgen05, FP16 operands            [fp16] */
    DGEMM_PATH_F8_E4M3 = 5, /* tcgen05, FP8 E4M3 operands        [fp8]  */
    DGEMM_PATH_F8_E5M2 = 6  /* tcgen05, FP8 E5M2 operands        [fp8]  */
} dgemm_path_t;

/* 8-bit float formats of gemm_f8_tc. */
typedef enum {
    DGEMM_F8_E4M3 = 0,  /* 1 sign, 4 exponent (bias 7), 3 mantissa bits; no infinities, max 448 */
    DGEMM_F8_E5M2 = 1   /* 1 sign, 5 exponent (bias 15), 2 mantissa bits; IEEE-style, max 57344 */
} dgemm_f8_format_t;

/* Tensor-core precision modes of gemm_f32_tc. */
typedef enum {
    DGEMM_TC_TF32 = 0,   /* operands read at TF32 precision (10-bit mantissa), FP32 accumulate */
    DGEMM_TC_3XTF32 = 1  /* split precision: a = a_hi + a_lo, three TF32 products, FP32-grade result */
} dgemm_tc_mode_t;

/*
 * gemm_f32_simt -- FP32 inputs, FP32 fused multiply-add on the CUDA cores.
 *
 * The register-blocked, shared-memory tiled form of the product: "SGEMM 优化旅程"
 * Levels 2-5 (shared-memory tiles, padding against bank conflicts, double
 * buffering, 8x8 register blocking per thread of a 128x128x8 block tile) and
 * Lesson 8 sections 九-十九 (tile decomposition C_tile = sum_t A_tile,t B_tile,t,
 * register accumulation, multi-level tiling, boundary zero-fill and masked
 * stores of section 二十六).
 * A: M x K fp32, row-major, leading dimension lda >= max(1, K).
 * B: K x N fp32, row-major, leading dimension ldb >= max(1, N).
 * C: M x N fp32, row-major, leading dimension ldc >= max(1, N); overwritten.
 * Accuracy: |C - C_exact| <= 1e-5 * (|A| x |B|) elementwise; exact when every
 * product and partial sum is an integer below 2^24.
 */
int gemm_f32_simt(int M, int N, int K,
                  const float *A, int lda,
                  const float *B, int ldb,
                  float *C, int ldc,
                  cudaStream_t stream);

/*
 * gemm_f32_tc -- FP32 inputs on the 5th-generation tensor cores (tcgen05).
 *
 * The tensor-core form of the product: "SGEMM 优化旅程" Level 6 and Lesson 8
 * sections 二十一-二十三 (the tensor core computes a small D = A x B + C per
 * instruction, and must be fed tiles through shared memory).  Operands are
 * staged by TMA into swizzled shared memory, accumulated in tensor memory.
 * mode = DGEMM_TC_TF32:   each operand is read at TF32 precision; accuracy
 *                         |C - C_exact| <= 2e-3 * (|A| x |B|).
 * mode = DGEMM_TC_3XTF32: each operand is split a ~ hi + lo (hi = a with the
 *                         low 13 mantissa bits cleared, lo = a - hi rounded
 *                         to TF32) and C = A_hi B_hi + A_hi B_lo + A_lo B_hi;
 *                         accuracy <= 1e-5 * (|A| x |B|).  Infinities and
 *                         NaNs propagate as in IEEE arithmetic, except that
 *                         an infinite entry meeting a finite one whose lo is
 *                         exactly 0 adds inf * 0 = NaN to that entry of C.
 *                         Large problems (those the CTA-pair kernel takes)
 *                         first write lo(A) and lo(B) to scratch the size of
 *                         A and B, one extra kernel; if that scratch cannot
 *                         be allocated, the single-CTA kernel splits the
 *                         staged tiles in shared memory instead (same result,
 *                         slower).
 * Argument layout as gemm_f32_simt.  Unknown mode: DGEMM_ERR_UNSUPPORTED.
 */
int gemm_f32_tc(int mode, int M, int N, int K,
                const float *A, int lda,
                const float *B, int ldb,
                float *C, int ldc,
                cudaStream_t stream);

/*
 * gemm_bf16_tc -- BF16 inputs, FP32 accumulate, FP32 output, on tcgen05.
 *
 * Lesson 8 section 二十二 lists BF16 among the tensor-core input types; this is
 * the BF16-in / FP32-accumulate form of gemm_f32_tc.
 * A: M x K bfloat16 (raw 16-bit patterns), row-major, lda >= max(1, K).
 * B: K x N bfloat16, row-major, ldb >= max(1, N).
 * C: M x N fp32, row-major, ldc >= max(1, N); overwritten.
 * Accuracy: |C - C_exact| <= 8e-3 * (|A| x |B|), C_exact the exact product of
 * the bf16 values.
 */
int gemm_bf16_tc(int M, int N, int K,
                 const unsigned short *A, int lda,
                 const unsigned short *B, int ldb,
                 float *C, int ldc,
                 cudaStream_t stream);

/*
 * gemm_f32_tc_noalloc -- gemm_f32_tc for callers that cannot allocate.
 *
 * The pages have no counterpart of this entry point; it exists for callers
 * that must not allocate device memory during the call: code that runs with
 * every byte of device memory reserved up front (a serving process that has
 * partitioned HBM among its models, where a new allocation can fail), code
 * called from inside an allocator or memory-manager callback (which must not
 * re-enter the allocator), and latency-critical loops that must not risk an
 * allocation failing or growing a memory pool in the middle of a run.
 *
 * Same arguments, semantics, accuracy and status codes as gemm_f32_tc.  The
 * difference is where the re-pitch scratch lives: gemm_f32_tc takes it from
 * the library's stream-ordered memory pool when A or B rows do not start on
 * 16-byte boundaries; this
 * entry point uses instead a fixed 16 MiB array (DGEMM_NOALLOC_SCRATCH_BYTES)
 * that the library holds in device memory on every GPU that loads it, until
 * the process exits.  It calls no cudaMalloc, cudaFree or other allocating
 * routine.
 *   - Limit: the re-pitched copies of A and/or B (rows rounded up to 16 bytes,
 *     each copy rounded up to 256 bytes) must fit in 16 MiB; otherwise the
 *     call returns DGEMM_ERR_SCRATCH_LIMIT and launches nothing.  Operands
 *     that need no re-pitch use no scratch, at any size.
 *   - 3xTF32 writes the lo parts of A and B into the rest of the array when
 *     they fit there; larger problems run on the single-CTA kernel, which
 *     needs no scratch for the split.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current.  Under CUDA's lazy
 *     module loading (the default) that lookup is also what loads the array
 *     into device memory, so the first call on each device must come before
 *     the caller reserves all device memory, and before any stream capture
 *     begins on the device.  The address is kept for the life of the process:
 *     do not use the library across cudaDeviceReset.
 *   - Results are bitwise those of gemm_f32_tc in TF32 mode, and in 3xTF32
 *     mode whenever the lo parts fit in the array (or the problem is small
 *     enough for the single-CTA kernel anyway); larger 3xTF32 problems run
 *     on a different kernel and agree with gemm_f32_tc only within the
 *     3xTF32 tolerance.
 *   - Every call on a device shares the one array, and it keeps the last
 *     call's contents.  Each call overwrites all the scratch it reads before
 *     reading it, so nothing needs clearing; but two calls whose work
 *     overlaps on the GPU (different streams, no ordering between them) race
 *     on the array and may corrupt each other's results.  Order such calls
 *     on one stream or with events.
 */
int gemm_f32_tc_noalloc(int mode, int M, int N, int K,
                        const float *A, int lda,
                        const float *B, int ldb,
                        float *C, int ldc,
                        cudaStream_t stream);

/* Size in bytes of the fixed scratch array gemm_f32_tc_noalloc uses. */
#define DGEMM_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * gemm_f16_tc -- FP16 inputs, FP32 accumulate, FP32 output, on tcgen05.
 *
 * The tensor-core input type of "SGEMM 优化旅程" Level 6 (half operands with
 * a float accumulator, there through WMMA fragments) and the first entry of
 * Lesson 8 section 二十二's list of tensor-core formats; the same kernels as
 * gemm_bf16_tc with IEEE binary16 operands.
 * A: M x K float16 (raw 16-bit patterns), row-major, lda >= max(1, K).
 * B: K x N float16, row-major, ldb >= max(1, N).
 * C: M x N fp32, row-major, ldc >= max(1, N); overwritten.
 * The fp16 inputs are exact, so only the FP32 accumulation rounds: at most
 * K/16 rounded additions of the accumulator, |C - C_exact| <= 2e-4 *
 * (|A| x |B|) for K <= 16384.
 */
int gemm_f16_tc(int M, int N, int K,
                const unsigned short *A, int lda,
                const unsigned short *B, int ldb,
                float *C, int ldc,
                cudaStream_t stream);

/*
 * gemm_f8_tc -- FP8 inputs (E4M3 or E5M2), FP32 accumulate, FP32 output, on
 * tcgen05 (kind::f8f6f4).
 *
 * Lesson 8 section 二十二 lists FP8 among the tensor cores' input formats;
 * the pages give it no scaling convention, so the 8-bit values are the
 * operands as given (scale 1; a caller with scaled data multiplies C by the
 * product of its scales).  `format` (dgemm_f8_format_t) applies to A and B.
 * A: M x K bytes, row-major, lda >= max(1, K).
 * B: K x N bytes, row-major, ldb >= max(1, N).
 * C: M x N fp32, row-major, ldc >= max(1, N); overwritten.
 * The tensor cores read 8-bit operands K-major only, so B (K x N, N
 * contiguous) is transposed into stream-ordered scratch (N x K) before the
 * GEMM: one extra kernel moving 2 x |B| bytes.  With B already stored N x K
 * (dgemm_gemm_ex, op_b = DGEMM_OP_T) nothing is moved.
 * The 8-bit inputs are exact and so are their products in fp32, so only the
 * FP32 accumulation rounds (once per MMA instruction, K/32 times):
 * |C - C_exact| <= 2e-4 * (|A| x |B|) for K <= 16384 (measured: 1e-7).
 * Unknown format: DGEMM_ERR_UNSUPPORTED.
 */
int gemm_f8_tc(int format, int M, int N, int K,
               const unsigned char *A, int lda,
               const unsigned char *B, int ldb,
               float *C, int ldc,
               cudaStream_t stream);

/*
 * dgemm_gemm_ex -- C = op(A) x op(B) on any path, with transposed operands.
 *
 * Lesson 8 section 二十八 ("矩阵布局为什么重要") describes row- and column-major
 * storage and the transpose flags that GEMM interfaces carry for them.  Here
 * every matrix is stored row-major; a transposed operand is simply stored
 * with its other dimension contiguous (a column-major op(X) is a row-major
 * X^T):
 *   op_a = DGEMM_OP_N: A is M x K, lda >= max(1, K);  op(A) = A
 *   op_a = DGEMM_OP_T: A is K x M, lda >= max(1, M);  op(A) = A^T
 *   op_b = DGEMM_OP_N: B is K x N, ldb >= max(1, N);  op(B) = B
 *   op_b = DGEMM_OP_T: B is N x K, ldb >= max(1, K);  op(B) = B^T
 * C is M x N fp32, row-major, ldc >= max(1, N); C[i][j] = sum_k op(A)[i][k]
 * op(B)[k][j].  `path` (dgemm_path_t) selects the arithmetic and the element
 * type of A and B; accuracy, semantics and status codes are those of the
 * corresponding entry point above (gemm_f32_simt, gemm_f32_tc, gemm_bf16_tc,
 * gemm_f16_tc, gemm_f8_tc), which equal dgemm_gemm_ex with op_a = op_b =
 * DGEMM_OP_N.  The FP8 paths read op(A) as M x K and op(B) as N x K natively
 * (op_a = N, op_b = T); other layouts are transposed into scratch first.
 * Unknown path or op: DGEMM_ERR_UNSUPPORTED.
 */
int dgemm_gemm_ex(int path, int op_a, int op_b, int M, int N, int K,
                  const void *A, int lda,
                  const void *B, int ldb,
                  float *C, int ldc,
                  cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Feed-forward operators: what a transformer layer runs around the product.
 *
 * Matrices are row-major with leading dimensions in elements, vectors are
 * contiguous; pointers, ownership, asynchrony, determinism and status codes
 * are those of the GEMM entry points.  Every element type below is `dtype`
 * (dgemm_dtype_t) unless a pointer says float.  Sums, statistics and
 * activations are computed in fp32; an output element is rounded once, to
 * nearest even.  Outputs must not overlap any other argument
 * (DGEMM_ERR_ALIAS) except where an entry point says so.  Matrices marked
 * "workspace" are outputs whose contents are unspecified afterwards beyond
 * what is stated.  A sum over nothing (K == 0, no rows) is zero.
 *
 * The sizes of a product and the columns of a layer norm are at most
 * DGEMM_OPS_MAX_SIZE (beyond it DGEMM_ERR_INVALID_VALUE): the kernels count
 * columns and tiles in 32 bits, and this leaves room for the last tile.
 */
#define DGEMM_OPS_MAX_SIZE 2147482624 /* 2^31 - 1024 */

/* Element types of the feed-forward operators. */
typedef enum {
    DGEMM_DTYPE_F32 = 0,  /* layer norm, dgemm_quantize_int8, dgemm_orthogonalize */
    DGEMM_DTYPE_BF16 = 1,
    DGEMM_DTYPE_F16 = 2
} dgemm_dtype_t;

/* Activations act(z). */
typedef enum {
    DGEMM_ACT_NONE = 0,       /* z */
    DGEMM_ACT_RELU = 1,       /* max(z, 0); derivative 0 at 0 */
    DGEMM_ACT_GELU = 2,       /* z Phi(z), Phi the normal distribution function */
    DGEMM_ACT_GELU_TANH = 3,  /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    DGEMM_ACT_SILU = 4        /* z / (1 + exp(-z)) */
} dgemm_activation_t;

/*
 * dgemm_layer_norm -- y = (x - mu) rstd weight + bias for every row x of X.
 *
 * mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), in two passes over
 * the row held on the SM (the variance is of the centred values).
 * X, Y: rows x cols.  weight, bias: cols elements, or NULL (1 and 0).
 * mean, rstd: rows floats, or NULL when the backward pass is not wanted; with
 * cols == 0 nothing is written, the statistics of no values included.
 * eps >= 0 and finite, else DGEMM_ERR_INVALID_VALUE.
 */
int dgemm_layer_norm(int dtype, int rows, int cols, float eps,
                     const void *X, int ldx,
                     const void *weight, const void *bias,
                     void *Y, int ldy, float *mean, float *rstd,
                     cudaStream_t stream);

/*
 * dgemm_layer_norm_backward -- with xh = (x - mean) rstd and p = dy weight:
 * dX = rstd (p - mean(p) - xh mean(p xh)) + dR, dweight = sum over rows of
 * dy xh, dbias = sum over rows of dy.
 *
 * dY, X, dX: rows x cols.  mean, rstd: as the forward pass wrote them.
 * weight: or NULL (1).  dR: rows x cols, a gradient that joins dX (a skip
 * connection's), or NULL.  dweight, dbias: cols elements, or NULL.
 */
int dgemm_layer_norm_backward(int dtype, int rows, int cols,
                              const void *dY, int lddy, const void *X, int ldx,
                              const void *weight, const float *mean, const float *rstd,
                              const void *dR, int lddr,
                              void *dX, int lddx, void *dweight, void *dbias,
                              cudaStream_t stream);

/*
 * dgemm_linear -- Z = X op(W) + bias, D = act(Z) + R, in one kernel.
 *
 * dtype BF16 or F16.  X: M x K.  op_w = DGEMM_OP_N: W is K x N; DGEMM_OP_T: W
 * is N x K and op(W) = W^T.  bias: N elements, or NULL.  R (residual): M x N,
 * or NULL; D may be R itself (same address and leading dimension).  D: M x N.
 * Z: M x N, or NULL when the backward pass does not need it.
 */
int dgemm_linear(int dtype, int activation, int op_w, int M, int N, int K,
                 const void *X, int ldx, const void *W, int ldw,
                 const void *bias, const void *R, int ldr,
                 void *D, int ldd, void *Z, int ldz,
                 cudaStream_t stream);

/*
 * dgemm_linear_backward -- dZ = dD act'(Z), dX = dZ op(W)^T, dW = X^T dZ
 * (stored as W is), dbias = sum over rows of dZ.
 *
 * Z: as dgemm_linear wrote it; dZ: M x N workspace, holding dZ afterwards;
 * both are ignored when activation is DGEMM_ACT_NONE (dZ is dD then).  dX, dW,
 * dbias: NULL for a gradient that is not wanted (X or W may then be NULL).
 * dZ is rounded to dtype before the two products; dbias sums unrounded values.
 */
int dgemm_linear_backward(int dtype, int activation, int op_w, int M, int N, int K,
                          const void *dD, int lddd, const void *X, int ldx,
                          const void *W, int ldw, const void *Z, int ldz,
                          void *dZ, int lddz,
                          void *dX, int lddx, void *dW, int lddw, void *dbias,
                          cudaStream_t stream);

/*
 * dgemm_gated_ffn -- G = X op(Wg), U = X op(Wu), H = act(G) U (one kernel),
 * Y = H op(Wd) + R (another).
 *
 * X, Y: M x D.  op_w = DGEMM_OP_N: Wg, Wu are D x F and Wd is F x D;
 * DGEMM_OP_T: F x D and D x F.  R: M x D, or NULL; Y may be R itself.  H: M x F
 * workspace, holding H rounded to dtype afterwards.  G, U: M x F, both or
 * neither NULL: kept for the backward pass.
 */
int dgemm_gated_ffn(int dtype, int activation, int op_w, int M, int D, int F,
                    const void *X, int ldx, const void *Wg, int ldwg,
                    const void *Wu, int ldwu, const void *Wd, int ldwd,
                    const void *R, int ldr, void *H, int ldh,
                    void *G, int ldg, void *U, int ldu, void *Y, int ldy,
                    cudaStream_t stream);

/*
 * dgemm_gated_ffn_backward -- the gradients of dgemm_gated_ffn from G and U.
 *
 * dH = dY op(Wd)^T stays in the accumulator of one kernel, which writes
 * dG = dH U act'(G), dU = dH act(G) and H = act(G) U (M x F workspaces);
 * dX = dG op(Wg)^T + dU op(Wu)^T, dWg = X^T dG, dWu = X^T dU, dWd = H^T dY
 * (stored as the weights are).  dX, dWd: or NULL; dWg, dWu: both or neither.
 */
int dgemm_gated_ffn_backward(int dtype, int activation, int op_w, int M, int D, int F,
                             const void *dY, int lddy, const void *X, int ldx,
                             const void *Wg, int ldwg, const void *Wu, int ldwu,
                             const void *Wd, int ldwd,
                             const void *G, int ldg, const void *U, int ldu,
                             void *H, int ldh, void *dG, int lddg, void *dU, int lddu,
                             void *dX, int lddx, void *dWg, int lddwg,
                             void *dWu, int lddwu, void *dWd, int lddwd,
                             cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Products with weights in 8-bit integers, and the rows in 8-bit integers
 * that they multiply.
 *
 * A row x is held as integers q of at most 127 in size and one float, its
 * scale: x_j is about q_j scale.  Weights are stored out x in (N x K), a row and
 * a scale for each output feature; tokens get theirs in the call.  Integers
 * are multiplied and summed in fp32, exactly while the partial sums stay
 * within 2^24 (any 1024 products of signed bytes do, 1040 where none is -128) and with fp32's
 * rounding beyond; for one to four tokens in 32-bit integers where that is quicker, always exactly.
 * A row with NaN or an infinity gets that as its scale and zeros as integers;
 * results computed from it are NaN.
 */

/*
 * dgemm_quantize_int8 -- q_j = round(127 x_j / top) to the nearest integer,
 * ties to even, and scale = top / 127, top = max |x_j| over a row (0, and scale
 * 0, where there is nothing but zeros).  The rounding is that of the exact
 * quotient for bf16 and fp16, of an fp32 one for fp32.
 *
 * X: rows x cols, of `dtype`.  op = DGEMM_OP_N: Q is rows x cols, scale rows floats.
 * op = DGEMM_OP_T: the rows are X's columns, Q is cols x rows and scale cols
 * floats (weights stored in x out, once, for the products below).
 */
int dgemm_quantize_int8(int dtype, int op, int rows, int cols,
                        const void *X, int ldx,
                        signed char *Q, int ldq, float *scale,
                        cudaStream_t stream);

/*
 * dgemm_linear_int8 -- D = act(Z + bias) + R with Z_ij = s_i w_scale_j
 * sum_k q_ik W_jk, q and s the rows of X in 8 bits.
 *
 * X: M x K of `dtype` (BF16 or F16), put into 8 bits here as dgemm_quantize_int8
 * does; or, with x_scale (M floats) not NULL, M x K signed bytes.  W: N x K
 * signed bytes, w_scale: N floats.  bias: N elements of dtype, or NULL.  R: M x
 * N, or NULL; D: M x N, may be R itself.  work: dgemm_linear_int8_workspace(M,
 * K) bytes on a 16-byte boundary.
 */
size_t dgemm_linear_int8_workspace(int M, int K);
int dgemm_linear_int8(int dtype, int activation, int M, int N, int K,
                      const void *X, int ldx, const float *x_scale,
                      const signed char *W, int ldw, const float *w_scale,
                      const void *bias, const void *R, int ldr,
                      void *D, int ldd, void *work,
                      cudaStream_t stream);

/*
 * dgemm_gated_ffn_int8 -- H = act(G) U with G and U the products above of X and
 * Wg, Wu (one kernel), Y = the product of H and Wd, plus R.
 *
 * X, Y, R: M x D of `dtype`; R or NULL, Y may be R itself.  Wg, Wu: F x D, Wd: D x
 * F signed bytes, their scales F, F and D floats.  H is kept in fp32 and put into
 * 8 bits row by row like X.  work: dgemm_gated_ffn_int8_workspace(M, D, F)
 * bytes on a 16-byte boundary.
 */
size_t dgemm_gated_ffn_int8_workspace(int M, int D, int F);
int dgemm_gated_ffn_int8(int dtype, int activation, int M, int D, int F,
                         const void *X, int ldx,
                         const signed char *Wg, int ldwg, const float *g_scale,
                         const signed char *Wu, int ldwu, const float *u_scale,
                         const signed char *Wd, int ldwd, const float *d_scale,
                         const void *R, int ldr, void *Y, int ldy, void *work,
                         cudaStream_t stream);

/* ------------------------------------------------------------------------
 * dgemm_orthogonalize -- a matrix with its singular values brought towards 1
 * (what the Muon optimiser makes of a weight's momentum), and the update of a
 * weight by it, by a Newton-Schulz iteration:
 *
 *   X_0 = X / (|X| + eps), |X| the root of the sum of squares,
 *   X_k+1 = a_k X_k + (b_k A + c_k A A) X_k, A = X_k X_k^T (X_k^T X_k on the right
 *           where X has more rows than columns: the same result),
 *   D = scale X_steps + residual_scale R.
 *
 * X: rows x cols of x_dtype; R (or NULL) and D: rows x cols of dtype; both any of
 * the three types; D may be R itself (w <- (1 - lr decay) w - lr update in place).
 * coefficients: 3 * steps finite floats in HOST memory, a_k, b_k, c_k in turn,
 * read during the call; at most 64 in size.  steps: 1 to DGEMM_NEWTON_MAX_STEPS.  eps >=
 * 0 and finite.  Anything else: DGEMM_ERR_INVALID_VALUE.
 * The iteration runs in fp16 with fp32 sums, whatever the types; an X in fp32 begins it as two
 * fp16 terms.  Five steps of a = 3.4445,
 * -4.7750, 2.0315 are off by some 0.0015 of the update's norm for gradients with a few strong
 * directions over noise, 0.004 to 0.008 where the singular values fall as i^-2 to i^-4, and at
 * most 0.02, which a matrix of rank one comes near to (all products in bf16: 0.005 to 0.26); 0.07 where
 * the smaller side is 2 to 7, too few for roundings to cancel.
 * A rounding of 2^-12 in directions that X does not have is enlarged by the a of every
 * step after the first two, so more steps, or steeper ones, are off by more.  So is an X whose norm
 * is far below eps (2^-10 of it): its elements leave fp16's range.  And so is an X with a side of millions:
 * the tensor cores cut their fp32 sums over it off, which is 0.007 at 4 x 4 million, 0.05 at 1 x 50
 * million, nothing to be seen at 512 x 131072.  With eps = 0 a
 * matrix of zeros, and always one with NaN or an infinity, gives NaN.  Coefficients
 * under which the iteration diverges give infinities and NaN past 2^7 or so.
 * work: dgemm_orthogonalize_workspace(rows, cols) bytes on a 16-byte boundary.
 */
#define DGEMM_NEWTON_MAX_STEPS 64
size_t dgemm_orthogonalize_workspace(int rows, int cols);
int dgemm_orthogonalize(int x_dtype, int dtype, int steps, const float *coefficients, float eps,
                        float scale, float residual_scale, int rows, int cols,
                        const void *X, int ldx, const void *R, int ldr,
                        void *D, int ldd, void *work,
                        cudaStream_t stream);

/* Static English text for a status code (never NULL). */
const char *dgemm_status_string(int status);

/* The CUDA error text behind the calling thread's last DGEMM_ERR_CUDA
 * ("" if none).  The pointer stays valid until the thread's next call. */
const char *dgemm_last_cuda_error(void);

/*
 * dgemm_watchdog_status -- synchronise `stream`, then read and clear the
 * current device's watchdog word.  The tensor-core kernels bound every wait
 * on a shared-memory barrier; a wait that runs out (a hardware or library
 * fault, never expected in normal use) makes the kernel record where it gave
 * up, drain its copies, free its tensor memory and return, leaving C
 * incomplete.  Returns DGEMM_OK when no kernel gave up since the last read,
 * DGEMM_ERR_WATCHDOG when one did (*where, if not NULL, gets the recorded
 * site code), DGEMM_ERR_CUDA on a CUDA error.  With the environment variable
 * DGEMM_TC_TEST_STALL=1 the first CTA of each tensor-core launch waits on a
 * barrier that nothing arrives at, so that this path can be tested: the call
 * returns after a few seconds with C incomplete and the status set.
 */
int dgemm_watchdog_status(cudaStream_t stream, int *where);

/* Library version as an integer, major*10000 + minor*100 + patch. */
int dgemm_version(void);

/* Number of kernels this library has launched in this process, on any
 * device or stream (a diagnostic for counting launches around a region). */
unsigned long long dgemm_kernel_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_H */
