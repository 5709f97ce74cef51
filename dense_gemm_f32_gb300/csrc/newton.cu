// newton.cu -- orthogonalising a matrix by a Newton-Schulz iteration:
//
//   X_0 = X / (|X| + eps),  |X| the root of the sum of squares,
//   X_k+1 = a X_k + (b A + c A^2) X_k,  A = X_k X_k^T   (X_k^T X_k on the right
//                                                        when X is taller than wide)
//
// which brings every singular value s to p(p(...p(s))), p(s) = a s + b s^3 + c s^5.
//
// Everything between X and the result is fp16 with fp32 accumulators: 11 bits, where
// bf16 has 8, at the same rate, and with the scales below nothing that matters
// leaves fp16's range.  Against 64 bits the result is off by 0.001 to 0.015 of its
// norm where one in bf16 is off by 0.006 to 0.26 (the small singular values, which
// the iteration enlarges, sit in the rounding of the large ones; by matrix in
// tests/newton_spectra.py), and storing the result in bf16 by 0.0017.
//  * X_0 is kept as X 2^(8 - e), 2^e the power of two next above |X| + eps: exact for
//    16-bit X but for elements of 2^-22 (fp16) or 2^-25 (bf16) of the norm and less.  The factor
//    2^e / (|X| + eps) that is missing goes into the first Gram matrix and the first product with X, in
//    fp32.  An fp32 X is kept in two fp16 terms until the first group ends, 22 bits of it: its Gram
//    matrix is then H H^T + H L^T + L H^T and the product Q H + Q L, the terms blocks of K of one
//    product.  (Rounded to 11 bits an fp32 matrix of rank one was off by 0.15 of the result's norm,
//    eight directions over a floor of 10^-3 by 0.03: the five steps enlarge what is rounded
//    where X has no direction by a^5 = 485.  The second terms cost 4096 x 4096 171 us of 1082,
//    14336 x 4096 738 of 2643.)  Later X_k are kept times 2^8, the m x m matrices times 2^6.
//  * Steps in groups.  All m x m matrices here are polynomials in A, so they are
//    symmetric and commute.  Within a group X stays where it is: with P = a I + b
//    A + c A^2, the next step's Gram matrix is P A P, the product of the P so far is Q, and
//    only the group's end forms Q X.  A step costs 4 products of m^3 / 2
//    multiplications then, instead of one such, a Gram matrix (m^2 n / 2) and a
//    product with X (m^2 n).  Two roundings work against each other.  One of A off
//    the true Gram matrix is not noticed before the group ends, and grows by a^2 in every step
//    where the singular values are small; how much of it is there depends on X, whose elements may
//    all round alike (a few distinct values, low rank), not on its size.  And X is rounded
//    when a group ends, which the steps after it enlarge by their a where X has no direction of its
//    own.  So the first group takes steps while that growth is at most 2^4 (two with the usual a =
//    3.4445; three, a growth of 2^7, put matrices of rank 1 and 2 off by 0.03 to 0.09), the second
//    is one step (as two it put gradients off by 0.005 for 0.0014: it is there that most of the
//    singular values come up to 1), and later ones take steps up to 2^4 again where that
//    saves work, in wide matrices: at n = 1.25 m five steps as 2 + 1 + 2 cost 2% less than as 2 + 1 + 1 +
//    1, at 3.5 m 15%.  In a small matrix, whose time is its launches, single steps are nearer.
//    In 64-bit simulations of these roundings five steps are off by 0.0003 to 0.004 of the norm
//    over spectra from flat to i^-1.5, 0.008 at i^-4, and at most 0.016, a matrix of rank one
//    (the limit that include/dgemm.h states, 0.02, is what the roundings can add up to).
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <type_traits>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace dg {
namespace {

constexpr int kThreads = 512;
constexpr int kAhead = 4;  // vectors of a thread in flight

// Sums of squares in three scales, one of which neither overflows nor loses a
// share that matters, whatever the elements' size: the plain one from 2^-80 to 2^100 (2^38
// elements of one size have squares of 2^-118 there, a normal number); below it (x 2^100)^2, which
// are 2^-98 for the smallest subnormal and 2^120 in sum at most; above it (x 2^-90)^2, 2^76 for the
// largest number and 2^-118 for 2^38 elements that reach 2^100 together.
constexpr float kUp = 0x1p100f, kDown = 0x1p-90f;
struct Squares {
  float mid = 0.f, big = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float u = x * kUp, d = x * kDown;
    mid = fmaf(x, x, mid);
    big = fmaf(d, d, big);
    small = fmaf(u, u, small);
  }
};

template <class T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
    squares_kernel(int rows, int cols, const T *X, int64_t ldx, float *partial) {
  constexpr int V = kVec<T>;
  __shared__ float fold[3][kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int vecs = (cols + V - 1) / V;
  const int64_t all = (int64_t)rows * vecs, step = (int64_t)gridDim.x * kThreads;
  Squares s;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < all; i0 += kAhead * step) {
    RowBlocks b[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = i0 + k * step, row = i / vecs;
      b[k] = fetch_row16<T, ALIGNED>(X + row * ldx, (int)(i - row * vecs) * V, i < all ? cols : 0);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = i0 + k * step, row = i / vecs;
      if (i >= all) break;
      float f[V];
      widen16<T>(take_row16<T, ALIGNED>(b[k], X + row * ldx, (int)(i - row * vecs) * V, cols), f);
#pragma unroll
      for (int j = 0; j < V; ++j) s.add(f[j]);
    }
  }
  float v[3] = {s.mid, s.big, s.small};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    for (int m = 16; m; m >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    if ((threadIdx.x & 31) == 0) fold[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) t += fold[threadIdx.x][w];
    partial[blockIdx.x * 3 + threadIdx.x] = t;
  }
}

// Every block adds the partial sums in the same order, then scales its share.
template <class T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(int rows, int cols, const T *X, int64_t ldx, float eps, const float *partial, int parts,
                 __half *out, __half *out_lo, int64_t ldo, float *factor) {
  constexpr int V = kVec<T>;
  __shared__ float fold[3][kThreads / 32];
  __shared__ float up[2];
  pdl_launch_dependents();
  pdl_wait();
  float v[3] = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x; i < parts; i += kThreads)
    for (int k = 0; k < 3; ++k) v[k] += partial[i * 3 + k];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    for (int m = 16; m; m >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    if ((threadIdx.x & 31) == 0) fold[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    float t[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      t[k] = fold[k][threadIdx.x % (kThreads / 32)];
      for (int m = kThreads / 64; m; m >>= 1) t[k] += __shfl_xor_sync(0xffffffffu, t[k], m);
    }
    // The plain sum where it is away from both ends of fp32's range.  64 bits from here, for
    // their range alone: sums in them took 3 us more.
    double norm;
    if (!(t[0] < 0x1p100f))
      norm = sqrtf(t[1]) * 0x1p90;
    else if (t[0] < 0x1p-80f)
      norm = sqrtf(t[2]) * 0x1p-100;
    else
      norm = sqrtf(t[0]);
    norm += (double)eps;
    int e = 0;
    const double f = frexp(norm, &e);  // norm = f 2^e, 1/2 <= f < 1
    const bool none = !(norm > 0.) || isinf(norm);  // nothing to divide by, an infinity or NaN
    if (blockIdx.x == 0 && threadIdx.x == 0) *factor = none ? __uint_as_float(0x7fc00000u) : 1.f / (float)f;
    // 2^(8 - e) in two factors that are fp32 numbers
    const int k = none ? 0 : 8 - e, k1 = k / 2;
    if (threadIdx.x == 0) up[0] = ldexpf(1.f, k1), up[1] = ldexpf(1.f, k - k1);
  }
  __syncthreads();
  const float u0 = up[0], u1 = up[1];
  const int vecs = (cols + V - 1) / V;
  const int64_t all = (int64_t)rows * vecs, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < all; i0 += kAhead * step) {
    RowBlocks b[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = i0 + k * step, row = i / vecs;
      b[k] = fetch_row16<T, ALIGNED>(X + row * ldx, (int)(i - row * vecs) * V, i < all ? cols : 0);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t i = i0 + k * step, row = i / vecs;
      const int col = (int)(i - row * vecs) * V;
      if (i >= all) break;
      float f[V];
      widen16<T>(take_row16<T, ALIGNED>(b[k], X + row * ldx, col, cols), f);
      uint32_t w[V / 2];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = f[j] * u0 * u1;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) w[j] = pack2<__half>(f[2 * j], f[2 * j + 1]);
      if constexpr (V == 8)  // rows of whole vectors, padded
        *reinterpret_cast<uint4 *>(out + row * ldo + col) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        *reinterpret_cast<uint2 *>(out + row * ldo + col) = make_uint2(w[0], w[1]);
      if constexpr (std::is_same<T, float>::value) {  // what fp16 leaves of an element
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 hi = unpack2<__half>(w[j]);
          w[j] = pack2<__half>(f[2 * j] - hi.x, f[2 * j + 1] - hi.y);
        }
        *reinterpret_cast<uint2 *>(out_lo + row * ldo + col) = make_uint2(w[0], w[1]);
      }
    }
  }
}

int scale_blocks(int num_sms) { return 2 * num_sms; }

template <class T>
cudaError_t launch_scale(int rows, int cols, const void *X, int64_t ldx, float eps, __half *out, __half *out_lo,
                         int64_t ldo, float *factor, float *partial, int num_sms, cudaStream_t stream) {
  const T *x = static_cast<const T *>(X);
  const bool al = rows_aligned(X, ldx, sizeof(T)) && cols % kVec<T> == 0;
  const int64_t vecs = (int64_t)rows * ((cols + kVec<T> - 1) / kVec<T>);
  const int64_t want = (vecs + kThreads * kAhead - 1) / (kThreads * kAhead);
  const int blocks = (int)(want < scale_blocks(num_sms) ? want : scale_blocks(num_sms));
  cudaError_t e = launch_kernel(al ? squares_kernel<T, true> : squares_kernel<T, false>, dim3(blocks),
                                dim3(kThreads), 0, stream, 1u, rows, cols, x, ldx, partial);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_kernel(al ? scale_kernel<T, true> : scale_kernel<T, false>, dim3(blocks), dim3(kThreads), 0,
                    stream, 1u, rows, cols, x, ldx, eps, static_cast<const float *>(partial), blocks,
                    out, out_lo, ldo, factor);
  if (e == cudaSuccess) count_launch();
  return e;
}

// -------------------------------------------------------------- the iteration
int64_t round256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// X, the next X, what fp16 leaves of an fp32 X, five m x m matrices, the factor and the partial
// sums (up to 512 SMs' worth).
struct Work {
  __half *x[3], *square[5];
  float *factor, *partial;
  size_t bytes;
  Work(void *base, int rows, int cols) {
    const int64_t m = rows < cols ? rows : cols;
    const int64_t x_bytes = round256((int64_t)rows * line_pitch(cols, 2) * 2), s_bytes = round256(m * line_pitch(m, 2) * 2);
    const uintptr_t begin = reinterpret_cast<uintptr_t>(base);
    uintptr_t p = begin;
    auto take = [&](int64_t n) {
      const uintptr_t at = p;
      p += (uintptr_t)n;
      return at;
    };
    for (auto &q : x) q = reinterpret_cast<__half *>(take(x_bytes));
    for (auto &q : square) q = reinterpret_cast<__half *>(take(s_bytes));
    factor = reinterpret_cast<float *>(take(256));
    partial = reinterpret_cast<float *>(take(round256(scale_blocks(512) * 3 * 4)));
    bytes = (size_t)(p - begin);
  }
};

// DGEMM_NEWTON_*: an environment variable's value in lo .. hi, or -1 (read at
// every launch, for tests and tuning).
int knob(const char *name, int lo, int hi) {
  const char *e = getenv(name);
  if (e == nullptr || e[0] < '0' || e[0] > '9') return -1;
  const int v = atoi(e);
  return v >= lo && v <= hi ? v : -1;
}

// The quicker kernel, tile and K split by time models (microseconds; graph replays on
// GB300).  Small kernel: on 128 x 128 tiles 3.4 us of launch, first load and epilogue, and
// 0.27 us for a CTA's stage of 64 k or its share where two run on an SM, 5 to 6.5 us for
// joining the parts of a K split; on 128 x 64 tiles, half an epilogue on twice as many SMs,
// 2.7 us and 0.255 for a stage, 0.165 its share.  (Five steps of 512 x 1408: 94 us on the
// narrow tiles, 110 on the square ones; 997 x 1013: 111, 126; of 2048 x 2048, where the narrow
// ones are two to an SM: 242, 213.)  Pair kernel: 8 us, and 0.28 us per 64 k of a wave of
// 256 x 256 tiles.
cudaError_t run(const NewtonGemm &p, int num_sms, int *wd, cudaStream_t stream) {
  const int f_pair = knob("DGEMM_NEWTON_PAIR", 0, 1), f_splits = knob("DGEMM_NEWTON_SPLITS", 1, 8);
  const int f_tn = knob("DGEMM_NEWTON_TN", 64, 128);
  auto tiles_of = [&](int t, int w) {  // t x w
    const int64_t tm = (p.M + t - 1) / t, tn = (p.N + w - 1) / w;
    return p.symmetric ? (tm * tn - t / w * (tm * (tm - 1) / 2)) * (p.A2 != nullptr ? 2 : 1) : tm * tn;
  };
  const int64_t small = tiles_of(128, 128), narrow = tiles_of(128, 64), large = tiles_of(256, 256);
  const int64_t kblocks = (p.K + 63) / 64 * (1 + (p.A_lo != nullptr) + (p.B_lo != nullptr));
  const int64_t waves = (large + num_sms / 2 - 1) / (num_sms / 2);
  const double pair_time = 8.0 + 0.28 * (double)(waves * kblocks);
  double best = 0;
  int splits = 1, tn = 128;
  for (int s = 1; s <= 8; s *= 2) {
    const int64_t ctas = small * s, per = (kblocks + s - 1) / s;
    const int64_t rounds = (ctas + num_sms - 1) / num_sms;
    const double t = 3.4 + (s > 1 ? 4.5 + 0.25 * s : 0.) + 0.27 * (double)(per * rounds);
    if (s == 1 || t < best) best = t, splits = s;
  }
  const double share = 0.165 * (double)((narrow + num_sms - 1) / num_sms);
  const double t64 = 2.7 + (share > 0.255 ? share : 0.255) * (double)kblocks;
  if (t64 < best) best = t64, splits = 1, tn = 64;
  if (f_splits >= 0) splits = f_splits;
  if (f_tn >= 0) tn = f_tn / 64 * 64;
  if (splits > 1) tn = 128;
  const bool pair = f_pair >= 0 ? f_pair == 1 : pair_time < best;
  return pair ? launch_newton_pair(p, wd, stream) : launch_newton_small(p, tn, splits, num_sms, wd, stream);
}

// Steps of group number `group`, which begins at step k.
int group_steps(const Orthogonalize &p, int k, int group) {
  const int64_t m = p.rows < p.cols ? p.rows : p.cols, n = p.rows < p.cols ? p.cols : p.rows;
  const double most = group == 0 || (group > 1 && m >= 512 && 4 * n > 5 * m) ? 16. : 0.;
  double growth = 1.;
  int steps = 1;
  while (k + steps < p.steps) {
    const double a = p.coefficients[3 * (k + steps - 1)];
    growth *= a * a;
    if (!(growth <= most)) break;
    ++steps;
  }
  return steps;
}

// X in fp16 (rows of `ldt`, a multiple of 8) as X 2^(8 - e), and *factor = 2^e /
// (norm + eps): X 2^(8 - e) factor / 256 is X / (norm + eps).  Of an fp32 X, T_lo is what T
// leaves.  partial: three floats for each of scale_blocks() blocks.
cudaError_t scale_to_fp16(int dtype, int rows, int cols, const void *X, int64_t ldx, float eps, __half *T,
                          __half *T_lo, int64_t ldt, float *factor, float *partial, int num_sms, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_F32:
      return launch_scale<float>(rows, cols, X, ldx, eps, T, T_lo, ldt, factor, partial, num_sms, stream);
    case DGEMM_DTYPE_BF16:
      return launch_scale<__nv_bfloat16>(rows, cols, X, ldx, eps, T, nullptr, ldt, factor, partial, num_sms, stream);
    default:
      return launch_scale<__half>(rows, cols, X, ldx, eps, T, nullptr, ldt, factor, partial, num_sms, stream);
  }
}

}  // namespace

size_t newton_workspace(int rows, int cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return Work(nullptr, rows, cols).bytes;
}

cudaError_t launch_orthogonalize(const Orthogonalize &p, void *work, int num_sms, cudaStream_t stream) {
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  if (num_sms > 512) return cudaErrorInvalidDevice;
  Work w(work, p.rows, p.cols);
  const bool tall = p.rows > p.cols;
  const int m = tall ? p.cols : p.rows, n = tall ? p.rows : p.cols;
  const int64_t ldx = line_pitch(p.cols, 2), ldm = line_pitch(m, 2);
  cudaError_t e = scale_to_fp16(p.x_dtype, p.rows, p.cols, p.X, p.ldx, p.eps, w.x[0], w.x[2], ldx,
                                w.factor, w.partial, num_sms, stream);
  const float x_up = 0x1p8f, m_up = 0x1p6f;  // what X and the m x m matrices are kept times
  __half *x = w.x[0], *x_next = w.x[1];
  // (one row or column has no other directions in which its rounding would be enlarged)
  const __half *lo = p.x_dtype == DGEMM_DTYPE_F32 && m > 1 ? w.x[2] : nullptr;
  for (int k = 0, group = 0; k < p.steps && e == cudaSuccess; ++group) {
    const int steps = group_steps(p, k, group);
    __half *A = w.square[0], *W = w.square[1], *P = w.square[2], *Q = nullptr;
    __half *spare[2] = {w.square[3], w.square[4]};
    {  // A = X X^T, or X^T X
      NewtonGemm g;
      g.symmetric = true, g.dtype = DGEMM_DTYPE_F16;
      g.layout = tall ? 2 : 1;
      g.M = g.N = m, g.K = n;
      g.A = g.B = x, g.lda = g.ldb = ldx;
      g.alpha = m_up / (x_up * x_up);
      if (k == 0) g.factor = w.factor, g.power = 2;
      if (k == 0) g.A_lo = g.B_lo = lo;
      g.out = A, g.ldo = g.out_cols = ldm;
      e = run(g, num_sms, wd, stream);
    }
    auto square = [&](const __half *left, const __half *right, __half *out, float alpha) {
      NewtonGemm g;
      g.symmetric = true, g.dtype = DGEMM_DTYPE_F16;
      g.M = g.N = g.K = m;
      g.A = left, g.B = right, g.lda = g.ldb = ldm;
      g.alpha = alpha / m_up;
      g.out = out, g.ldo = g.out_cols = ldm;
      return g;
    };
    for (int i = 0; i < steps && e == cudaSuccess; ++i) {
      const float *c = p.coefficients + 3 * (k + i);
      __half *poly = i == 0 ? spare[0] : P;
      NewtonGemm g = square(A, A, poly, c[2]);  // P = a I + b A + c A^2
      g.in0 = A, g.ldi0 = ldm, g.beta = c[1], g.gamma = c[0] * m_up;
      e = run(g, num_sms, wd, stream);
      const bool more = i + 1 < steps;
      if (e == cudaSuccess && (more || i > 0)) {  // W = A P and Q = Q P, together where both are wanted
        NewtonGemm h = more ? square(A, poly, W, 1.f) : square(Q, poly, spare[1], 1.f);
        if (more && i > 0) h.A2 = Q, h.out2 = spare[1];
        e = run(h, num_sms, wd, stream);
      }
      if (i == 0) {
        Q = poly;  // spare[0]
      } else {
        __half *old = Q;
        Q = spare[1];
        spare[1] = old;
      }
      if (e == cudaSuccess && more) e = run(square(W, poly, A, 1.f), num_sms, wd, stream);
    }
    if (e != cudaSuccess) break;
    {  // X = Q X, or X Q
      const bool last = k + steps == p.steps;
      NewtonGemm g;
      g.layout = tall ? 1 : 0;
      g.M = p.rows, g.N = p.cols, g.K = m;
      g.A = tall ? x : Q, g.lda = tall ? ldx : ldm;
      g.B = tall ? Q : x, g.ldb = tall ? ldm : ldx;
      if (k == 0) g.factor = w.factor, g.power = 1;
      if (k == 0) (tall ? g.A_lo : g.B_lo) = lo;
      if (last) {
        g.dtype = p.dtype;
        g.alpha = p.scale / (x_up * m_up);
        g.beta = p.residual_scale, g.in0 = p.R, g.ldi0 = p.ldr;
        g.out = p.D, g.ldo = p.ldd, g.out_cols = p.cols;
      } else {
        g.dtype = DGEMM_DTYPE_F16;
        g.alpha = 1.f / m_up;
        g.out = x_next, g.ldo = g.out_cols = ldx;
      }
      e = run(g, num_sms, wd, stream);
    }
    __half *t = x;
    x = x_next, x_next = t;
    k += steps;
  }
  return e;
}

}  // namespace dg
