// norm.cu -- layer norm over the rows of a matrix, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps)
//   y = (x - mu) rstd w + b
//   with xh = (x - mu) rstd and p = dy w:
//   dx = rstd (p - mean(p) - xh mean(p xh)) [+ dr]
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: forward one read and one write of the matrix, backward two
// (three) reads and one write.  A row is held in registers by the threads that
// share it, so it is read once and the variance is that of the centred values
// (two passes over registers).  Short rows take a warp each (no block
// barrier), longer ones a block of 256 to 1024 threads, at most 16 (32 for a
// warp) elements per thread; rows beyond 16384 elements are read again for
// each pass (from L2).  The backward kernel is persistent: a thread keeps the
// same columns for every row its block takes, so the column sums of dw and db
// stay in its registers and each block writes one partial sum, which a second
// launch adds up in a fixed order.
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace dg {
namespace {

// A row's share of a thread: CH vectors, vector c at column (c * GROUP + index
// in the group) * V.  GROUP threads share a row; a block holds BLOCK / GROUP
// rows.  The share does not depend on the rows' alignment, so neither do the
// sums.
template <class T_, bool ALIGNED_, int CH_, int GROUP_>
struct Shape {
  using T = T_;
  static constexpr bool ALIGNED = ALIGNED_;
  static constexpr int V = kVec<T_>, CH = CH_, GROUP = GROUP_;
  static constexpr int BLOCK = GROUP == 32 ? 128 : GROUP, ROWS = BLOCK / GROUP;
  static constexpr int CAPACITY = GROUP * CH * V;
};

// Sums of N values over the threads of a row; every thread gets them.  `red`
// alternates between two buffers, so one barrier per sum is enough.
template <class S, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[32]) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (S::GROUP > 32) {
    constexpr int W = S::GROUP / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = lane < W ? red[i][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (o < W) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[i] = __shfl_sync(0xffffffffu, s, 0);
    }
  }
}

template <class S>
__global__ void __launch_bounds__(S::BLOCK)
    ln_fwd_kernel(int rows, int cols, float eps, const typename S::T *X, int64_t ldx,
                  const typename S::T *w, const typename S::T *b, typename S::T *Y, int64_t ldy,
                  float *mean, float *rstd) {
  using T = typename S::T;
  constexpr int V = S::V, CH = S::CH, GROUP = S::GROUP;
  __shared__ float red[2][1][32];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % GROUP;
  const int64_t row = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / GROUP;
  if (GROUP == 32 && row >= rows) return;
  const T *x = X + row * ldx;
  float v[CH][V], s[1] = {0.f};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    widen16<T>(load_row16<T, S::ALIGNED>(x, (c * GROUP + t) * V, cols), v[c]);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) s[0] += v[c][j];
  row_sum<S>(s, red[0]);
  const float mu = s[0] / cols;
  s[0] = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[c][j] -= mu;
      if ((c * GROUP + t) * V + (S::ALIGNED ? 0 : j) < cols) s[0] += v[c][j] * v[c][j];
    }
  row_sum<S>(s, red[1]);
  const float r = rsqrtf(s[0] / cols + eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * GROUP + t) * V;
    float g[V], h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = 1.f, h[j] = 0.f;
    if (w) widen16<T>(load_row16<T, S::ALIGNED>(w, col, cols), g);
    if (b) widen16<T>(load_row16<T, S::ALIGNED>(b, col, cols), h);
#pragma unroll
    for (int j = 0; j < V; ++j) v[c][j] = v[c][j] * r * g[j] + h[j];
    store_row16<T, S::ALIGNED>(Y + row * ldy, col, cols, narrow16<T>(v[c]));
  }
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

// dX, and this block's partial sums of dw and db: partial[block][0][col] and
// partial[block][1][col] (or dw and db themselves when there is one block).
template <class S>
__global__ void __launch_bounds__(S::BLOCK, S::BLOCK <= 256 ? 2 : 1)
    ln_bwd_kernel(int rows, int cols, const typename S::T *dY, int64_t lddy,
                  const typename S::T *X, int64_t ldx, const typename S::T *w, const float *mean,
                  const float *rstd, const typename S::T *dR, int64_t lddr, typename S::T *dX,
                  int64_t lddx, float *partial, typename S::T *dw, typename S::T *db) {
  using T = typename S::T;
  constexpr int V = S::V, CH = S::CH, GROUP = S::GROUP;
  __shared__ float red[2][2][32];
  __shared__ float fold[S::ROWS > 1 ? S::ROWS : 1][S::ROWS > 1 ? S::CAPACITY : 1];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % GROUP, sub = threadIdx.x / GROUP;
  const bool grads = partial != nullptr || dw != nullptr || db != nullptr;
  float sw[CH][V], sb[CH][V], g[CH][V];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < V; ++j) sw[c][j] = sb[c][j] = 0.f, g[c][j] = 1.f;
    if (w) widen16<T>(load_row16<T, S::ALIGNED>(w, (c * GROUP + t) * V, cols), g[c]);
  }
  const float inv = 1.f / cols;
  const int64_t step = (int64_t)gridDim.x * S::ROWS;
  int64_t row = (int64_t)blockIdx.x * S::ROWS + sub;
  // the next row's loads are in flight while a row is reduced
  uint4 rd[CH], rx[CH], rr[CH];
  float mu = 0.f, r = 0.f;
  auto fetch = [&](int64_t i) {
    mu = mean[i], r = rstd[i];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * GROUP + t) * V;
      rd[c] = load_row16<T, S::ALIGNED>(dY + i * lddy, col, cols);
      rx[c] = load_row16<T, S::ALIGNED>(X + i * ldx, col, cols);
    }
  };
  auto fetch_skip = [&](int64_t i) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      rr[c] = make_uint4(0u, 0u, 0u, 0u);
      if (dR != nullptr)
        rr[c] = load_row16<T, S::ALIGNED>(dR + i * lddr, (c * GROUP + t) * V, cols);
    }
  };
  if (row < rows) {
    fetch(row);
    fetch_skip(row);
  }
  int buf = 0;
  for (; row < rows; row += step) {
    float d[CH][V], xh[CH][V], s[2] = {0.f, 0.f};
    const float r_now = r;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      widen16<T>(rd[c], d[c]);
      widen16<T>(rx[c], xh[c]);
#pragma unroll
      for (int j = 0; j < V; ++j) {  // past the row's end d is 0, and with it every term
        xh[c][j] = (xh[c][j] - mu) * r;
        const float p = d[c][j] * g[c][j];
        s[0] += p;
        s[1] += p * xh[c][j];
        sw[c][j] += d[c][j] * xh[c][j];
        sb[c][j] += d[c][j];
      }
    }
    if (row + step < rows) fetch(row + step);
    row_sum<S>(s, red[buf]);
    buf ^= 1;
    const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * GROUP + t) * V;
      float e[V];
      widen16<T>(rr[c], e);
#pragma unroll
      for (int j = 0; j < V; ++j) e[j] += r_now * (d[c][j] * g[c][j] - m1 - xh[c][j] * m2);
      store_row16<T, S::ALIGNED>(dX + row * lddx, col, cols, narrow16<T>(e));
    }
    if (row + step < rows) fetch_skip(row + step);
  }
  if (!grads) return;
  // the block's rows side by side, added in their order
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float(&sum)[CH][V] = k ? sb : sw;
    if constexpr (S::ROWS > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) fold[sub][(c * GROUP + t) * V + j] = sum[c][j];
      __syncthreads();
    }
    T *out = k ? db : dw;
    float *part = partial ? partial + ((int64_t)blockIdx.x * 2 + k) * cols : nullptr;
    if constexpr (S::ROWS > 1) {
      for (int col = threadIdx.x; col < cols; col += S::BLOCK) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < S::ROWS; ++i) v += fold[i][col];
        if (part)
          part[col] = v;
        else if (out)
          out[col] = from_f32<T>(v);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int col = (c * GROUP + t) * V + j;
          if (col >= cols) continue;
          if (part)
            part[col] = sum[c][j];
          else if (out)
            out[col] = from_f32<T>(sum[c][j]);
        }
    }
  }
}

// ---------------------------------------------- rows too long for registers
template <class T>
struct LongShape {
  static constexpr int GROUP = 1024;
};

template <class T>
__global__ void __launch_bounds__(1024)
    ln_fwd_long_kernel(int cols, float eps, const T *X, int64_t ldx, const T *w, const T *b, T *Y,
                       int64_t ldy, float *mean, float *rstd) {
  __shared__ float red[2][1][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T *x = X + row * ldx;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < cols; c += 1024) s[0] += to_f32<T>(x[c]);
  row_sum<LongShape<T>>(s, red[0]);
  const float mu = s[0] / cols;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < cols; c += 1024) {
    const float d = to_f32<T>(x[c]) - mu;
    s[0] += d * d;
  }
  row_sum<LongShape<T>>(s, red[1]);
  const float r = rsqrtf(s[0] / cols + eps);
  for (int c = threadIdx.x; c < cols; c += 1024)
    Y[row * ldy + c] = from_f32<T>((to_f32<T>(x[c]) - mu) * r * (w ? to_f32<T>(w[c]) : 1.f) +
                                   (b ? to_f32<T>(b[c]) : 0.f));
  if (threadIdx.x == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

template <class T>
__global__ void __launch_bounds__(1024)
    ln_dx_long_kernel(int cols, const T *dY, int64_t lddy, const T *X, int64_t ldx, const T *w,
                      const float *mean, const float *rstd, const T *dR, int64_t lddr, T *dX,
                      int64_t lddx) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const float mu = mean[row], r = rstd[row];
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < cols; c += 1024) {
    const float p = to_f32<T>(dY[row * lddy + c]) * (w ? to_f32<T>(w[c]) : 1.f);
    s[0] += p;
    s[1] += p * (to_f32<T>(X[row * ldx + c]) - mu) * r;
  }
  row_sum<LongShape<T>>(s, red);
  const float m1 = s[0] / cols, m2 = s[1] / cols;
  for (int c = threadIdx.x; c < cols; c += 1024) {
    const float p = to_f32<T>(dY[row * lddy + c]) * (w ? to_f32<T>(w[c]) : 1.f);
    const float xh = (to_f32<T>(X[row * ldx + c]) - mu) * r;
    const float d = r * (p - m1 - xh * m2);
    dX[row * lddx + c] = from_f32<T>(dR ? d + to_f32<T>(dR[row * lddr + c]) : d);
  }
}

// Partial sums of dw and db over the rows of one part, a column per thread.
template <class T>
__global__ void __launch_bounds__(256)
    ln_dw_long_kernel(int rows, int cols, const T *dY, int64_t lddy, const T *X, int64_t ldx,
                      const float *mean, const float *rstd, float *partial) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * 256 + threadIdx.x, parts = gridDim.y, part = blockIdx.y;
  if (c >= cols) return;
  float sw = 0.f, sb = 0.f;
  for (int64_t i = part; i < rows; i += parts) {
    const float d = to_f32<T>(dY[i * lddy + c]);
    sw += d * (to_f32<T>(X[i * ldx + c]) - mean[i]) * rstd[i];
    sb += d;
  }
  partial[((int64_t)part * 2) * cols + c] = sw;
  partial[((int64_t)part * 2 + 1) * cols + c] = sb;
}

// ------------------------------------------------------------- host side
constexpr int kMaxRegisterCols = 16384;

// f(shape) for the shape a row of `cols` elements is held in: the smallest
// group that holds it in at most 16 elements per thread (32 for a warp), since
// more rows per SM then have their loads in flight.
template <class T, bool ALIGNED, class F>
cudaError_t with_shape(int cols, F &&f) {
  constexpr int K = 8 / kVec<T>;  // vectors in 8 elements
  if (cols <= 256) return f(Shape<T, ALIGNED, K, 32>{});
  if (cols <= 512) return f(Shape<T, ALIGNED, 2 * K, 32>{});
  if (cols <= 1024) return f(Shape<T, ALIGNED, 4 * K, 32>{});
  if (cols <= 2048) return f(Shape<T, ALIGNED, K, 256>{});
  if (cols <= 4096) return f(Shape<T, ALIGNED, 2 * K, 256>{});
  if (cols <= 8192) return f(Shape<T, ALIGNED, 2 * K, 512>{});
  return f(Shape<T, ALIGNED, 2 * K, 1024>{});
}
template <class T, class F>
cudaError_t with_shape(int cols, bool aligned, F &&f) {
  return aligned ? with_shape<T, true>(cols, f) : with_shape<T, false>(cols, f);
}

template <class T>
bool vec_ok(const void *p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
}

template <class T>
cudaError_t fwd(int rows, int cols, float eps, const void *X, int64_t ldx, const void *weight,
                const void *bias, void *Y, int64_t ldy, float *mean, float *rstd,
                cudaStream_t stream) {
  const T *x = static_cast<const T *>(X), *w = static_cast<const T *>(weight);
  const T *b = static_cast<const T *>(bias);
  T *y = static_cast<T *>(Y);
  cudaError_t e;
  if (cols > kMaxRegisterCols) {
    e = launch_kernel(ln_fwd_long_kernel<T>, dim3((unsigned)rows), dim3(1024), 0, stream, 1u, cols,
                      eps, x, ldx, w, b, y, ldy, mean, rstd);
  } else {
    const bool vec = vec_ok<T>(X, ldx) && vec_ok<T>(Y, ldy) && vec_ok<T>(w, 0) &&
                     vec_ok<T>(b, 0) && (cols * (int)sizeof(T)) % 16 == 0;
    e = with_shape<T>(cols, vec, [&](auto shape) {
      using S = decltype(shape);
      return launch_kernel(ln_fwd_kernel<S>, dim3((unsigned)((rows + S::ROWS - 1) / S::ROWS)),
                           dim3(S::BLOCK), 0, stream, 1u, rows, cols, eps, x, ldx, w, b, y, ldy,
                           mean, rstd);
    });
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

// Blocks of the backward kernel, each one partial sum: two per SM.
int bwd_parts(int rows, int rows_per_block, int num_sms) {
  const int64_t need = ((int64_t)rows + rows_per_block - 1) / rows_per_block;
  const int64_t most = 2 * (int64_t)num_sms;
  return (int)(need < 1 ? 1 : need < most ? need : most);
}

template <class T>
cudaError_t bwd(int dtype, int rows, int cols, const void *dY, int64_t lddy, const void *X,
                int64_t ldx, const void *weight, const float *mean, const float *rstd,
                const void *dR, int64_t lddr, void *dX, int64_t lddx, void *dweight, void *dbias,
                float *partial, int num_sms, cudaStream_t stream) {
  const T *dy = static_cast<const T *>(dY), *x = static_cast<const T *>(X);
  const T *w = static_cast<const T *>(weight), *dr = static_cast<const T *>(dR);
  T *dx = static_cast<T *>(dX), *dw = static_cast<T *>(dweight), *db = static_cast<T *>(dbias);
  const bool grads = dw != nullptr || db != nullptr;
  cudaError_t e = cudaSuccess;
  int parts = 1;
  if (cols > kMaxRegisterCols) {
    if (rows > 0) {
      e = launch_kernel(ln_dx_long_kernel<T>, dim3((unsigned)rows), dim3(1024), 0, stream, 1u, cols,
                        dy, lddy, x, ldx, w, mean, rstd, dr, lddr, dx, lddx);
      if (e != cudaSuccess) return e;
      count_launch();
    }
    if (!grads) return e;
    const unsigned gx = (unsigned)((cols + 255) / 256);
    parts = rows < 16 ? (rows < 1 ? 1 : rows) : 16;
    e = launch_kernel(ln_dw_long_kernel<T>, dim3(gx, (unsigned)parts), dim3(256), 0, stream, 1u,
                      rows, cols, dy, lddy, x, ldx, mean, rstd, partial);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_column_sums(dtype, partial, parts, cols, dw, db, stream);
  }
  const bool vec = vec_ok<T>(dY, lddy) && vec_ok<T>(X, ldx) && vec_ok<T>(w, 0) &&
                   vec_ok<T>(dr, dr ? lddr : 0) && vec_ok<T>(dX, lddx) &&
                   (cols * (int)sizeof(T)) % 16 == 0;
  e = with_shape<T>(cols, vec, [&](auto shape) {
    using S = decltype(shape);
    parts = bwd_parts(rows, S::ROWS, num_sms);
    return launch_kernel(ln_bwd_kernel<S>, dim3((unsigned)parts), dim3(S::BLOCK), 0, stream, 1u,
                         rows, cols, dy, lddy, x, ldx, w, mean, rstd, dr, lddr, dx, lddx,
                         grads && parts > 1 ? partial : nullptr, dw, db);
  });
  if (e != cudaSuccess) return e;
  count_launch();
  return grads && parts > 1 ? launch_column_sums(dtype, partial, parts, cols, dw, db, stream) : e;
}

}  // namespace

cudaError_t launch_layer_norm(int dtype, int rows, int cols, float eps, const void *X, int64_t ldx,
                              const void *weight, const void *bias, void *Y, int64_t ldy,
                              float *mean, float *rstd, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return fwd<__nv_bfloat16>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
    case DGEMM_DTYPE_F16:
      return fwd<__half>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
    default:
      return fwd<float>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
  }
}

size_t layer_norm_scratch(int rows, int cols, bool with_grads, int num_sms) {
  if (!with_grads) return 0;
  const int parts = cols > kMaxRegisterCols ? 16 : bwd_parts(rows, 1, num_sms);
  return (size_t)parts * 2 * cols * sizeof(float);
}

cudaError_t launch_layer_norm_backward(int dtype, int rows, int cols, const void *dY, int64_t lddy,
                                       const void *X, int64_t ldx, const void *weight,
                                       const float *mean, const float *rstd, const void *dR,
                                       int64_t lddr, void *dX, int64_t lddx, void *dweight,
                                       void *dbias, float *partial, int num_sms,
                                       cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return bwd<__nv_bfloat16>(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr,
                                dX, lddx, dweight, dbias, partial, num_sms, stream);
    case DGEMM_DTYPE_F16:
      return bwd<__half>(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX,
                         lddx, dweight, dbias, partial, num_sms, stream);
    default:
      return bwd<float>(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX,
                        lddx, dweight, dbias, partial, num_sms, stream);
  }
}

}  // namespace dg
