// norm.cu -- layer norm over the rows of a matrix, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps)
//   y = (x - mu) rstd w + b
//   with xh = (x - mu) rstd and p = dy w:
//   dx = rstd (p - mean(p) - xh mean(p xh)) [+ dr]
//   dw = sum over rows of dy xh,  db = sum over rows of dy
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"

namespace dg {
namespace {

constexpr int kThreads = 256;

// Sum over the block; every thread gets it.  `red` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float *red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];
  return s;
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    ln_fwd_kernel(int cols, float eps, const T *X, int64_t ldx, const T *w, const T *b, T *Y,
                  int64_t ldy, float *mean, float *rstd) {
  __shared__ float red[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const T *x = X + (int64_t)blockIdx.x * ldx;
  float s = 0.f;
  for (int c = threadIdx.x; c < cols; c += kThreads) s += to_f32<T>(x[c]);
  const float mu = block_sum(s, red) / cols;
  s = 0.f;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const float d = to_f32<T>(x[c]) - mu;
    s += d * d;
  }
  const float r = rsqrtf(block_sum(s, red) / cols + eps);
  for (int c = threadIdx.x; c < cols; c += kThreads)
    Y[(int64_t)blockIdx.x * ldy + c] =
        from_f32<T>((to_f32<T>(x[c]) - mu) * r * (w ? to_f32<T>(w[c]) : 1.f) +
                    (b ? to_f32<T>(b[c]) : 0.f));
  if (threadIdx.x == 0) {
    if (mean) mean[blockIdx.x] = mu;
    if (rstd) rstd[blockIdx.x] = r;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    ln_dx_kernel(int cols, const T *dY, int64_t lddy, const T *X, int64_t ldx, const T *w,
                 const float *mean, const float *rstd, const T *dR, int64_t lddr, T *dX,
                 int64_t lddx) {
  __shared__ float red[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const float mu = mean[row], r = rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const float p = to_f32<T>(dY[row * lddy + c]) * (w ? to_f32<T>(w[c]) : 1.f);
    s1 += p;
    s2 += p * (to_f32<T>(X[row * ldx + c]) - mu) * r;
  }
  const float m1 = block_sum(s1, red) / cols, m2 = block_sum(s2, red) / cols;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const float p = to_f32<T>(dY[row * lddy + c]) * (w ? to_f32<T>(w[c]) : 1.f);
    const float xh = (to_f32<T>(X[row * ldx + c]) - mu) * r;
    const float d = r * (p - m1 - xh * m2);
    dX[row * lddx + c] = from_f32<T>(dR ? d + to_f32<T>(dR[row * lddr + c]) : d);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    ln_dw_kernel(int rows, int cols, const T *dY, int64_t lddy, const T *X, int64_t ldx,
                 const float *mean, const float *rstd, T *dw, T *db) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= cols) return;
  float sw = 0.f, sb = 0.f;
  for (int64_t i = 0; i < rows; ++i) {
    const float d = to_f32<T>(dY[i * lddy + c]);
    sw += d * (to_f32<T>(X[i * ldx + c]) - mean[i]) * rstd[i];
    sb += d;
  }
  if (dw) dw[c] = from_f32<T>(sw);
  if (db) db[c] = from_f32<T>(sb);
}

template <class T>
cudaError_t fwd(int rows, int cols, float eps, const void *X, int64_t ldx, const void *weight,
                const void *bias, void *Y, int64_t ldy, float *mean, float *rstd,
                cudaStream_t stream) {
  const cudaError_t e = launch_kernel(
      ln_fwd_kernel<T>, dim3((unsigned)rows), dim3(kThreads), 0, stream, 1u, cols, eps,
      static_cast<const T *>(X), ldx, static_cast<const T *>(weight), static_cast<const T *>(bias),
      static_cast<T *>(Y), ldy, mean, rstd);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class T>
cudaError_t bwd(int rows, int cols, const void *dY, int64_t lddy, const void *X, int64_t ldx,
                const void *weight, const float *mean, const float *rstd, const void *dR,
                int64_t lddr, void *dX, int64_t lddx, void *dweight, void *dbias,
                cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    e = launch_kernel(
      ln_dx_kernel<T>, dim3((unsigned)rows), dim3(kThreads), 0, stream, 1u, cols,
      static_cast<const T *>(dY), lddy, static_cast<const T *>(X), ldx,
      static_cast<const T *>(weight), mean, rstd, static_cast<const T *>(dR), lddr,
      static_cast<T *>(dX), lddx);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  if (!dweight && !dbias) return e;
  e = launch_kernel(ln_dw_kernel<T>, dim3((unsigned)((cols + kThreads - 1) / kThreads)),
                    dim3(kThreads), 0, stream, 1u, rows, cols, static_cast<const T *>(dY), lddy,
                    static_cast<const T *>(X), ldx, mean, rstd, static_cast<T *>(dweight),
                    static_cast<T *>(dbias));
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_layer_norm(int dtype, int rows, int cols, float eps, const void *X, int64_t ldx,
                              const void *weight, const void *bias, void *Y, int64_t ldy,
                              float *mean, float *rstd, int, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return fwd<__nv_bfloat16>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
    case DGEMM_DTYPE_F16:
      return fwd<__half>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
    default:
      return fwd<float>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
  }
}

size_t layer_norm_scratch(int, int, bool, int) { return 0; }

cudaError_t launch_layer_norm_backward(int dtype, int rows, int cols, const void *dY, int64_t lddy,
                                       const void *X, int64_t ldx, const void *weight,
                                       const float *mean, const float *rstd, const void *dR,
                                       int64_t lddr, void *dX, int64_t lddx, void *dweight,
                                       void *dbias, float *, int, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return bwd<__nv_bfloat16>(rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX,
                                lddx, dweight, dbias, stream);
    case DGEMM_DTYPE_F16:
      return bwd<__half>(rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX, lddx,
                         dweight, dbias, stream);
    default:
      return bwd<float>(rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX, lddx,
                        dweight, dbias, stream);
  }
}

}  // namespace dg
