// rowops.cu -- the element-wise half of a linear layer's backward pass,
// dZ = dD act'(Z), with the bias gradient's column sums in the same pass, the
// join of column sums that several blocks hold parts of, and the re-pitching
// of 16-bit operands.
//
// dZ is rounded to 16 bits, as the products that read it multiply 16-bit operands;
// the column sums add the values before that rounding.
// Bound by memory: dZ is two reads and one write of an M x N matrix.  A thread
// owns eight columns (16 bytes of a row) and walks every eighth row of its
// block's share, so the column sums stay in registers; the eight row groups of
// a block are added in shared memory, and each block's sums are joined by a
// second launch, everything in a fixed order.
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace dg {
namespace {

constexpr int kGroups = 8;  // row groups (warps) of a block
constexpr int kAhead = 4;   // rows of a thread in flight

template <class T, bool ALIGNED>
__global__ void __launch_bounds__(32 * kGroups)
    act_grad_kernel(int act, int M, int N, const T *dD, int64_t lddd, const T *Z, int64_t ldz,
                    T *dZ, int64_t lddz, float *partial, T *dbias) {
  constexpr int V = kVec<T>, TILE = 32 * V;
  __shared__ float fold[kGroups][TILE];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int col = blockIdx.x * TILE + lane * V;
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.f;
  with_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    const int64_t step = (int64_t)gridDim.y * kGroups;
    for (int64_t i0 = (int64_t)blockIdx.y * kGroups + group; i0 < M; i0 += kAhead * step) {
      RowBlocks dr[kAhead], zr[kAhead];  // all of them in flight before the first is used
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t i = i0 + k * step;
        const int n = i < M ? N : 0;
        dr[k] = fetch_row16<T, ALIGNED>(dD + i * lddd, col, n);
        if (ACT != DGEMM_ACT_NONE) zr[k] = fetch_row16<T, ALIGNED>(Z + i * ldz, col, n);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t i = i0 + k * step;
        if (i >= M) break;
        float d[V];
        widen16<T>(take_row16<T, ALIGNED>(dr[k], dD + i * lddd, col, N), d);
        if constexpr (ACT != DGEMM_ACT_NONE) {
          float z[V];
          widen16<T>(take_row16<T, ALIGNED>(zr[k], Z + i * ldz, col, N), z);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float value, slope;
            act_grad_f32<ACT>(z[j], value, slope);
            d[j] *= slope;
          }
          const uint4 out[1] = {narrow16<T>(d)};
          store_row16<T, ALIGNED>(dZ + i * lddz, col, N, out);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += d[j];
      }
    }
  });
  if (partial == nullptr && dbias == nullptr) return;
#pragma unroll
  for (int j = 0; j < V; ++j) fold[group][lane * V + j] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < TILE; c += 32 * kGroups) {
    const int out = blockIdx.x * TILE + c;
    if (out >= N) break;
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) v += fold[g][c];
    if (partial)
      partial[(int64_t)blockIdx.y * N + out] = v;
    else
      dbias[out] = from_f32<T>(v);
  }
}

// out[k][col] = sum over parts of partial[part][k][col], k < nvec (gridDim.y).
// 32 columns per block; 16 warps take every 16th part, eight in flight.
constexpr int kSumWarps = 16;
template <class T>
__global__ void __launch_bounds__(32 * kSumWarps)
    column_sums_kernel(const float *partial, int parts, int cols, T *out0, T *out1) {
  __shared__ float fold[kSumWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5, k = blockIdx.y, nvec = gridDim.y;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < cols)
#pragma unroll 8
    for (int i = group; i < parts; i += kSumWarps)
      v += partial[((int64_t)i * nvec + k) * cols + col];
  fold[group][lane] = v;
  __syncthreads();
  T *out = k ? out1 : out0;
  if (group != 0 || col >= cols || out == nullptr) return;
  v = 0.f;
#pragma unroll
  for (int g = 0; g < kSumWarps; ++g) v += fold[g][lane];
  out[col] = from_f32<T>(v);
}

struct RepitchJobs {
  RepitchJob job[kMaxRepitch];
  int64_t first[kMaxRepitch + 1];  // units (256 columns of a row) before each job
  int n;
};

// A warp takes kUnits neighbouring units (256 columns of a row each), all of
// their loads in flight at once: 16-byte blocks shifted to the aligned pitch,
// 16-byte stores.  One division per warp and round, the units after the first
// follow by counting, and every load of a round is issued before the first is
// used (GB300: staging 33 MB of weights for 15 rows takes 12 us; one vector at a
// time took 18).
constexpr int kUnits = 4;
__global__ void __launch_bounds__(256) repitch_kernel(const __grid_constant__ RepitchJobs jobs) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t total = jobs.first[jobs.n];
  for (int64_t u0 = kUnits * ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)); u0 < total;
       u0 += 8 * kUnits * (int64_t)gridDim.x) {
    int j = 0;
    while (u0 >= jobs.first[j + 1]) ++j;
    int per_row = (int)((jobs.job[j].ldd + 255) / 256);
    int64_t row = (u0 - jobs.first[j]) / per_row;
    int unit = (int)(u0 - jobs.first[j] - row * per_row);
    RowBlocks v[kUnits];
    const __half *src[kUnits];
    __half *dst[kUnits];
    int cols[kUnits], at[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      dst[k] = nullptr;
      if (u0 + k >= total) continue;
      const RepitchJob &job = jobs.job[j];
      const int col = unit * 256 + lane * 8;
      src[k] = static_cast<const __half *>(job.src) + row * job.lds;
      at[k] = col, cols[k] = (int)job.cols;
      v[k] = fetch_row16<__half, false>(src[k], col, cols[k]);
      if (col < job.ldd) dst[k] = static_cast<__half *>(job.dst) + row * job.ldd + col;
      if (++unit == per_row) {
        unit = 0;
        if (++row == job.rows && j + 1 < jobs.n) {
          row = 0;
          ++j;
          per_row = (int)((jobs.job[j].ldd + 255) / 256);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
      if (dst[k] != nullptr)
        *reinterpret_cast<uint4 *>(dst[k]) = take_row16<__half, false>(v[k], src[k], at[k], cols[k]);
  }
}

template <class T>
cudaError_t column_sums(const float *partial, int parts, int cols, void *out0, void *out1, int nvec,
                        cudaStream_t stream) {
  const cudaError_t e = launch_kernel(
      column_sums_kernel<T>, dim3((unsigned)((cols + 31) / 32), (unsigned)nvec),
      dim3(32 * kSumWarps), 0, stream, 1u, partial, parts, cols, static_cast<T *>(out0), static_cast<T *>(out1));
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t column_sums(int dtype, const float *partial, int parts, int cols, void *out0,
                        void *out1, int nvec, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return column_sums<__nv_bfloat16>(partial, parts, cols, out0, out1, nvec, stream);
    case DGEMM_DTYPE_F16:
      return column_sums<__half>(partial, parts, cols, out0, out1, nvec, stream);
    default:
      return column_sums<float>(partial, parts, cols, out0, out1, nvec, stream);
  }
}

// Shares of the rows: four blocks per SM over all column tiles, at least four
// rows per row group; up to 128 rows one share, which needs no second launch.
int act_grad_parts(int M, int N, int num_sms) {
  const int64_t tiles = (N + 255) / 256;
  int64_t parts = (4 * (int64_t)num_sms + tiles - 1) / tiles;
  if (M <= 16 * kGroups) return 1;
  const int64_t most = ((int64_t)M + 4 * kGroups - 1) / (4 * kGroups);
  parts = parts < most ? parts : most;
  return (int)(parts < 1 ? 1 : parts);
}

template <class T, bool ALIGNED>
cudaError_t act_grad(int act, int M, int N, const void *dD, int64_t lddd, const void *Z,
                     int64_t ldz, void *dZ, int64_t lddz, void *dbias, float *partial, int parts,
                     cudaStream_t stream) {
  const cudaError_t e = launch_kernel(
      act_grad_kernel<T, ALIGNED>, dim3((unsigned)((N + 255) / 256), (unsigned)parts),
      dim3(32 * kGroups), 0, stream, 1u, act, M, N, static_cast<const T *>(dD), lddd,
      static_cast<const T *>(Z), ldz, static_cast<T *>(dZ), lddz,
      dbias != nullptr && parts > 1 ? partial : nullptr, static_cast<T *>(dbias));
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_column_sums(int dtype, const float *partial, int parts, int cols, void *out0,
                               void *out1, cudaStream_t stream) {
  return column_sums(dtype, partial, parts, cols, out0, out1, 2, stream);
}

size_t act_grad_scratch(int M, int N, bool with_bias, int num_sms) {
  if (!with_bias) return 0;
  return (size_t)act_grad_parts(M, N, num_sms) * N * sizeof(float);
}

cudaError_t launch_act_grad(int dtype, int act, int M, int N, const void *dD, int64_t lddd,
                            const void *Z, int64_t ldz, void *dZ, int64_t lddz, void *dbias,
                            float *partial, int num_sms, cudaStream_t stream) {
  const bool vec = N % 8 == 0 && rows_aligned(dD, lddd) &&
                   (act == DGEMM_ACT_NONE || (rows_aligned(Z, ldz) && rows_aligned(dZ, lddz)));
  const int parts = act_grad_parts(M, N, num_sms);
  auto f = dtype == DGEMM_DTYPE_BF16
               ? (vec ? act_grad<__nv_bfloat16, true> : act_grad<__nv_bfloat16, false>)
               : (vec ? act_grad<__half, true> : act_grad<__half, false>);
  const cudaError_t e =
      f(act, M, N, dD, lddd, Z, ldz, dZ, lddz, dbias, partial, parts, stream);
  if (e != cudaSuccess || dbias == nullptr || parts == 1) return e;
  return column_sums(dtype, partial, parts, N, dbias, nullptr, 1, stream);
}

cudaError_t launch_repitch(const RepitchJob *jobs, int njobs, int num_sms, cudaStream_t stream) {
  RepitchJobs a;
  if (njobs < 1 || njobs > kMaxRepitch) return cudaErrorInvalidValue;
  a.n = njobs;
  a.first[0] = 0;
  for (int j = 0; j < njobs; ++j) {
    a.job[j] = jobs[j];
    a.first[j + 1] = a.first[j] + jobs[j].rows * ((jobs[j].ldd + 255) / 256);
  }
  const int64_t blocks = (a.first[njobs] + 8 * kUnits - 1) / (8 * kUnits), most = 8 * (int64_t)num_sms;
  const cudaError_t e = launch_kernel(repitch_kernel, dim3((unsigned)(blocks < most ? blocks : most)),
                                      dim3(256), 0, stream, 1u, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace dg
