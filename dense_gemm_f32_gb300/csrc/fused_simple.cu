// fused_simple.cu -- the fused products of the feed-forward operators on the
// CUDA cores: one 64 x 64 tile of the output per block, operands widened to
// fp32 in shared memory, 4 x 4 accumulators per thread.  Right for every
// shape, layout and alignment; bound by fp32 FMA and shared-memory reads.
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"

namespace dg {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;

template <class T>
__device__ __forceinline__ void accumulate(float (&acc)[4][4], const T *A, int64_t lda, bool a_t,
                                           const T *B, int64_t ldb, bool b_t, int M, int N, int K,
                                           int m0, int n0, float (*as)[TM + 1],
                                           float (*bs)[TN + 1]) {
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (int k0 = 0; k0 < K; k0 += TK) {
    for (int e = tid; e < TM * TK; e += 256) {
      const int k = a_t ? e / TM : e % TK, m = a_t ? e % TM : e / TK;
      const bool in = m0 + m < M && k0 + k < K;
      const int64_t at = a_t ? (int64_t)(k0 + k) * lda + m0 + m : (int64_t)(m0 + m) * lda + k0 + k;
      as[k][m] = in ? to_f32<T>(A[at]) : 0.f;
    }
    for (int e = tid; e < TN * TK; e += 256) {
      const int k = b_t ? e % TK : e / TN, n = b_t ? e / TK : e % TN;
      const bool in = n0 + n < N && k0 + k < K;
      const int64_t at = b_t ? (int64_t)(n0 + n) * ldb + k0 + k : (int64_t)(k0 + k) * ldb + n0 + n;
      bs[k][n] = in ? to_f32<T>(B[at]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < TK; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ty * 4 + i] * bs[k][tx * 4 + j];
    __syncthreads();
  }
}

template <class T>
__global__ void __launch_bounds__(256) fused_simple_kernel(FusedGemm p) {
  __shared__ float as[TK][TM + 1], bs[TK][TN + 1];
  pdl_launch_dependents();
  pdl_wait();
  const T *A = static_cast<const T *>(p.A), *B = static_cast<const T *>(p.B);
  const T *A2 = static_cast<const T *>(p.A2), *B2 = static_cast<const T *>(p.B2);
  const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN;
  float acc[4][4] = {}, acc2[4][4] = {};
  if (p.dual == Dual::kPair && blockIdx.z == 1)
    accumulate<T>(acc, A2, p.lda2, p.a_t, B2, p.ldb2, p.b_t, p.M, p.N, p.K, m0, n0, as, bs);
  else
    accumulate<T>(acc, A, p.lda, p.a_t, B, p.ldb, p.b_t, p.M, p.N, p.K, m0, n0, as, bs);
  if (p.dual == Dual::kSum)
    accumulate<T>(acc, A2, p.lda2, p.a_t, B2, p.ldb2, p.b_t, p.M, p.N, p.K, m0, n0, as, bs);
  if (p.dual == Dual::kGated)
    accumulate<T>(acc2, A, p.lda, p.a_t, B2, p.ldb2, p.b_t, p.M, p.N, p.K, m0, n0, as, bs);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  auto out = [&](void *o, int64_t ld, int m, int n, float v) {
    static_cast<T *>(o)[(int64_t)m * ld + n] = from_f32<T>(v);
  };
  auto in = [&](const void *i, int64_t ld, int m, int n) {
    return to_f32<T>(static_cast<const T *>(i)[(int64_t)m * ld + n]);
  };
  with_act(p.act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m >= p.M || n >= p.N) continue;
        const float v = acc[i][j];
        if (p.epi == Epi::kLinear) {
          if (p.dual == Dual::kPair) {
            if (blockIdx.z)
              out(p.out1, p.ldo1, m, n, v);
            else
              out(p.out0, p.ldo0, m, n, v);
            continue;
          }
          const float z = p.bias ? v + to_f32<T>(static_cast<const T *>(p.bias)[n]) : v;
          if (p.out1) out(p.out1, p.ldo1, m, n, z);
          const float d = act_f32<ACT>(z);
          out(p.out0, p.ldo0, m, n, p.in0 ? d + in(p.in0, p.ldi0, m, n) : d);
        } else if (p.epi == Epi::kGated) {
          const float u = acc2[i][j];
          if (p.out1) {
            out(p.out1, p.ldo1, m, n, v);
            out(p.out2, p.ldo2, m, n, u);
          }
          out(p.out0, p.ldo0, m, n, act_f32<ACT>(v) * u);
        } else {
          const float g = in(p.in0, p.ldi0, m, n), u = in(p.in1, p.ldi1, m, n);
          float value, slope;
          act_grad_f32<ACT>(g, value, slope);
          out(p.out0, p.ldo0, m, n, v * u * slope);
          out(p.out1, p.ldo1, m, n, v * value);
          out(p.out2, p.ldo2, m, n, value * u);
        }
      }
  });
}

}  // namespace

cudaError_t launch_fused(const FusedGemm &p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const int64_t gx = (p.N + TN - 1) / TN, gy = (p.M + TM - 1) / TM;
  if (gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)gy, p.dual == Dual::kPair ? 2u : 1u);
  const cudaError_t e =
      p.dtype == DGEMM_DTYPE_BF16
          ? launch_kernel(fused_simple_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, 1u, p)
          : launch_kernel(fused_simple_kernel<__half>, grid, dim3(256), 0, stream, 1u, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace dg
