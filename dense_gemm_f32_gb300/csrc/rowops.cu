// rowops.cu -- the element-wise half of a linear layer's backward pass:
// dZ = dD act'(Z), with the bias gradient's column sums in the same pass.
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"

namespace dg {
namespace {

template <class T>
__global__ void act_grad_kernel(int act, int M, int N, const T *dD, int64_t lddd, const T *Z,
                                int64_t ldz, T *dZ, int64_t lddz, T *dbias) {
  pdl_launch_dependents();
  pdl_wait();
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= N) return;
  float sum = 0.f;
  for (int i = 0; i < M; ++i) {
    float d = to_f32<T>(dD[(int64_t)i * lddd + j]);
    with_act(act, [&](auto a) {
      constexpr int ACT = decltype(a)::value;
      if constexpr (ACT != DGEMM_ACT_NONE) {
        float value, slope;
        act_grad_f32<ACT>(to_f32<T>(Z[(int64_t)i * ldz + j]), value, slope);
        d *= slope;
        dZ[(int64_t)i * lddz + j] = from_f32<T>(d);
      }
    });
    sum += d;
  }
  if (dbias) dbias[j] = from_f32<T>(sum);
}

template <class T>
cudaError_t act_grad(int act, int M, int N, const void *dD, int64_t lddd, const void *Z,
                     int64_t ldz, void *dZ, int64_t lddz, void *dbias, cudaStream_t stream) {
  const cudaError_t e = launch_kernel(
      act_grad_kernel<T>, dim3((unsigned)((N + 127) / 128)), dim3(128), 0, stream, 1u, act, M, N,
      static_cast<const T *>(dD), lddd, static_cast<const T *>(Z), ldz, static_cast<T *>(dZ), lddz,
      static_cast<T *>(dbias));
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

size_t act_grad_scratch(int, int, bool, int) { return 0; }

cudaError_t launch_act_grad(int dtype, int act, int M, int N, const void *dD, int64_t lddd,
                            const void *Z, int64_t ldz, void *dZ, int64_t lddz, void *dbias,
                            float *, int, cudaStream_t stream) {
  return dtype == DGEMM_DTYPE_BF16
             ? act_grad<__nv_bfloat16>(act, M, N, dD, lddd, Z, ldz, dZ, lddz, dbias, stream)
             : act_grad<__half>(act, M, N, dD, lddd, Z, ldz, dZ, lddz, dbias, stream);
}

}  // namespace dg
