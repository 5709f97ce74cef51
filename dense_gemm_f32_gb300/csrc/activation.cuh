// activation.cuh -- element types and activation functions of the
// feed-forward operators (norm.cu, rowops.cu, the fused GEMM epilogues).
//
// Every activation and derivative is evaluated in fp32; only the store of a
// result rounds to 16 bits.  A value is off by less than 2^-15 of itself on |z| <=
// 8, in the lower tail too, and a derivative by that much of its terms, far below
// the 2^-8 or 2^-11 of the store (the arguments of the exponentials are rounded, and
// exp amplifies that by up to 50).  The special-function unit's 2^x and 1/x
// without subnormals are 4 instructions per sigmoid against 14 with CUDA's
// subnormal-safe forms, which made the epilogue of a 16384 x 14336 x 4096
// gelu_tanh layer as long as its main loop.
#pragma once

#include <cstdint>
#include <cstring>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/dgemm.h"

namespace dg {

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Two neighbouring 16-bit elements packed in a 32-bit word.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 2^x and 1/x by the special-function unit (about 2 units in the last place,
// subnormals to zero).
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + 2^-t), the sigmoid of t / log2(e): 2^-t overflows to infinity for
// t < -128, giving 0.
__device__ __forceinline__ float sigmoid2(float t) { return rcp_approx(1.f + exp2_approx(-t)); }

// Phi(-|z|), and e = exp(-z^2 / 2).  Phi(-y) exp(y^2 / 2) falls smoothly from 1/2
// like 1 / y, so with t = 1 / (1 + 0.24 y) it is t times a polynomial in t: degree 7,
// coefficients from a weighted least-squares fit iterated to the least largest
// relative error on 0 <= y <= 40 (4.3e-7 of the value; in fp32 3.4e-6 on y <= 9, most
// of it the rounding of the exponential's argument).  erff loses the lower tail,
// 1 + erf(z / sqrt 2) is 5% off at z = -5 and 0 at -6; erfcf keeps it.  A linear
// layer of 8192 x 4096 x 1024 (rows, outputs, K) took 103 us with erff, 148 with
// erfcf, 95 with this.
__device__ __forceinline__ float normal_tail(float z, float &e) {
  const float t = rcp_approx(fmaf(0.24f, fabsf(z), 1.f));
  e = exp2_approx(-0.5f * kLog2e * z * z);
  float p = -0.0529904554f;
  p = fmaf(p, t, 0.152788501f);
  p = fmaf(p, t, -0.0656932143f);
  p = fmaf(p, t, 0.118379911f);
  p = fmaf(p, t, 0.0634018759f);
  p = fmaf(p, t, 0.0928374757f);
  p = fmaf(p, t, 0.0955223062f);
  p = fmaf(p, t, 0.095753786f);
  return p * t * e;
}

// act(z):
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z sigmoid(2 a (z + b z^3)) = z / 2 (1 + tanh(a (z + b z^3)))
//   silu       z sigmoid(z)
template <int ACT>
__device__ __forceinline__ float act_f32(float z) {
  if constexpr (ACT == DGEMM_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays a NaN
  if constexpr (ACT == DGEMM_ACT_GELU) {
    float e;
    const float tail = normal_tail(z, e);
    return z * (z < 0.f ? tail : 1.f - tail);
  }
  if constexpr (ACT == DGEMM_ACT_GELU_TANH)
    return z * sigmoid2(z * fmaf(2.f * kGeluA * kGeluB * kLog2e, z * z, 2.f * kGeluA * kLog2e));
  if constexpr (ACT == DGEMM_ACT_SILU) return z * sigmoid2(kLog2e * z);
  return z;
}

// act(z) and act'(z) together; the derivative of relu at 0 is 0.
template <int ACT>
__device__ __forceinline__ void act_grad_f32(float z, float &value, float &slope) {
  if constexpr (ACT == DGEMM_ACT_RELU) {
    value = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == DGEMM_ACT_GELU) {
    float e;
    const float tail = normal_tail(z, e), cdf = z < 0.f ? tail : 1.f - tail;
    value = z * cdf;
    slope = fmaf(z * 0.3989422804014327f, e, cdf);
  } else if constexpr (ACT == DGEMM_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float s = sigmoid2(z * fmaf(2.f * kGeluA * kGeluB * kLog2e, z2, 2.f * kGeluA * kLog2e));
    value = z * s;
    // where z^2 is past fp32's range value (1 - s) is 0, and has to stay 0
    slope = fmaf(value * (1.f - s), fmaf(6.f * kGeluA * kGeluB, fminf(z2, 1e30f), 2.f * kGeluA), s);
  } else if constexpr (ACT == DGEMM_ACT_SILU) {
    const float s = sigmoid2(kLog2e * z);
    value = z * s;
    slope = fmaf(value, 1.f - s, s);
  } else {
    value = z;
    slope = 1.f;
  }
}

// The activation is a run-time argument of the kernels (a warp-uniform
// branch per group of elements).
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
  switch (act) {
    case DGEMM_ACT_RELU: f(std::integral_constant<int, DGEMM_ACT_RELU>{}); break;
    case DGEMM_ACT_GELU: f(std::integral_constant<int, DGEMM_ACT_GELU>{}); break;
    case DGEMM_ACT_GELU_TANH: f(std::integral_constant<int, DGEMM_ACT_GELU_TANH>{}); break;
    case DGEMM_ACT_SILU: f(std::integral_constant<int, DGEMM_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, DGEMM_ACT_NONE>{}); break;
  }
}

}  // namespace dg
