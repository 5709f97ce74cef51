// quant.cuh -- putting a row into 8-bit integers (quant.cu, int8_row.cu).
//
// A row x becomes q_j = round(127 x_j / top), top = max |x_j|, to the nearest
// integer (ties to even), and its scale top / 127, so that x_j is about q_j scale.
// The quotient's nearest integer is exact for 16-bit elements: with a power of
// two that brings top into [1, 4), t = 127 x is exact in fp32 (7 + 11 bits), the
// product with 127 / top finds an integer that is at most one off, next to a
// half, and e = t - q top, exact as well, says on which side of it the quotient
// lies.  (An element costs three products, two of them with a sum, a subtraction and a
// comparison; a division would cost several times that.)  For
// fp32 elements t is rounded once.  The maximum is taken of the bits of |x|, in
// which NaN is the largest: a row with NaN or an infinity gets that as its scale
// and zeros, so that what is computed from it is NaN.  A row of zeros has scale
// 0.
#pragma once

#include <cstdint>

#include "activation.cuh"

namespace dg {

// What a row's largest size says about quantising it.
struct RowScale {
  float up, top, inv;  // a power of two; top times it; 127 / that
  float scale;         // top / 127
  bool none;           // zeros, an infinity or NaN: every q is 0
};
__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  RowScale r;
  const float top = __uint_as_float(top_bits);
  r.none = top_bits == 0u || top_bits >= 0x7f800000u;
  r.scale = r.none ? top : __fdiv_rn(top, 127.f);
  int e = (int)(top_bits >> 23);
  e = e < 1 ? 1 : e > 253 ? 253 : e;
  r.up = __uint_as_float((uint32_t)(254 - e) << 23);
  r.top = top * r.up;
  r.inv = r.none ? 0.f : __fdiv_rn(127.f, r.top);
  return r;
}

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: a sum with it is rounded to an integer

// The integer of one element.
__device__ __forceinline__ float quantised(float x, const RowScale &r) {
  if (r.none) return 0.f;
  x *= r.up;
  const float t = 127.f * x, m = fmaf(x, r.inv, kRound), q = m - kRound;
  const float e = fmaf(-q, r.top, t), twice = 2.f * fabsf(e);
  const bool odd = __float_as_uint(m) & 1u;
  return twice > r.top || (twice == r.top && odd) ? q + copysignf(1.f, e) : q;
}

// The integers of N elements: the side of the half is looked at only where an element
// lies on one or beyond, which takes half the instructions.
template <int N>
__device__ __forceinline__ void quantise_vec(float (&v)[N], const RowScale &r) {
  const float half = 0.5f * r.top;
  bool off = r.none;
  float q[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float x = v[j] * r.up;
    q[j] = fmaf(x, r.inv, kRound) - kRound;
    off |= fabsf(fmaf(-q[j], r.top, 127.f * x)) >= half;
  }
  if (off) {
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = quantised(v[j], r);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = q[j];
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// V integers to `out`: signed bytes, or fp16.
template <int V>
__device__ __forceinline__ void put(int8_t *out, const float (&q)[V], int valid, bool vec) {
  uint32_t w[V / 4];
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    w[j] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[j] |= ((uint32_t)(int)q[4 * j + k] & 0xFFu) << (8 * k);
  }
  if (vec && valid >= V) {
    if constexpr (V == 8)
      *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t *>(out) = w[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < valid) out[j] = (int8_t)(w[j / 4] >> (8 * (j & 3)));
  }
}
template <int V>
__device__ __forceinline__ void put(__half *out, const float (&q)[V], int valid, bool) {
  // the products' tokens: rows of whole vectors, padded
  uint32_t w[V / 2];
#pragma unroll
  for (int j = 0; j < V / 2; ++j) w[j] = pack2<__half>(q[2 * j], q[2 * j + 1]);
  if constexpr (V == 8)
    *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
}

}  // namespace dg
