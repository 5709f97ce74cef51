// epilogue.cuh -- the arithmetic of the fused products' epilogues, on 32
// consecutive columns of one row held by one thread.
#pragma once

#include <cstdint>

#include "activation.cuh"
#include "ops.h"

namespace dg {

// 32 columns of one row of a 16-bit matrix, packed in pairs; columns from
// `valid` on read as zero.  vec: the row is 16-byte aligned here.  Plain
// loads: the row may be overwritten by this call's own output later on.
template <class T>
__device__ __forceinline__ void load32(const T *p, int valid, bool vec, uint32_t (&w)[16]) {
  if (vec && valid >= 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + 8 * q);
      w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
    }
  } else {
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t lo = 2 * j < valid ? h[2 * j] : 0u, hi = 2 * j + 1 < valid ? h[2 * j + 1] : 0u;
      w[j] = lo | (hi << 16);
    }
  }
}

// kLinear: z (with the bias added) in a, the residual's words in i0 when
// has_in0; D in w0, Z in w1.
// kGated: g in a, u in b; H in w0, G in w1, U in w2.
// kGatedBwd: dh in a, the words of G and U in i0 and i1; dG, dU, H in w0..w2.
// Everything is fp32 until the one rounding of each packed result.
template <Epi EPI, class T>
__device__ __forceinline__ void epilogue32(int act, bool has_in0, const float (&a)[32],
                                           const float (&b)[32], const uint32_t (&i0)[16],
                                           const uint32_t (&i1)[16], uint32_t (&w0)[16],
                                           uint32_t (&w1)[16], uint32_t (&w2)[16]) {
  if constexpr (EPI != Epi::kGatedBwd) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      w1[j] = pack2<T>(a[2 * j], a[2 * j + 1]);
      if constexpr (EPI == Epi::kGated) w2[j] = pack2<T>(b[2 * j], b[2 * j + 1]);
    }
  }
  with_act(act, [&](auto c) {
    constexpr int ACT = decltype(c)::value;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if constexpr (EPI == Epi::kLinear) {
        float lo = act_f32<ACT>(a[2 * j]), hi = act_f32<ACT>(a[2 * j + 1]);
        if (has_in0) {
          const float2 r = unpack2<T>(i0[j]);
          lo += r.x, hi += r.y;
        }
        w0[j] = pack2<T>(lo, hi);
      } else if constexpr (EPI == Epi::kGated) {
        w0[j] = pack2<T>(act_f32<ACT>(a[2 * j]) * b[2 * j],
                         act_f32<ACT>(a[2 * j + 1]) * b[2 * j + 1]);
      } else {
        const float2 g = unpack2<T>(i0[j]), u = unpack2<T>(i1[j]);
        float v0, s0, v1, s1;
        act_grad_f32<ACT>(g.x, v0, s0);
        act_grad_f32<ACT>(g.y, v1, s1);
        w0[j] = pack2<T>(a[2 * j] * u.x * s0, a[2 * j + 1] * u.y * s1);
        w1[j] = pack2<T>(a[2 * j] * v0, a[2 * j + 1] * v1);
        w2[j] = pack2<T>(v0 * u.x, v1 * u.y);
      }
    }
  });
}

}  // namespace dg
