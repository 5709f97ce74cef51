// epilogue.cuh -- the arithmetic of the fused products' epilogues, on
// consecutive columns of one row held by one thread.
//
// Everything is fp32 until a result is stored.  Results that the next product of
// the same call reads (H; dG, dU; and dZ in rowops.cu) are rounded to the operands'
// 16 bits there, because that is what the tensor cores multiply at full rate; kept in
// 32 bits they would be read and multiplied at half of it.  It costs one rounding per
// element of an intermediate: against the formulas in 64 bits a gated block in bf16 is off by
// 0.0019 of its norm forward and 0.0023 backward, where rounding the results alone gives
// 0.0017 (fp16 0.00024 and 0.00029, 0.00021).  In fp16 an intermediate past 65504 becomes
// infinite.
#pragma once

#include <cstdint>

#include "activation.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace dg {

// Columns col .. col + 31 (col a multiple of 32) of a row on any alignment,
// from the at most five 16-byte blocks they lie in; from column `cols` on zero.
// Not inlined: the loop around it runs from the instruction cache only while
// it is short.
template <class T>
__device__ __noinline__ void load32_unaligned(const T *row, int col, int cols, uint32_t (&w)[16]) {
  const int valid = min(32, cols - col);
  const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15);
  const uint4 *block = reinterpret_cast<const uint4 *>(
      reinterpret_cast<const uint8_t *>(row) - off + (int64_t)col * (int)sizeof(T));
  const int blocks = valid > 0 ? (off + 2 * valid + 15) / 16 : 0;
  uint4 b[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) b[k] = k < blocks ? block[k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 v = shift16<T>(b[q], b[q + 1], off);
    w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
  }
  if (valid < 32) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = 2 * j + 1 < valid ? w[j] : 2 * j < valid ? w[j] & 0xFFFFu : 0u;
  }
}

// 32 columns of one row of a 16-bit matrix, packed in pairs; columns from
// `cols` on read as zero (cols = 0: none are read).  vec: the row is 16-byte
// aligned.  Plain loads: the row may be overwritten by this call's own output
// later on.
template <class T>
__device__ __forceinline__ void load32(const T *row, int col, int cols, bool vec,
                                       uint32_t (&w)[16]) {
  if (vec && col + 32 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 v = *reinterpret_cast<const uint4 *>(row + col + 8 * q);
      w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
    }
  } else {
    uint32_t x[16];
    load32_unaligned<T>(row, col, cols, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = x[j];
  }
}

// One element.  kLinear: z (with the bias added) in a, the residual in i0 when
// has_in0; D in o0 (Z is a itself).  kGated: g in a, u in b; H in o0.
// kGatedBwd: dh in a, G and U in i0 and i1; dG, dU, H in o0, o1, o2.
template <Epi EPI, int ACT>
__device__ __forceinline__ void epilogue1(bool has_in0, float a, float b, float i0, float i1,
                                          float &o0, float &o1, float &o2) {
  if constexpr (EPI == Epi::kLinear) {
    o0 = act_f32<ACT>(a);
    if (has_in0) o0 += i0;
  } else if constexpr (EPI == Epi::kGated) {
    o0 = act_f32<ACT>(a) * b;
  } else {
    float value, slope;
    act_grad_f32<ACT>(i0, value, slope);
    o0 = a * i1 * slope;
    o1 = a * value;
    o2 = value * i1;
  }
}

// 2 N consecutive elements; packed inputs i0 and i1, packed results w0, w1, w2:
// kLinear D, Z; kGated H, G, U; kGatedBwd dG, dU, H.  Everything is fp32 until
// the one rounding of each packed result.
// kept: whether Z (G and U) are wanted at all.
template <Epi EPI, class T, int N>
__device__ __forceinline__ void epilogue_row(int act, bool has_in0, bool kept,
                                             const float (&a)[2 * N],
                                             const float (&b)[2 * N], const uint32_t (&i0)[N],
                                             const uint32_t (&i1)[N], uint32_t (&w0)[N],
                                             uint32_t (&w1)[N], uint32_t (&w2)[N]) {
  if (EPI != Epi::kGatedBwd && kept) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      w1[j] = pack2<T>(a[2 * j], a[2 * j + 1]);
      if constexpr (EPI == Epi::kGated) w2[j] = pack2<T>(b[2 * j], b[2 * j + 1]);
    }
  }
  with_act(act, [&](auto c) {
    constexpr int ACT = decltype(c)::value;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float2 x = make_float2(0.f, 0.f), y = x;
      float lo[3], hi[3];
      if (EPI == Epi::kGatedBwd || (EPI == Epi::kLinear && has_in0)) x = unpack2<T>(i0[j]);
      if constexpr (EPI == Epi::kGatedBwd) y = unpack2<T>(i1[j]);
      epilogue1<EPI, ACT>(has_in0, a[2 * j], b[2 * j], x.x, y.x, lo[0], lo[1], lo[2]);
      epilogue1<EPI, ACT>(has_in0, a[2 * j + 1], b[2 * j + 1], x.y, y.y, hi[0], hi[1], hi[2]);
      w0[j] = pack2<T>(lo[0], hi[0]);
      if constexpr (EPI == Epi::kGatedBwd) {
        w1[j] = pack2<T>(lo[1], hi[1]);
        w2[j] = pack2<T>(lo[2], hi[2]);
      }
    }
  });
}

}  // namespace dg
