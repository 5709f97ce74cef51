// int8.cuh -- what the two kernels of the 8-bit integer products share.
//
// The products run on the tensor cores in fp16: every 8-bit integer is an fp16
// number, so are all products of two in the fp32 accumulator, and a sum is exact
// while it stays within 2^24 (1024 products of the largest size, -128 by -128; 1040 of integers
// that are quantised here, which stop at 127; beyond that an
// addition is rounded to 24 bits, as in every fp32 sum).  GB300's integer tensor rate
// is a small part of its fp16 rate (an eighth or less), and two 4-bit halves in 8-bit floats would
// take four products at twice the rate.  Weights are read from memory in 8 bits
// and widened on the SM: a converter warp takes a row of 64 bytes from shared
// memory and writes 64 halves into its lane of tensor memory, from where the MMA
// reads them as its A operand.  Widened in shared memory instead they would be
// written and read there once more, 48 KB more per 128 x 64 weights and 256
// tokens, which shared memory does not have time for next to the MMA.
#pragma once

#include <cstdint>

#include "epilogue.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "tc_tile.cuh"

namespace dg {

// Four signed bytes as four halves: u = byte + 128 in the low bits of 1024 + u,
// less 1152.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x5140), b = __byte_perm(u, 0x64646464u, 0x5342);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// What a sum of integer products stands for: the feature's scale first, so that a
// row's scale at either end of fp32's range neither overflows nor vanishes before the
// result does; a sum of 0 in a row whose scale is not finite is NaN.
__device__ __forceinline__ float scaled(float sum, float row, float feature) { return sum * feature * row; }

// A whole warp's wait for a phase of a barrier.  False after `site` was recorded or
// another wait of the CTA had given up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int lane, int *watchdog, int site,
                                          volatile int *abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const bool ok = !*abort_flag && mbar_wait(bar, parity);
  if (!ok && lane == 0 && !*abort_flag) watchdog_trip(watchdog, site, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

// 64 bytes of weights from shared memory (16-byte pieces c ^ swizzle from `at`) as 64
// halves.
__device__ __forceinline__ void widen64(const uint8_t *at, int first, int swizzle, uint32_t (&r)[32]) {
  uint4 v[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4 *>(at + (((first + c) ^ swizzle) << 4));
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    widen4(v[c].x, r[8 * c], r[8 * c + 1]);
    widen4(v[c].y, r[8 * c + 2], r[8 * c + 3]);
    widen4(v[c].z, r[8 * c + 4], r[8 * c + 5]);
    widen4(v[c].w, r[8 * c + 6], r[8 * c + 7]);
  }
}

// True once every lane of the warp holds what widen64 loads: a vote over a value of each of
// the four loads.  A widened integer is no NaN, so the vote is always true, but the
// compiler cannot know that and what depends on it waits for the loads.
__device__ __forceinline__ bool warp_has(const uint32_t (&r)[32]) {
  return __all_sync(0xffffffffu, (r[0] & r[8] & r[16] & r[24]) != 0x7fff7fffu);
}

}  // namespace dg
