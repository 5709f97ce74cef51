// newton.cuh -- 32 x 32 pieces of 16-bit results that a warp turns over in shared
// memory, for the symmetric products of newton_pair.cu and newton_small.cu.
//
// A piece is 32 rows of 64 bytes, 16-byte part q of row r at q ^ (r >> 1 & 3), as
// TMA's 64-byte swizzle has it.  Lane i holds row i in 16 packed words.
#pragma once

#include <cstdint>

namespace dg {

// Blocks of K in the order in which a product with operands of two terms goes through them:
// A B, then A B_lo (bit 0 of `lo`), then A_lo B (bit 1), `one` blocks each.
struct TermBlock {
  int k;              // block of K
  bool a_lo, b_lo;    // of A_lo, B_lo
};
__host__ __device__ __forceinline__ int terms_of(int lo) { return 1 + (lo & 1) + (lo >> 1); }
__device__ __forceinline__ TermBlock term_block(int kq, int one, int lo) {
  const int all = one * terms_of(lo), k = kq >= 2 * one ? kq - 2 * one : kq >= one ? kq - one : kq;
  return {k, (lo & 2) && kq >= all - one, (lo & 1) && kq >= one && kq < 2 * one};
}

// gamma on the diagonal of a piece.  As a choice of what is added: a choice of where to
// is compiled into a branch for every lane, 1400 cycles.
__device__ __forceinline__ void add_diagonal(float (&v)[32], int lane, float gamma) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float x;
    asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, %2;\n\tselp.f32 %0, %3, 0f00000000, p;\n\t}"
        : "=f"(x)
        : "r"(lane), "r"(j), "f"(gamma));
    v[j] += x;
  }
}

// Row `lane` of the piece at shared address `piece`.
__device__ __forceinline__ void piece_store_row(uint32_t piece, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                     piece + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4))),
                 "r"(w[4 * q]), "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
}

// The rows as columns.  Two neighbouring lanes exchange a word, so that each has two
// neighbours of a column and the warp writes two rows of the turned piece at once
// (element by element the 32 columns took 1100 cycles).
__device__ __forceinline__ void piece_store_turned(uint32_t piece, int lane, const uint32_t (&w)[16]) {
  const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
  const uint32_t at = piece + (uint32_t)((lane & 1) * 64 + ((lane >> 1) & 3) * 4);
#pragma unroll
  for (int j = 0; j < 16; ++j) {  // rows 2 j and 2 j + 1
    const uint32_t y = __byte_perm(w[j], __shfl_xor_sync(0xffffffffu, w[j], 1), pick);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (uint32_t)(j * 128 + (((lane >> 3) ^ (j & 3)) << 4))),
                 "r"(y)
                 : "memory");
  }
}

// On the diagonal: what is below it in the warp's rows becomes what is above it
// turned over, read from the piece that piece_store_turned wrote.
__device__ __forceinline__ void piece_mirror(uint32_t turned, int lane, uint32_t (&w)[16]) {
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t t[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(t[0]), "=r"(t[1]), "=r"(t[2]), "=r"(t[3])
                 : "r"(turned + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)))
                 : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = 8 * q + 2 * k;  // columns c and c + 1 of row `lane`
      uint32_t &x = w[4 * q + k];
      x = c >= lane ? x : c + 1 < lane ? t[k] : __byte_perm(t[k], x, 0x7610);
    }
  }
}

}  // namespace dg
