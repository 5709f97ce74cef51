// rowvec.cuh -- 16 bytes' worth of a row at a time, whatever the row's
// alignment.
//
// A vector is V = 16 / sizeof(T) elements starting at a column that is a
// multiple of V.  On aligned rows it is one 16-byte access.  On other rows
// (ALIGNED = false) the two 16-byte blocks it lies in are loaded and the
// elements shifted out of them, and a warp whose lanes hold neighbouring
// vectors stores whole aligned blocks put together from two lanes, so every
// access but those at the ends still moves 16 bytes.  A block is touched only
// if it holds an element of the row, so no access leaves the row's own 16-byte
// blocks, and only elements of the row are written.
#pragma once

#include <cstdint>

#include "activation.cuh"

namespace dg {

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// Bytes off .. off + 15 of the 32 bytes a then b; off is a multiple of
// sizeof(T), below 16.
template <class T>
__device__ __forceinline__ uint4 shift16(uint4 a, uint4 b, int off) {
  // two selects per word and a funnel shift; `off` belongs to the row, so what
  // depends on it alone is computed once per row
  const bool two = (off & 8) != 0, one = (off & 4) != 0;
  const uint32_t b0 = two ? a.z : a.x, b1 = two ? a.w : a.y, b2 = two ? b.x : a.z;
  const uint32_t b3 = two ? b.y : a.w, b4 = two ? b.z : b.x, b5 = two ? b.w : b.y;
  const uint32_t r0 = one ? b1 : b0, r1 = one ? b2 : b1, r2 = one ? b3 : b2, r3 = one ? b4 : b3;
  if constexpr (sizeof(T) == 4) {
    return make_uint4(r0, r1, r2, r3);
  } else {
    const uint32_t r4 = one ? b5 : b4;
    const int sh = 8 * (off & 3);
    return make_uint4(__funnelshift_r(r0, r1, sh), __funnelshift_r(r1, r2, sh),
                      __funnelshift_r(r2, r3, sh), __funnelshift_r(r3, r4, sh));
  }
}

// A vector as loaded: the one or two blocks it lies in.  fetch_row16 of several
// vectors before take_row16 of the first keeps all their loads in flight.
struct RowBlocks {
  uint4 a, b;
};
template <class T, bool ALIGNED>
__device__ __forceinline__ RowBlocks fetch_row16(const T *row, int col, int cols) {
  constexpr int V = kVec<T>;
  RowBlocks r;
  r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
  const int off = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(row) & 15);  // col: whole vectors
  const uint4 *block = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(row) - off +
                                                       (int64_t)col * (int)sizeof(T));
  if (col < cols) r.a = block[0];
  if constexpr (!ALIGNED) {
    if (off != 0 && col + V - off / (int)sizeof(T) < cols) r.b = block[1];
  }
  return r;
}

// The elements of a fetched vector; those from `cols` on are zero.
template <class T, bool ALIGNED>
__device__ __forceinline__ uint4 take_row16(const RowBlocks &r, const T *row, int col, int cols) {
  constexpr int V = kVec<T>;
  if constexpr (ALIGNED) {
    return r.a;
  } else {
    uint4 v = shift16<T>(r.a, r.b, (int)(reinterpret_cast<uintptr_t>(row) & 15));
    const int valid = cols - col;  // the row's last vector may be short
    if (valid < V) {
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4)
          w[j] = j < valid ? w[j] : 0u;
        else
          w[j] = 2 * j + 1 < valid ? w[j] : 2 * j < valid ? w[j] & 0xFFFFu : 0u;
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
}

// The vector of `row` at `col`; elements from `cols` on are zero.
template <class T, bool ALIGNED>
__device__ __forceinline__ uint4 load_row16(const T *row, int col, int cols) {
  return take_row16<T, ALIGNED>(fetch_row16<T, ALIGNED>(row, col, cols), row, col, cols);
}

// Store N vectors of `row`, vector k at column col + k * LANES * V.  The whole
// warp calls it; each group of LANES lanes shares a row, lane i of the group
// holding column col0 + i * V (vectors past `cols` are not stored), so the
// group's N * LANES vectors are neighbours and only its first and last element
// blocks are put together from single elements.
template <class T, bool ALIGNED, int N = 1, int LANES = 32>
__device__ __forceinline__ void store_row16(T *row, int col, int cols, const uint4 (&v)[N]) {
  constexpr int V = kVec<T>;
  if constexpr (ALIGNED) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (col + k * LANES * V < cols) *reinterpret_cast<uint4 *>(row + col + k * LANES * V) = v[k];
  } else {
    const int lane = threadIdx.x & (LANES - 1);
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15);  // col is whole vectors
    const int head = V - off / (int)sizeof(T);  // elements of a vector in the block it begins in
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = col + k * LANES * V;
      uint8_t *dst = reinterpret_cast<uint8_t *>(row) - off + (int64_t)c * (int)sizeof(T);
      // the vector before: the lane before's, and for the first lane the last
      // lane's of the round before
      const uint4 send = k > 0 && lane == LANES - 1 ? v[k > 0 ? k - 1 : 0] : v[k];
      const int from = (threadIdx.x & 31 & ~(LANES - 1)) | ((lane + LANES - 1) & (LANES - 1));
      uint4 prev;
      prev.x = __shfl_sync(0xffffffffu, send.x, from);
      prev.y = __shfl_sync(0xffffffffu, send.y, from);
      prev.z = __shfl_sync(0xffffffffu, send.z, from);
      prev.w = __shfl_sync(0xffffffffu, send.w, from);
      auto whole = [&](int x) { return x + head <= cols; };  // column x's lane stores its block
      const bool block = (off == 0 || lane > 0 || k > 0) && whole(c);
      if (block) *reinterpret_cast<uint4 *>(dst) = off == 0 ? v[k] : shift16<T>(prev, v[k], 16 - off);
      // elements that no block holds
      const bool tail = off != 0 && ((lane == LANES - 1 && k == N - 1) || !whole(c + V));
      if ((!block || tail) && c < cols) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (c + j < cols && (j < head ? !block : tail)) {
            if constexpr (sizeof(T) == 4)
              reinterpret_cast<uint32_t *>(row + c)[j] = w[j];
            else
              reinterpret_cast<uint16_t *>(row + c)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
          }
        }
      }
    }
  }
}

// Widened elements of a vector, and back (rounded to nearest even).
template <class T>
__device__ __forceinline__ void widen16(uint4 v, float *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) {
      f[j] = __uint_as_float(w[j]);
    } else {
      const float2 t = unpack2<T>(w[j]);
      f[2 * j] = t.x, f[2 * j + 1] = t.y;
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 narrow16(const float *f) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  else
    return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                      pack2<T>(f[6], f[7]));
}

}  // namespace dg
