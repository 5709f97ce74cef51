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
  // `off` is the same in every lane that shares a row: branches, not selects
  uint32_t r0, r1, r2, r3, r4;
  switch (off >> 2) {
    case 0: r0 = a.x, r1 = a.y, r2 = a.z, r3 = a.w, r4 = b.x; break;
    case 1: r0 = a.y, r1 = a.z, r2 = a.w, r3 = b.x, r4 = b.y; break;
    case 2: r0 = a.z, r1 = a.w, r2 = b.x, r3 = b.y, r4 = b.z; break;
    default: r0 = a.w, r1 = b.x, r2 = b.y, r3 = b.z, r4 = b.w; break;
  }
  if constexpr (sizeof(T) == 4) {
    return make_uint4(r0, r1, r2, r3);
  } else {
    const int sh = 8 * (off & 3);
    return make_uint4(__funnelshift_r(r0, r1, sh), __funnelshift_r(r1, r2, sh),
                      __funnelshift_r(r2, r3, sh), __funnelshift_r(r3, r4, sh));
  }
}

// The vector of `row` at `col`; elements from `cols` on are zero.
template <class T, bool ALIGNED>
__device__ __forceinline__ uint4 load_row16(const T *row, int col, int cols) {
  constexpr int V = kVec<T>;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (col >= cols) return v;
  if constexpr (ALIGNED) {
    return *reinterpret_cast<const uint4 *>(row + col);
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + col);
    const int off = (int)(at & 15);
    const uint4 *block = reinterpret_cast<const uint4 *>(at - off);
    v = block[0];
    uint4 next = make_uint4(0u, 0u, 0u, 0u);
    if (off != 0 && col + V - off / (int)sizeof(T) < cols) next = block[1];
    v = shift16<T>(v, next, off);
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

// Store v at `col` of `row`.  The whole warp calls it; each group of LANES
// lanes holds neighbouring vectors of one row, lane i of the group that of
// column col0 + i * V (lanes past `cols` store nothing).
template <class T, bool ALIGNED, int LANES = 32>
__device__ __forceinline__ void store_row16(T *row, int col, int cols, uint4 v) {
  constexpr int V = kVec<T>;
  if constexpr (ALIGNED) {
    if (col < cols) *reinterpret_cast<uint4 *>(row + col) = v;
  } else {
    const int lane = threadIdx.x & (LANES - 1);
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + col);
    const int off = (int)(at & 15);  // the same in every lane of the group
    uint4 prev;
    prev.x = __shfl_up_sync(0xffffffffu, v.x, 1);
    prev.y = __shfl_up_sync(0xffffffffu, v.y, 1);
    prev.z = __shfl_up_sync(0xffffffffu, v.z, 1);
    prev.w = __shfl_up_sync(0xffffffffu, v.w, 1);
    const int head = V - off / (int)sizeof(T);  // own elements in the block at `at - off`
    auto whole = [&](int c) { return c + head <= cols; };  // a lane at column c stores its block
    const bool block = (off == 0 || lane > 0) && whole(col);
    if (block)
      *reinterpret_cast<uint4 *>(at - off) = off == 0 ? v : shift16<T>(prev, v, 16 - off);
    // elements that no lane's block holds
    const bool tail = off != 0 && (lane == LANES - 1 || !whole(col + V));
    if ((!block || tail) && col < cols) {
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (col + j < cols && (j < head ? !block : tail)) {
          if constexpr (sizeof(T) == 4)
            reinterpret_cast<uint32_t *>(row + col)[j] = w[j];
          else
            reinterpret_cast<uint16_t *>(row + col)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
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
