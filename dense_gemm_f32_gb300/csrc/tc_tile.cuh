// tc_tile.cuh -- what the tensor-core kernels share: shared-memory operand
// descriptors, the tile raster, the watchdog, 3-D maps of MN-major operands.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tmap.cuh"

namespace dg {

// Bits of the kernels' `mn3d` argument: that MN-major operand is read through
// a 3-D tensor map, one TMA instruction per stage (else one per 128-byte
// column block; see make_map3).
constexpr int kA3d = 1, kB3d = 2;

// Shared-memory matrix descriptor of a swizzled operand tile: start address,
// leading / stride byte offsets (16-byte units), version 1, base offset 0
// (tiles are 1024-byte aligned), layout type at bits 61-63 (2 = 128-byte
// swizzle, 1 = 128-byte swizzle with 32-byte atoms).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo,
                                              uint32_t layout = 2u) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | ((uint64_t)layout << 61);
}

// Descriptor of the k-th MMA slice (UMMA_K elements of K) of an operand tile
// at saddr: K-major tiles advance 32 bytes inside the swizzle row; MN-major
// tiles advance UMMA_K / 8 groups of 8 K-rows.  box_bytes is the distance
// between the 128-byte MN blocks of an MN-major tile.
template <class G, bool kMN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, int k, uint32_t box_bytes) {
  if constexpr (kMN)
    return smem_desc(saddr + (uint32_t)(k * (G::UMMA_K / 8) * 1024), box_bytes, G::MN_SBO,
                     G::MN_LAYOUT);
  else  // K-major: 4 MMAs of 32 bytes of K per 128-byte box, boxes box_bytes apart
    return smem_desc(saddr + (uint32_t)((k >> 2) * box_bytes + (k & 3) * 32), 16, 1024);
}

// Tile id -> (tile row, tile col): tiles are walked in groups of `group_m`
// tile rows, column by column inside a group, so that the CTAs working at the
// same time share A row panels and B column panels in L2.
__device__ __forceinline__ void tile_coords(int tile, int tiles_m, int tiles_n, int group_m,
                                            int &tm, int &tn) {
  const int per_group = group_m * tiles_n;
  const int group = tile / per_group;
  const int first = group * group_m;
  const int gsize = min(tiles_m - first, group_m);
  const int r = tile - group * per_group;
  tm = first + r % gsize;
  tn = r / gsize;
}

__device__ __forceinline__ void watchdog_trip(int *watchdog, int site, volatile int *abort_flag) {
  atomicCAS(watchdog, 0, site);
  *abort_flag = 1;
}

// 3-D view of a row-major rows x cols matrix whose cols are a multiple of
// `blk`: (c, r, j) -> X[r][j * blk + c], so that one box of blk x box_rows x
// nblk lands in shared memory exactly as nblk 2-D boxes of blk x box_rows
// side by side.  One TMA instruction then loads what took nblk.
inline bool make_map3(CUtensorMap *map, const void *ptr, CUtensorMapDataType dt, int es, int64_t rows,
               int64_t cols, int64_t ld, int blk, int box_rows, int nblk, CUtensorMapSwizzle swz) {
  auto enc = get_encode();
  if (!enc || cols % blk != 0) return false;
  cuuint64_t dims[3] = {(cuuint64_t)blk, (cuuint64_t)rows, (cuuint64_t)(cols / blk)};
  cuuint64_t strides[2] = {(cuuint64_t)(ld * es), (cuuint64_t)(blk * es)};
  cuuint32_t box[3] = {(cuuint32_t)blk, (cuuint32_t)box_rows, (cuuint32_t)nblk};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, dt, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace dg
