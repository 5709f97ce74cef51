// newton_pair.cu -- the products of a Newton-Schulz iteration on CTA pairs.
//
// The main loop is fused_pair.cu's: two CTAs accumulate 256 x 256 with
// tcgen05.mma.cta_group::2 from fp16 tiles that one producer thread per operand
// loads by TMA, two accumulators, eight epilogue warps.  What is different:
//  * Symmetric results.  X X^T and every product of polynomials in it are
//    symmetric, so only the tiles on and above the diagonal are computed, and a
//    warp writes each 32 x 32 piece above the diagonal twice: as it is, and
//    transposed through shared memory to the mirrored place.  4096^3 takes 136 tiles
//    for 256.  The results are symmetric to the last bit, which the steps of a group
//    need: what a rounding adds that is not grows from product to product
//    (2 x 3, five steps: 0.45 of the norm off with the diagonal tiles as they
//    come out of the sums, 0.004 mirrored).
//  * The epilogue: alpha f^power acc + beta in0 + gamma I in fp32, rounded once to
//    fp16, or for the last product to the type of the update.
//  * A second product with the same B in one launch (the next Gram matrix's and
//    the polynomials' products read the same polynomial).
//  * Operands of two terms (an fp32 X): the terms are further blocks of K of one sum.
// Bound by waves and by the ends of each product, not by the tensor pipe: 4096^3 symmetric takes 48
// to 51 us where its 136 tiles are 37 at cuBLAS's measured rate, as they are 1.8 waves of 76
// pairs (89%) and nothing covers the first loads and the last epilogue, the next product needing all
// of this one (tensor pipe 62 to 65% busy); with X, 256 tiles, 83 us (71; 72% busy).
// Every wait is bounded (ptx.cuh).
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "newton.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "tc_tile.cuh"
#include "tmap.cuh"

namespace dg {
namespace {

template <int LAYOUT>
struct Cfg {
  static constexpr bool kAT = LAYOUT == 2, kBT = LAYOUT == 1;
  static constexpr int BM = 256, BN = 256, HM = 128, HN = 128;  // pair tile, per-CTA halves
  static constexpr int BK = 64, UMMA_K = 16, KSTEPS = BK / UMMA_K;
  static constexpr int BOX = 64;  // elements in one 128-byte swizzle row
  static constexpr int A_BYTES = HM * 128, B_BYTES = HN * 128;
  static constexpr int A_BOXES = kAT ? HM / BOX : 1, B_BOXES = kBT ? 1 : HN / BOX;
  static constexpr int A_BOX_BYTES = kAT ? BK * 128 : A_BYTES;
  static constexpr int B_BOX_BYTES = kBT ? B_BYTES : BK * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES, MAX_STAGES = 6;
  static constexpr int TMEM_COLS = 512;
  static constexpr int kEpiWarps = 8, kProdBWarp = 2 + kEpiWarps;
  static constexpr int THREADS = 32 * (3 + kEpiWarps);
  // full, empty, accf[2], acce[2], drain, stall, two per epilogue warp
  static constexpr int NUM_BARS = 2 * MAX_STAGES + 6 + 2 * kEpiWarps;
  static constexpr int PIECE_BYTES = 32 * 64;      // 32 rows of 64 bytes
  static constexpr int EPI_BYTES = kEpiWarps * 2 * PIECE_BYTES;
  static constexpr int TAIL_BYTES = NUM_BARS * 8 + 16 + 1024;
  // in0's pieces, 4 KB for a warp, take a stage's place
  static constexpr int SMEM_BYTES = MAX_STAGES * STAGE_BYTES + EPI_BYTES + TAIL_BYTES;
  static_assert(SMEM_BYTES <= 232448 && kEpiWarps * 4096 <= STAGE_BYTES,
                "fits the 227 KB opt-in shared memory of a CTA");
  [[maybe_unused]] static constexpr uint32_t MN_LAYOUT = 2u, MN_SBO = 1024u;
  static constexpr uint32_t IDESC = (1u << 4) | ((kAT ? 1u : 0u) << 15) | ((kBT ? 0u : 1u) << 16) |
                                    ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
};

// Site codes of the bounded waits.
enum : int {
  kSite6ProducerEmpty = 0xe1,
  kSite6ProducerTail = 0xe2,
  kSite6MmaFull = 0xe3,
  kSite6MmaAccEmpty = 0xe4,
  kSite6MmaDrain = 0xe5,
  kSite6MmaTail = 0xe6,
  kSite6EpiAccFull = 0xe7,
  kSite6EpiInput = 0xe9,
  kSite6TestStall = 0xe8,  // DGEMM_TC_TEST_STALL: the MMA thread's test wait ran out
};

struct Maps {
  CUtensorMap a, a2, b, b2, o[2], in;  // a2: of A2, or of A_lo; b2: of B_lo
};

struct Args {
  int M, N, K;
  int mn3d, stall, products;
  int o_tma;  // outputs may be written by TMA
  int in_vec, in_tma;  // rows of in0 are aligned; it may be read by TMA
  int stages;
  int lo;  // B_lo (1), A_lo (2)
  float alpha, beta, gamma;
  const float *factor;
  int power;
  const void *in0;
  int64_t ldi0;
  void *out[2];
  int64_t ldo;
  int out_cols;
  int *watchdog;
};

constexpr int kGroup = 16;  // tile rows of a raster group

// Tiles on and above the diagonal of a t x t grid, in groups of kGroup tile rows,
// column by column inside a group (tile_coords' order without the mirrored ones).
__host__ __device__ __forceinline__ int upper_tiles(int t) { return t * (t + 1) / 2; }
__device__ __forceinline__ void upper_coords(int tile, int t, int &tm, int &tn) {
  int g0 = 0;
  for (;;) {
    const int rows = min(kGroup, t - g0), all = rows * (t - g0) - rows * (rows - 1) / 2;
    if (tile < all) {
      const int corner = rows * (rows + 1) / 2;  // columns g0 .. g0 + rows - 1 grow by one
      if (tile >= corner) {
        tm = g0 + (tile - corner) % rows;
        tn = g0 + rows + (tile - corner) / rows;
      } else {
        int c = 0;
        while (tile >= c + 1) tile -= ++c;
        tm = g0 + tile;
        tn = g0 + c;
      }
      return;
    }
    tile -= all;
    g0 += rows;
  }
}

template <class O>
constexpr int kPieceCols = 64 / (int)sizeof(O);

// 64 bytes of a row in registers from global memory; columns from `cols` on are zero.
template <class O>
__device__ __forceinline__ void load_piece(const O *row, int col, int cols, bool vec, uint32_t (&w)[16]) {
  if constexpr (sizeof(O) == 2) {
    load32<O>(row, col, cols, vec, w);
  } else {
    if (vec && col + 16 <= cols) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + col + 4 * q);
        w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = col + j < cols ? __float_as_uint(row[col + j]) : 0u;
    }
  }
}

// Row `lane` of a 32 x 64-byte piece that TMA loaded (64-byte swizzle).
__device__ __forceinline__ void take_piece(const uint8_t *piece, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 v = *reinterpret_cast<const uint4 *>(piece + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4));
    w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
  }
}

// A staged piece written element by element, a row per instruction: pieces that TMA may not write.
template <class O>
__device__ __noinline__ void store_piece(const uint8_t *piece, O *out, int64_t ld, int rows, int valid,
                                         int lane) {
  constexpr int C = kPieceCols<O>, PER = 32 / C;  // rows of an instruction
  const int c = lane % C;
  for (int r = lane / C; r < 32; r += PER) {
    const uint8_t *p = piece + r * 64 + ((((c * (int)sizeof(O)) >> 4) ^ ((r >> 1) & 3)) << 4) +
                       ((c * (int)sizeof(O)) & 15);
    if (r < rows && c < valid) out[r * ld + c] = *reinterpret_cast<const O *>(p);
  }
}

template <class O, int LAYOUT, bool SYM>
__global__ void __launch_bounds__(Cfg<LAYOUT>::THREADS, 1)
    newton_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  using G = Cfg<LAYOUT>;
  constexpr bool kAT = G::kAT, kBT = G::kBT;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_base);
  const uint32_t epi_base = base + G::MAX_STAGES * G::STAGE_BYTES;
  const uint32_t bars = epi_base + G::EPI_BYTES;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (G::MAX_STAGES + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * G::MAX_STAGES + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * G::MAX_STAGES + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * G::MAX_STAGES + 4);
  const uint32_t stall_bar = bars + 8u * (2 * G::MAX_STAGES + 5);  // nothing ever arrives here
  auto in_bar = [&](int i) { return bars + 8u * (2 * G::MAX_STAGES + 6 + i); };
  uint8_t *tail = smem + G::MAX_STAGES * G::STAGE_BYTES + G::EPI_BYTES + G::NUM_BARS * 8;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  auto a_tile = [&](int s) { return base + (uint32_t)(s * G::STAGE_BYTES); };
  auto b_tile = [&](int s) { return base + (uint32_t)(s * G::STAGE_BYTES + G::A_BYTES); };

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int tiles_m = (p.M + G::BM - 1) / G::BM, tiles_n = (p.N + G::BN - 1) / G::BN;
  const int tiles1 = SYM ? upper_tiles(tiles_m) : tiles_m * tiles_n;  // of one product
  const int num_tiles = SYM ? p.products * tiles1 : tiles1;
  const int kblocks1 = (p.K + G::BK - 1) / G::BK, kblocks = kblocks1 * terms_of(p.lo);
  auto coords = [&](int tile, int &tm, int &tn) {
    if constexpr (SYM)
      upper_coords(tile >= tiles1 ? tile - tiles1 : tile, tiles_m, tm, tn);
    else
      tile_coords(tile, tiles_m, tiles_n, kGroup, tm, tn);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 2);  // one arrival per producer thread
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * G::kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    mbar_init(stall_bar, 1);
    for (int i = 0; i < 2 * G::kEpiWarps; ++i) mbar_init(in_bar(i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t *>(tmem_slot)), G::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();  // the peer's barriers are initialised before any signal crosses
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // set-up done; the previous kernel on the stream has completed

  if (warp == 0 || warp == G::kProdBWarp) {
    // ----------------------------------------------------------- producers
    if (lane == 0) {
      const bool is_a = warp == 0;
      const uint32_t bytes = is_a ? (uint32_t)G::A_BYTES : (uint32_t)G::B_BYTES;
      const uint32_t fb0 = mapa_shared(full_bar(0), 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
        int tm, tn;
        coords(tile, tm, tn);
        const bool second = SYM && tile >= tiles1;
        const int m0 = tm * G::BM + (int)rank * G::HM, n0 = tn * G::BN + (int)rank * G::HN;
        for (int kq = 0; kq < kblocks; ++kq) {
          if (!mbar_try_wait(empty_bar(stage), phase ^ 1u) &&
              (*abort_flag || !mbar_wait(empty_bar(stage), phase ^ 1u))) {
            if (!*abort_flag) watchdog_trip(p.watchdog, kSite6ProducerEmpty, abort_flag);
            ok = false;
            break;
          }
          const uint32_t fb = fb0 + 8u * (uint32_t)stage;
          const TermBlock at = term_block(kq, kblocks1, p.lo);
          const CUtensorMap *map_a = second || at.a_lo ? &maps.a2 : &maps.a;
          const CUtensorMap *map_b = at.b_lo ? &maps.b2 : &maps.b;
          const int k0 = at.k * G::BK;
          if (is_a) {
            if (kAT && (p.mn3d & kA3d)) {
              tma_load_3d_pair(a_tile(stage), map_a, fb, 0, k0, m0 / G::BOX);
            } else {
#pragma unroll
              for (int j = 0; j < G::A_BOXES; ++j)
                tma_load_2d_pair(a_tile(stage) + j * G::A_BOX_BYTES, map_a, fb,
                                 kAT ? m0 + j * G::BOX : k0, kAT ? k0 : m0);
            }
          } else {
            if (!kBT && (p.mn3d & kB3d)) {
              tma_load_3d_pair(b_tile(stage), map_b, fb, 0, k0, n0 / G::BOX);
            } else {
#pragma unroll
              for (int j = 0; j < G::B_BOXES; ++j)
                tma_load_2d_pair(b_tile(stage) + j * G::B_BOX_BYTES, map_b, fb,
                                 kBT ? k0 : n0 + j * G::BOX, kBT ? n0 : k0);
            }
          }
          if (leader) mbar_arrive_expect_tx(full_bar(stage), 2u * bytes);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Tail: every stage-free signal aimed at this CTA has landed, and no
      // copy is still writing its shared memory.
      for (int i = 0; i < p.stages; ++i) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u)) {
          atomicCAS(p.watchdog, 0, kSite6ProducerTail);
          break;
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA (even CTA only)
    // The whole warp goes through the loop, so that one elected lane issues the MMAs
    // from uniform registers.
    if (leader) {
      auto wait = [&](uint32_t bar, uint32_t parity, int site) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool got = !*abort_flag && mbar_wait(bar, parity);
        if (!got && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, site, abort_flag);
        return __all_sync(0xffffffffu, got) != 0;
      };
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      if (p.stall && cluster == 0) {  // test hook: a wait that runs out
        wait(stall_bar, 0, kSite6TestStall);
        ok = false;
      }
      for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
        if (!wait(acce_bar(acc), acc_phase ^ 1u, kSite6MmaAccEmpty)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * G::BN);
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = wait(full_bar(stage), phase, kSite6MmaFull);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < G::KSTEPS; ++k)
              umma_f16_pair(d_tmem, operand_desc<G, kAT>(a_tile(stage), k, G::A_BOX_BYTES),
                            operand_desc<G, !kBT>(b_tile(stage), k, G::B_BOX_BYTES), G::IDESC,
                            (kb > 0 || k > 0) ? 1u : 0u);
            umma_commit_pair(empty_bar(stage), 0x3);  // frees the stage in both CTAs
          }
          __syncwarp();
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair(accf_bar(acc), 0x3);  // accumulator ready in both CTAs
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (elect_one()) umma_commit_pair(drain_bar, 0x1);
      __syncwarp();
      if (!mbar_wait(drain_bar, 0)) atomicCAS(p.watchdog, 0, kSite6MmaDrain);
      // Tail: both accumulators released by both epilogues.
      for (int i = 0; i < 2; ++i) {
        if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u)) {
          atomicCAS(p.watchdog, 0, kSite6MmaTail);
          break;
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int C = kPieceCols<O>;
    const int quarter = warp & 3;          // TMEM lanes this warp may access
    const int half = (warp - 2) >> 2;      // which of the two warps of the quarter
    const uint32_t slots = epi_base + (uint32_t)((warp - 2) * 2 * G::PIECE_BYTES);
    const uint32_t acce_leader0 = mapa_shared(acce_bar(0), 0);
    const uint32_t acce_leader1 = mapa_shared(acce_bar(1), 0);
    float alpha = p.alpha;
    if (p.factor != nullptr) {
      const float f = *p.factor;
      for (int i = 0; i < p.power; ++i) alpha *= f;
    }
    int stores = 0;  // pieces staged by this warp
    int acc = 0;
    uint32_t acc_phase = 0;
    // in0 comes by TMA where its rows are aligned, IN_AHEAD pieces of 32 x 32 ahead of
    // the epilogue.  (A row per thread read directly is 32 lines of memory for an
    // instruction.)  in_tile, in_c0: the next piece to send for, `sent` how many were.
    constexpr int IN_BYTES = 32 * 32 * (int)sizeof(O), IN_AHEAD = 4096 / IN_BYTES;
    const uint32_t in_buf = base + (uint32_t)(p.stages * G::STAGE_BYTES + (warp - 2) * 4096);
    int in_tile = cluster, in_c0 = 32 * half, sent = 0, taken = 0;
    auto send_for_input = [&] {
      while (in_tile < num_tiles && !(SYM && in_tile >= tiles1)) {
        int tm, tn;
        coords(in_tile, tm, tn);
        const int r0 = tm * G::BM + (int)rank * G::HM + quarter * 32;
        while (SYM && in_c0 < G::BN && tn * G::BN + in_c0 < r0) in_c0 += 64;  // below the diagonal
        const int col = tn * G::BN + in_c0;
        if (in_c0 >= G::BN || col >= p.N || r0 >= p.M) {
          in_tile += clusters, in_c0 = 32 * half;
          continue;
        }
        const int slot = sent % IN_AHEAD;
        const uint32_t bar = in_bar(2 * (warp - 2) + slot), to = in_buf + (uint32_t)(slot * IN_BYTES);
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, IN_BYTES);
          for (int h = 0; h < 32 / C; ++h)
            tma_load_2d(to + (uint32_t)(h * G::PIECE_BYTES), &maps.in, bar, col + h * C, r0);
        }
        ++sent;
        in_c0 += 64;
        return;
      }
    };
    if (p.in_tma)
      for (int i = 0; i < IN_AHEAD; ++i) send_for_input();
    // After the last tile's products the stages are idle: its pieces are staged there, each in
    // a place of its own, and none waits for a store.
    int idle = -1;
    // The next of this warp's two pieces, free to be written.
    auto next_piece = [&] {
      if (idle >= 0)
        return base + (uint32_t)((warp - 2) * (4 * (32 / C) * (SYM ? 2 : 1)) + idle++) * (uint32_t)G::PIECE_BYTES;
      if (lane == 0 && stores >= 2) bulk_wait_group_read<1>();  // the store two pieces ago
      __syncwarp();
      return slots + (uint32_t)((stores & 1) * G::PIECE_BYTES);
    };
    auto send_piece = [&](int o, uint32_t buf, int row0, int col) {
      if (idle >= 0) return;  // all together at the tile's end
      const int valid = min(C, p.out_cols - col);
      // TMA writes whole 16-byte granules: a piece that ends inside one goes
      // out element by element.
      const bool tma = p.o_tma && (valid == C || (p.out_cols * (int)sizeof(O)) % 16 == 0);
      if (tma) fence_proxy_async_smem();
      __syncwarp();
      if (tma) {
        if (lane == 0) tma_store_2d(&maps.o[o], buf, col, row0);
      } else {
        store_piece<O>(smem + (buf - base), static_cast<O *>(p.out[o]) + (int64_t)row0 * p.ldo + col, p.ldo,
                       p.M - row0, valid, lane);
      }
      if (lane == 0) bulk_commit_group();  // one (possibly empty) group per piece
      __syncwarp();
      ++stores;
    };
    for (int tile = cluster; tile < num_tiles; tile += clusters) {
      int tm, tn;
      coords(tile, tm, tn);
      const int o = SYM && tile >= tiles1 ? 1 : 0;
      const bool ok = !*abort_flag && mbar_wait(accf_bar(acc), acc_phase);
      if (!ok && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite6EpiAccFull, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (tile + clusters >= num_tiles) idle = 0;
      const int row0 = tm * G::BM + (int)rank * G::HM + quarter * 32;  // the warp's first row
      const int row = row0 + lane;
      const uint32_t t_row =
          tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * G::BN);
#pragma unroll 1
      for (int c0 = 32 * half; c0 < G::BN; c0 += 64) {
        const int col = tn * G::BN + c0;
        if (col >= p.N || row0 >= p.M) break;  // the same for the whole warp
        if (SYM && col < row0) continue;       // written from the piece above the diagonal
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_row + (uint32_t)c0, r);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = alpha * __uint_as_float(r[j]);
        if (p.in0 != nullptr && o == 0) {
          const int slot = taken % IN_AHEAD;
          if (p.in_tma) {
            const uint32_t bar = in_bar(2 * (warp - 2) + slot), phase = (uint32_t)(taken / IN_AHEAD) & 1u;
            bool got = __all_sync(0xffffffffu, mbar_try_wait(bar, phase));
            if (!got) {
              got = !*abort_flag && mbar_wait(bar, phase);
              if (!got && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite6EpiInput, abort_flag);
              // nothing more is sent for: the copies in flight are waited for at the end
              if (!__all_sync(0xffffffffu, got)) break;
            }
            ++taken;
          }
          const O *in = static_cast<const O *>(p.in0) + (int64_t)row * p.ldi0;
#pragma unroll
          for (int h = 0; h < 32 / C; ++h) {
            uint32_t w[16];
            if (p.in_tma)
              take_piece(smem + (in_buf - base) + slot * IN_BYTES + h * G::PIECE_BYTES, lane, w);
            else
              load_piece<O>(in, col + h * C, row < p.M ? p.N : 0, p.in_vec, w);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if constexpr (sizeof(O) == 2) {
                const float2 x = unpack2<O>(w[j]);
                v[2 * j] += p.beta * x.x, v[2 * j + 1] += p.beta * x.y;
              } else {
                v[h * C + j] += p.beta * __uint_as_float(w[j]);
              }
            }
          }
          if (p.in_tma) {
            fence_proxy_async_smem();  // the next copy comes after these reads
            __syncwarp();
            send_for_input();
          }
        }
        if (SYM && o == 0 && col == row0) add_diagonal(v, lane, p.gamma);
#pragma unroll
        for (int h = 0; h < 32 / C; ++h) {
          if (h > 0 && col + h * C >= p.N) break;
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if constexpr (sizeof(O) == 2)
              w[j] = pack2<O>(v[2 * j], v[2 * j + 1]);
            else
              w[j] = __float_as_uint(v[h * C + j]);
          }
          uint32_t buf = next_piece();
          if constexpr (SYM) {
            if (col == row0) {  // below the diagonal what is above it
              piece_store_turned(buf, lane, w);
              piece_mirror(buf, lane, w);
              __syncwarp();
            }
          }
          piece_store_row(buf, lane, w);
          send_piece(o, buf, row0, col + h * C);
          if constexpr (SYM) {
            if (col > row0) {  // the mirrored place
              buf = next_piece();
              piece_store_turned(buf, lane, w);
              send_piece(o, buf, col, row0);
            }
          }
        }
      }
      if (idle > 0) {
        // the last tile's pieces, in the order in which they were staged, after one fence
        const int last = idle;
        idle = -1;
        fence_proxy_async_smem();
        __syncwarp();
        uint32_t buf = base + (uint32_t)((warp - 2) * (4 * (32 / C) * (SYM ? 2 : 1))) * (uint32_t)G::PIECE_BYTES;
        int n = 0;
#pragma unroll 1
        for (int c0 = 32 * half; c0 < G::BN; c0 += 64) {
          const int col = tn * G::BN + c0;
          if (col >= p.N || row0 >= p.M) break;
          if (SYM && col < row0) continue;
#pragma unroll 1
          for (int h = 0; h < 32 / C && col + h * C < p.N && n < last; ++h) {
            send_piece(o, buf, row0, col + h * C);
            buf += G::PIECE_BYTES, ++n;
            if (SYM && col > row0) {
              send_piece(o, buf, col, row0);
              buf += G::PIECE_BYTES, ++n;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_tmem(acc ? acce_leader1 : acce_leader0);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) {
      bulk_wait_group<0>();  // every TMA store of this warp complete
      for (; taken < sent; ++taken)  // after an abort: its inputs have landed
        mbar_wait(in_bar(2 * (warp - 2) + taken % IN_AHEAD), (uint32_t)(taken / IN_AHEAD) & 1u);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, G::TMEM_COLS);
  }
}

// ------------------------------------------------------------- host side
template <class O>
constexpr CUtensorMapDataType map_type() {
  return sizeof(O) == 4                       ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : std::is_same<O, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <class O, int LAYOUT, bool SYM>
cudaError_t launch(const NewtonGemm &p, int *watchdog, cudaStream_t stream) {
  using G = Cfg<LAYOUT>;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  Args a;
  memset(&a, 0, sizeof a);
  const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  auto map_a = [&](CUtensorMap *map, const void *A) {
    if (!G::kAT) return make_map(map, A, dt, 2, p.M, p.K, p.lda, G::BOX, G::HM, swz);
    if (p.M % G::BOX == 0) {  // the same for A and A2
      a.mn3d |= kA3d;
      return make_map3(map, A, dt, 2, p.K, p.M, p.lda, G::BOX, G::BK, G::HM / G::BOX, swz);
    }
    return make_map(map, A, dt, 2, p.K, p.M, p.lda, G::BOX, G::BK, swz);
  };
  auto map_b = [&](CUtensorMap *map, const void *B) {
    if (G::kBT) return make_map(map, B, dt, 2, p.N, p.K, p.ldb, G::BOX, G::HN, swz);
    if (p.N % G::BOX == 0) {
      a.mn3d |= kB3d;
      return make_map3(map, B, dt, 2, p.K, p.N, p.ldb, G::BOX, G::BK, G::HN / G::BOX, swz);
    }
    return make_map(map, B, dt, 2, p.K, p.N, p.ldb, G::BOX, G::BK, swz);
  };
  bool ok = map_a(&maps.a, p.A) && map_b(&maps.b, p.B);
  if (p.A2 != nullptr) ok = ok && SYM && p.A_lo == nullptr && p.B_lo == nullptr && map_a(&maps.a2, p.A2);
  if (p.A_lo != nullptr) ok = ok && map_a(&maps.a2, p.A_lo);
  if (p.B_lo != nullptr) ok = ok && map_b(&maps.b2, p.B_lo);
  a.lo = (p.B_lo != nullptr ? 1 : 0) | (p.A_lo != nullptr ? 2 : 0);
  if (!ok || p.K < 1 || (SYM && p.M != p.N)) return cudaErrorInvalidValue;
  a.M = p.M, a.N = p.N, a.K = p.K;
  a.products = p.A2 != nullptr ? 2 : 1;
  a.stall = test_stall();
  a.alpha = p.alpha, a.beta = p.beta, a.gamma = p.gamma;
  a.factor = p.factor, a.power = p.power;
  a.in0 = p.in0, a.ldi0 = p.ldi0;
  a.in_vec = rows_aligned(p.in0, p.ldi0, sizeof(O));
  a.in_tma = p.in0 != nullptr && a.in_vec &&
             make_map(&maps.in, p.in0, map_type<O>(), sizeof(O), p.M, p.N, p.ldi0, kPieceCols<O>, 32,
                      CU_TENSOR_MAP_SWIZZLE_64B);
  a.stages = a.in_tma ? G::MAX_STAGES - 1 : G::MAX_STAGES;
  a.out[0] = p.out, a.out[1] = p.out2;
  a.ldo = p.ldo, a.out_cols = (int)p.out_cols;
  a.o_tma = rows_aligned(p.out, p.ldo, sizeof(O)) && rows_aligned(p.out2, p.ldo, sizeof(O));
  for (int i = 0; i < a.products && a.o_tma; ++i)
    a.o_tma = make_map(&maps.o[i], a.out[i], map_type<O>(), sizeof(O), p.M, p.out_cols, p.ldo,
                       kPieceCols<O>, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  a.watchdog = watchdog;
  auto kern = newton_pair_kernel<O, LAYOUT, SYM>;
  static std::atomic<int> max_clusters[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int maxc = max_clusters[dev].load(std::memory_order_acquire);
  if (maxc == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&maxc, (void *)kern, &cfg);
    if (e != cudaSuccess) return e;
    if (maxc < 1) return cudaErrorInvalidConfiguration;
    max_clusters[dev].store(maxc, std::memory_order_release);
  }
  const int64_t tm = (p.M + G::BM - 1) / G::BM, tn = (p.N + G::BN - 1) / G::BN;
  const int64_t tiles = SYM ? a.products * (tm * (tm + 1) / 2) : tm * tn;
  if (tm * tn > 0x3fffffff) return cudaErrorInvalidValue;
  const int clusters = (int)(tiles < maxc ? tiles : maxc);
  e = launch_kernel(kern, dim3(2 * clusters), dim3(G::THREADS), G::SMEM_BYTES, stream, 2u, maps, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class O>
cudaError_t launch_plain(const NewtonGemm &p, int *watchdog, cudaStream_t stream) {
  return p.layout == 0 ? launch<O, 0, false>(p, watchdog, stream)
                       : launch<O, 1, false>(p, watchdog, stream);
}

}  // namespace

cudaError_t launch_newton_pair(const NewtonGemm &p, int *watchdog, cudaStream_t stream) {
  if (p.symmetric) {
    if (p.dtype != DGEMM_DTYPE_F16 || p.layout == 0) return cudaErrorInvalidValue;
    return p.layout == 1 ? launch<__half, 1, true>(p, watchdog, stream)
                         : launch<__half, 2, true>(p, watchdog, stream);
  }
  if (p.layout == 2) return cudaErrorInvalidValue;
  switch (p.dtype) {
    case DGEMM_DTYPE_F32: return launch_plain<float>(p, watchdog, stream);
    case DGEMM_DTYPE_BF16: return launch_plain<__nv_bfloat16>(p, watchdog, stream);
    default: return launch_plain<__half>(p, watchdog, stream);
  }
}

}  // namespace dg
