// fused_pair.cu -- the fused products of the feed-forward operators on CTA
// pairs (tcgen05.mma.cta_group::2), for outputs of many 256 x 256 tiles and
// K > 0.
//
// The main loop is that of tc.cu's pair kernel: a cluster of two CTAs
// accumulates 256 x 256 in the two SMs' tensor memory, CTA r holding rows
// [128 r, 128 r + 128) of the accumulator and loading half of each operand
// tile by TMA (5 or 6 stages of 32 KB, one producer thread per operand), two
// accumulators so that the epilogue of one tile overlaps the next tile's
// main loop.  What is different:
//  * A second operand pair.  kSum walks the k-blocks of A B, then those of
//    A2 B2, into one accumulator (dX = dG Wg^T + dU Wu^T without an
//    intermediate); kPair walks the tiles of two products in one launch
//    (dWg, dWu); kGated loads the even CTA's half of the B tile from Wg and
//    the odd CTA's from Wu, so that columns [0, 128) of the accumulator are g
//    and [128, 256) the u of the same 128 hidden units, and one MMA stream
//    gives each thread of the epilogue both projections of its row.
//  * The epilogue (epilogue.cuh): eight warps, two per quarter of the TMEM
//    lanes taking alternate 32-column pieces.  A thread holds 32 columns of
//    one row; it reads the residual of that row segment from global memory (g
//    and u have come by TMA while the piece before was finished), computes in
//    fp32, and packs 16-bit results into a 64-byte-swizzled 32 x 32 piece of
//    shared memory that goes out as one TMA store per output (pieces that TMA
//    may not write go out element by element).  Each warp owns two 2 KB pieces
//    and runs on its own, with no barrier among the epilogue warps.
// Bound by the tensor pipe under the power limit: 16384 x 14336 x 4096 bf16
// with bias, gelu_tanh and both outputs 1.20 ms, 1607 TFLOP/s, where a cuBLAS
// product of 8192^3 without an epilogue sustains 1708.  With little K (1024 and less) the
// epilogue bounds it: a warp's chain through one piece takes about 900 cycles.
// Every wait is bounded (ptx.cuh).
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "tc_tile.cuh"
#include "tmap.cuh"

// Compiled once per operand layout (DGEMM_FUSED_UNIT): 0: A M x K, B K x N;
// 1: A M x K, B N x K; 2: A K x M, B K x N.
#ifndef DGEMM_FUSED_UNIT
#define DGEMM_FUSED_UNIT 0
#endif
#define DG_CAT2(a, b) a##b
#define DG_CAT(a, b) DG_CAT2(a, b)
#define DG_UNIT_LAUNCHER DG_CAT(launch_fused_pair_unit_, DGEMM_FUSED_UNIT)

namespace dg {
namespace {

constexpr bool kAT = DGEMM_FUSED_UNIT == 2, kBT = DGEMM_FUSED_UNIT == 1;

template <class T, Epi EPI>
struct PairCfg {
  static constexpr int BM = 256, BN = 256, HM = 128, HN = 128;  // pair tile, per-CTA halves
  static constexpr int ES = 2, BK = 64, UMMA_K = 16, KSTEPS = BK / UMMA_K;
  static constexpr int BOX = 64;  // elements in one 128-byte swizzle row
  static constexpr int A_BYTES = HM * 128, B_BYTES = HN * 128;
  static constexpr int A_BOXES = kAT ? HM / BOX : 1, B_BOXES = kBT ? 1 : HN / BOX;
  static constexpr int A_BOX_BYTES = kAT ? BK * 128 : A_BYTES;
  static constexpr int B_BOX_BYTES = kBT ? B_BYTES : BK * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // Inputs of the epilogue that come by TMA, in one stage's place: G and U
  // (4096 x 1024 x 8192: 101 us with 16-byte loads of a row per thread, 87).  A
  // residual is read by the threads: the sixth stage is worth more (8192 x 4096
  // x 14336: 565 us with six, 579 with five and the residual by TMA).
  static constexpr int INS = EPI == Epi::kGatedBwd ? 2 : 0;
  static constexpr int STAGES = INS ? 5 : 6;
  static constexpr int TMEM_COLS = 512;
  static constexpr int kEpiWarps = 8, kProdBWarp = 2 + kEpiWarps;
  static constexpr int THREADS = 32 * (3 + kEpiWarps);
  // full, empty, accf[2], acce[2], drain, stall, one per epilogue warp
  static constexpr int NUM_BARS = 2 * STAGES + 6 + kEpiWarps;
  static constexpr int PIECE_BYTES = 32 * 64;      // 32 rows x 32 columns of 2 bytes
  static constexpr int OUT_BYTES = kEpiWarps * 2 * PIECE_BYTES;
  static constexpr int EPI_BYTES = OUT_BYTES + kEpiWarps * INS * PIECE_BYTES;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + NUM_BARS * 8 + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "fits the 227 KB opt-in shared memory of a CTA");
  static constexpr uint32_t MN_LAYOUT = 2u, MN_SBO = 1024u;
  static constexpr uint32_t kFmt = std::is_same<T, __half>::value ? 0u : 1u;
  static constexpr uint32_t IDESC = (1u << 4) | (kFmt << 7) | (kFmt << 10) |
                                    ((kAT ? 1u : 0u) << 15) | ((kBT ? 0u : 1u) << 16) |
                                    ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
};

// Site codes of the bounded waits.
enum : int {
  kSite3ProducerEmpty = 0xa1,
  kSite3ProducerTail = 0xa2,
  kSite3MmaFull = 0xa3,
  kSite3MmaAccEmpty = 0xa4,
  kSite3MmaDrain = 0xa5,
  kSite3MmaTail = 0xa6,
  kSite3EpiAccFull = 0xa7,
  kSite3EpiInput = 0xa9,
  kSite3TestStall = 0xa8,  // DGEMM_TC_TEST_STALL: the MMA thread's test wait ran out
};

struct PairMaps {
  CUtensorMap a, b, a2, b2;  // operands
  CUtensorMap o[3];          // outputs, 32 x 32 boxes
  CUtensorMap i[2];          // the epilogue's inputs, likewise
};

struct PairArgs {
  int M, N, K;
  int dual, act, group_m, mn3d, stall;
  int o_tma;       // bit i: output i may be written by TMA
  int i_vec;       // bit i: rows of input i are 16-byte aligned; bit 2: the bias is
  const void *in0, *in1, *bias;
  int64_t ldi0, ldi1;
  void *out[3];
  int64_t ldo[3];
  int *watchdog;
};

// Row `lane` of a 32 x 32 piece that TMA loaded (64-byte swizzle).
__device__ __forceinline__ void take_piece(const uint8_t *piece, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 v =
        *reinterpret_cast<const uint4 *>(piece + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4));
    w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
  }
}

// A staged 32 x 32 piece written element by element, a row per instruction:
// pieces that TMA may not write.  Not inlined, to keep the epilogue's loop
// short (it runs from the instruction cache: with it inlined, 2048 x 4096 x 512
// silu with bias and residual took 21.1 us, now 19.7).
__device__ __noinline__ void store_piece(const uint16_t *wb, uint16_t *out, int64_t ld, int rows,
                                         int valid, int lane) {
  out += lane;
  const uint16_t *col = wb + (lane & 7);
  const int q = lane >> 3;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 16) {
    uint16_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i] = col[(r0 + i) * 32 + ((q ^ (((r0 + i) >> 1) & 3)) << 3)];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (r0 + i < rows && lane < valid) *out = v[i];
      out += ld;
    }
  }
}

template <class T, Epi EPI>
__global__ void __launch_bounds__(PairCfg<T, EPI>::THREADS, 1)
    fused_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairArgs p) {
  using G = PairCfg<T, EPI>;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_base);
  const uint32_t epi_base = base + G::STAGES * G::STAGE_BYTES;
  const uint32_t bars = epi_base + G::EPI_BYTES;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (G::STAGES + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * G::STAGES + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * G::STAGES + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * G::STAGES + 4);
  const uint32_t stall_bar = bars + 8u * (2 * G::STAGES + 5);  // nothing ever arrives here
  auto in_bar = [&](int w) { return bars + 8u * (2 * G::STAGES + 6 + w); };
  uint8_t *tail = smem + G::STAGES * G::STAGE_BYTES + G::EPI_BYTES + G::NUM_BARS * 8;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  auto a_tile = [&](int s) { return base + (uint32_t)(s * G::STAGE_BYTES); };
  auto b_tile = [&](int s) { return base + (uint32_t)(s * G::STAGE_BYTES + G::A_BYTES); };

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  constexpr int TN = EPI == Epi::kGated ? G::HN : G::BN;  // output columns of a tile
  const int tiles_m = (p.M + G::BM - 1) / G::BM, tiles_n = (p.N + TN - 1) / TN;
  const int tiles1 = tiles_m * tiles_n;  // tiles of one product
  const bool pair_out = EPI == Epi::kLinear && p.dual == (int)Dual::kPair;
  const bool sum = EPI == Epi::kLinear && p.dual == (int)Dual::kSum;
  const int num_tiles = pair_out ? 2 * tiles1 : tiles1;
  const int kb1 = (p.K + G::BK - 1) / G::BK;  // k-blocks of one product
  const int kblocks = sum ? 2 * kb1 : kb1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(full_bar(s), 2);  // one arrival per producer thread
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * G::kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    mbar_init(stall_bar, 1);
    for (int w = 0; w < G::kEpiWarps; ++w) mbar_init(in_bar(w), 1);
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
        const bool second = tile >= tiles1;  // kPair: a tile of A2 B2
        tile_coords(second ? tile - tiles1 : tile, tiles_m, tiles_n, p.group_m, tm, tn);
        const int m0 = tm * G::BM + (int)rank * G::HM;
        const int n0 = EPI == Epi::kGated ? tn * TN : tn * TN + (int)rank * G::HN;
        for (int kq = 0; kq < kblocks; ++kq) {
          if (!mbar_try_wait(empty_bar(stage), phase ^ 1u) &&
              (*abort_flag || !mbar_wait(empty_bar(stage), phase ^ 1u))) {
            if (!*abort_flag) watchdog_trip(p.watchdog, kSite3ProducerEmpty, abort_flag);
            ok = false;
            break;
          }
          const uint32_t fb = fb0 + 8u * (uint32_t)stage;
          const bool set2 = second || kq >= kb1;
          const int k0 = (kq >= kb1 ? kq - kb1 : kq) * G::BK;
          if (is_a) {
            const CUtensorMap *map = set2 ? &maps.a2 : &maps.a;
            if (kAT && (p.mn3d & kA3d)) {
              tma_load_3d_pair(a_tile(stage), map, fb, 0, k0, m0 / G::BOX);
            } else {
#pragma unroll
              for (int j = 0; j < G::A_BOXES; ++j)
                tma_load_2d_pair(a_tile(stage) + j * G::A_BOX_BYTES, map, fb,
                                 kAT ? m0 + j * G::BOX : k0, kAT ? k0 : m0);
            }
          } else {
            const bool b2 = EPI == Epi::kGated ? rank == 1 : set2;
            const CUtensorMap *map = b2 ? &maps.b2 : &maps.b;
            if (!kBT && (p.mn3d & kB3d)) {
              tma_load_3d_pair(b_tile(stage), map, fb, 0, k0, n0 / G::BOX);
            } else {
#pragma unroll
              for (int j = 0; j < G::B_BOXES; ++j)
                tma_load_2d_pair(b_tile(stage) + j * G::B_BOX_BYTES, map, fb,
                                 kBT ? k0 : n0 + j * G::BOX, kBT ? n0 : k0);
            }
          }
          if (leader) mbar_arrive_expect_tx(full_bar(stage), 2u * bytes);
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Tail: every stage-free signal aimed at this CTA has landed, and no
      // copy is still writing its shared memory.
      for (int i = 0; i < G::STAGES; ++i) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u)) {
          atomicCAS(p.watchdog, 0, kSite3ProducerTail);
          break;
        }
        if (++stage == G::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA (even CTA only)
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      if (p.stall && cluster == 0) {  // test hook: a wait that runs out
        if (!mbar_wait(stall_bar, 0)) watchdog_trip(p.watchdog, kSite3TestStall, abort_flag);
        ok = false;
      }
      for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
        if (*abort_flag || !mbar_wait(acce_bar(acc), acc_phase ^ 1u)) {
          if (!*abort_flag) watchdog_trip(p.watchdog, kSite3MmaAccEmpty, abort_flag);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * G::BN);
        for (int kb = 0; kb < kblocks; ++kb) {
          const bool got = mbar_try_wait(full_bar(stage), phase) ||
                           (!*abort_flag && mbar_wait(full_bar(stage), phase));
          if (!got) {
            if (!*abort_flag) watchdog_trip(p.watchdog, kSite3MmaFull, abort_flag);
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < G::KSTEPS; ++k)
            umma_f16_pair(d_tmem, operand_desc<G, kAT>(a_tile(stage), k, G::A_BOX_BYTES),
                          operand_desc<G, !kBT>(b_tile(stage), k, G::B_BOX_BYTES), G::IDESC,
                          (kb > 0 || k > 0) ? 1u : 0u);
          umma_commit_pair(empty_bar(stage), 0x3);  // frees the stage in both CTAs
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(accf_bar(acc), 0x3);  // accumulator ready in both CTAs
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      umma_commit_pair(drain_bar, 0x1);
      if (!mbar_wait(drain_bar, 0)) atomicCAS(p.watchdog, 0, kSite3MmaDrain);
      // Tail: both accumulators released by both epilogues.
      for (int i = 0; i < 2; ++i) {
        if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u)) {
          atomicCAS(p.watchdog, 0, kSite3MmaTail);
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
    const int quarter = warp & 3;          // TMEM lanes this warp may access
    const int half = (warp - 2) >> 2;      // which of the two warps of the quarter
    const uint32_t slots = epi_base + (uint32_t)((warp - 2) * 2 * G::PIECE_BYTES);
    const uint32_t acce_leader0 = mapa_shared(acce_bar(0), 0);
    const uint32_t acce_leader1 = mapa_shared(acce_bar(1), 0);
    const bool kept = !pair_out && p.out[1] != nullptr;
    int stores = 0;  // pieces staged by this warp
    // G and U come by TMA where their rows are aligned, a piece ahead: the first
    // from (tile, c0) on that has elements inside the output.
    const bool in_tma = G::INS > 0 && (p.i_vec & 3) == 3;
    const uint32_t in_buf =
        epi_base + (uint32_t)(G::OUT_BYTES + (warp - 2) * G::INS * G::PIECE_BYTES);
    const uint32_t my_bar = in_bar(warp - 2);
    uint32_t in_phase = 0;
    bool in_flight = false;
    auto send_for_inputs = [&](int tile, int c0) {
      for (; tile < num_tiles; tile += clusters, c0 = 32 * half) {
        int tm, tn;
        tile_coords(tile, tiles_m, tiles_n, p.group_m, tm, tn);
        const int r0 = tm * G::BM + (int)rank * G::HM + quarter * 32, col = tn * TN + c0;
        if (c0 >= TN || col >= p.N || r0 >= p.M) continue;
        if (lane == 0) {
          mbar_arrive_expect_tx(my_bar, (uint32_t)(G::INS * G::PIECE_BYTES));
          for (int i = 0; i < G::INS; ++i)
            tma_load_2d(in_buf + (uint32_t)(i * G::PIECE_BYTES), &maps.i[i], my_bar, col, r0);
        }
        in_flight = true;
        return;
      }
      in_flight = false;
    };
    if (in_tma) send_for_inputs(cluster, 32 * half);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = cluster; tile < num_tiles; tile += clusters) {
      int tm, tn;
      const bool second = tile >= tiles1;
      tile_coords(second ? tile - tiles1 : tile, tiles_m, tiles_n, p.group_m, tm, tn);
      const bool ok = !*abort_flag && mbar_wait(accf_bar(acc), acc_phase);
      if (!ok && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite3EpiAccFull, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int row0 = tm * G::BM + (int)rank * G::HM + quarter * 32;  // the warp's first row
      const int row = row0 + lane;
      const uint32_t t_row =
          tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * G::BN);
#pragma unroll 1
      for (int c0 = 32 * half; c0 < TN; c0 += 64) {
        const int col = tn * TN + c0;
        const int valid = min(32, p.N - col);  // columns of the piece inside the output
        if (valid <= 0 || row0 >= p.M) break;  // the same for the whole warp
        uint32_t i0[16], i1[16];
        const bool has_in0 = EPI == Epi::kGatedBwd || (EPI == Epi::kLinear && p.in0 != nullptr);
        if (G::INS > 0 && in_tma) {
          const bool got = !*abort_flag && mbar_wait(my_bar, in_phase);
          if (!got && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite3EpiInput, abort_flag);
          // nothing more is sent for: the copy in flight is waited for at the end
          if (!__all_sync(0xffffffffu, got)) break;
          in_phase ^= 1u;
          take_piece(smem + (in_buf - base), lane, i0);
          take_piece(smem + (in_buf - base) + G::PIECE_BYTES, lane, i1);
          __syncwarp();
          send_for_inputs(tile, c0 + 64);
        } else if (has_in0) {
          load32<T>(static_cast<const T *>(p.in0) + (int64_t)row * p.ldi0, col,
                    row < p.M ? p.N : 0, p.i_vec & 1, i0);
          if constexpr (EPI == Epi::kGatedBwd)
            load32<T>(static_cast<const T *>(p.in1) + (int64_t)row * p.ldi1, col,
                      row < p.M ? p.N : 0, p.i_vec & 2, i1);
        }
        float a[32], b[32];
        {
          uint32_t r[32], q[32];
          tmem_ld_32x32b_x32(t_row + (uint32_t)c0, r);
          if constexpr (EPI == Epi::kGated) tmem_ld_32x32b_x32(t_row + (uint32_t)(G::HN + c0), q);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            a[j] = __uint_as_float(r[j]);
            if constexpr (EPI == Epi::kGated) b[j] = __uint_as_float(q[j]);
          }
        }
        if (EPI == Epi::kLinear && p.bias != nullptr) {
          uint32_t w[16];
          load32<T>(static_cast<const T *>(p.bias), col, p.N, p.i_vec & 4, w);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 v = unpack2<T>(w[j]);
            a[2 * j] += v.x, a[2 * j + 1] += v.y;
          }
        }
        uint32_t w[3][16];
        epilogue_row<EPI, T, 16>(p.act, has_in0, kept, a, b, i0, i1, w[0], w[1], w[2]);
        constexpr int kOuts = EPI == Epi::kLinear ? 2 : 3;
#pragma unroll
        for (int o = 0; o < kOuts; ++o) {
          // kLinear: out[0] is D and out[1] is Z, or (kPair) the products in turn
          int slot_out = o;
          if constexpr (EPI == Epi::kLinear) {
            if (pair_out) {
              if (o) continue;
              slot_out = second ? 1 : 0;
            }
          }
          if (p.out[slot_out] == nullptr) continue;
          const uint32_t buf = slots + (uint32_t)((stores & 1) * G::PIECE_BYTES);
          if (lane == 0 && stores >= 2) bulk_wait_group_read<1>();  // the store two pieces ago
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             buf + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4))),
                         "r"(w[o][4 * q]), "r"(w[o][4 * q + 1]), "r"(w[o][4 * q + 2]),
                         "r"(w[o][4 * q + 3])
                         : "memory");
          // TMA writes whole 16-byte granules: a piece that ends inside one
          // goes out element by element.
          const bool tma = ((p.o_tma >> slot_out) & 1) && (valid == 32 || (p.N & 7) == 0);
          if (tma) fence_proxy_async_smem();
          __syncwarp();
          if (tma) {
            if (lane == 0) tma_store_2d(&maps.o[slot_out], buf, col, row0);
          } else {
            store_piece(reinterpret_cast<const uint16_t *>(smem + (buf - base)),
                        static_cast<uint16_t *>(p.out[slot_out]) +
                            (int64_t)row0 * p.ldo[slot_out] + col,
                        p.ldo[slot_out], p.M - row0, valid, lane);
          }
          if (lane == 0) bulk_commit_group();  // one (possibly empty) group per piece
          __syncwarp();
          ++stores;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc ? acce_leader1 : acce_leader0);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) {
      bulk_wait_group<0>();  // every TMA store of this warp complete
      if (in_flight) mbar_wait(my_bar, in_phase);  // after an abort: its input has landed
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
template <class T>
constexpr CUtensorMapDataType map_type() {
  return std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Maps of one operand pair; mn3d gets which of them are 3-D.
template <class T, Epi EPI>
bool pair_operand_maps(CUtensorMap *ta, CUtensorMap *tb, const FusedGemm &p, const void *A,
                       int64_t lda, const void *B, int64_t ldb, int *mn3d) {
  using G = PairCfg<T, EPI>;
  const CUtensorMapDataType dt = map_type<T>();
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  *mn3d = 0;
  bool ok_a, ok_b;
  if (kAT && make_map3(ta, A, dt, G::ES, p.K, p.M, lda, G::BOX, G::BK, G::HM / G::BOX, swz)) {
    *mn3d |= kA3d;
    ok_a = true;
  } else {
    ok_a = kAT ? make_map(ta, A, dt, G::ES, p.K, p.M, lda, G::BOX, G::BK, swz)
               : make_map(ta, A, dt, G::ES, p.M, p.K, lda, G::BOX, G::HM, swz);
  }
  if (!kBT && make_map3(tb, B, dt, G::ES, p.K, p.N, ldb, G::BOX, G::BK, G::HN / G::BOX, swz)) {
    *mn3d |= kB3d;
    ok_b = true;
  } else {
    ok_b = kBT ? make_map(tb, B, dt, G::ES, p.N, p.K, ldb, G::BOX, G::HN, swz)
               : make_map(tb, B, dt, G::ES, p.K, p.N, ldb, G::BOX, G::BK, swz);
  }
  return ok_a && ok_b;
}

template <class T, Epi EPI>
cudaError_t launch_pair(const FusedGemm &p, int *watchdog, cudaStream_t stream) {
  using G = PairCfg<T, EPI>;
  PairMaps maps;
  memset(&maps, 0, sizeof maps);
  PairArgs a;
  memset(&a, 0, sizeof a);
  if (!pair_operand_maps<T, EPI>(&maps.a, &maps.b, p, p.A, p.lda, p.B, p.ldb, &a.mn3d))
    return cudaErrorInvalidValue;
  if (p.dual != Dual::kNone) {
    int mn3d2 = 0;
    const bool gated = p.dual == Dual::kGated;
    if (!pair_operand_maps<T, EPI>(&maps.a2, &maps.b2, p, gated ? p.A : p.A2, gated ? p.lda : p.lda2,
                              p.B2, p.ldb2, &mn3d2) ||
        mn3d2 != a.mn3d)
      return cudaErrorInvalidValue;
  }
  a.M = p.M, a.N = p.N, a.K = p.K;
  a.dual = (int)p.dual, a.act = p.act;
  a.group_m = 16;
  a.stall = test_stall();
  a.in0 = p.in0, a.in1 = p.in1, a.bias = p.bias;
  a.ldi0 = p.ldi0, a.ldi1 = p.ldi1;
  a.i_vec = (rows_aligned(p.in0, p.ldi0) ? 1 : 0) | (rows_aligned(p.in1, p.ldi1) ? 2 : 0) |
            (rows_aligned(p.bias, 0) ? 4 : 0);
  void *outs[3] = {p.out0, p.out1, p.out2};
  const int64_t lds[3] = {p.ldo0, p.ldo1, p.ldo2};
  for (int i = 0; i < 3; ++i) {
    a.out[i] = outs[i];
    a.ldo[i] = lds[i];
    if (outs[i] != nullptr && rows_aligned(outs[i], lds[i]) &&
        make_map(&maps.o[i], outs[i], map_type<T>(), G::ES, p.M, p.N, lds[i], 32, 32,
                 CU_TENSOR_MAP_SWIZZLE_64B))
      a.o_tma |= 1 << i;
  }
  const void *ins[2] = {p.in0, p.in1};
  const int64_t ldi[2] = {p.ldi0, p.ldi1};
  for (int i = 0; i < 2; ++i)
    if (i < G::INS && ((a.i_vec >> i) & 1) &&
        !make_map(&maps.i[i], ins[i], map_type<T>(), G::ES, p.M, p.N, ldi[i], 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  a.watchdog = watchdog;
  auto kern = fused_pair_kernel<T, EPI>;
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
  const int tile_n = EPI == Epi::kGated ? G::HN : G::BN;
  const int64_t tiles = (int64_t)((p.M + G::BM - 1) / G::BM) * ((p.N + tile_n - 1) / tile_n) *
                        (p.dual == Dual::kPair ? 2 : 1);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const int clusters = (int)(tiles < maxc ? tiles : maxc);
  e = launch_kernel(kern, dim3(2 * clusters), dim3(G::THREADS), G::SMEM_BYTES, stream, 2u, maps, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class T>
cudaError_t launch_epi(const FusedGemm &p, int *watchdog, cudaStream_t stream) {
  if (p.epi == Epi::kLinear) return launch_pair<T, Epi::kLinear>(p, watchdog, stream);
  if constexpr (!kAT) {  // the gated epilogues' A is activations, M x K
    if (p.epi == Epi::kGated) return launch_pair<T, Epi::kGated>(p, watchdog, stream);
    return launch_pair<T, Epi::kGatedBwd>(p, watchdog, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t DG_UNIT_LAUNCHER(const FusedGemm &p, int *watchdog, cudaStream_t stream) {
  return p.dtype == DGEMM_DTYPE_BF16 ? launch_epi<__nv_bfloat16>(p, watchdog, stream)
                                     : launch_epi<__half>(p, watchdog, stream);
}

}  // namespace dg
