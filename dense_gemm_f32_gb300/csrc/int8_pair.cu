// int8_pair.cu -- products with 8-bit weights on CTA pairs, for many tokens.
//
// A cluster of two CTAs accumulates D^T = W T^T, 256 features x NT tokens (up to
// 192), CTA r holding features [128 r, 128 r + 128) in its tensor memory: two
// accumulators of 192 columns, so that the epilogue of one tile overlaps the next
// tile's main loop, and behind them two places of 64 columns for weights of 128 k
// widened to fp16.  Tokens are halves already (quant.cu) and come by TMA, half of
// the tile's to each CTA.  The weights are the operand in tensor memory because
// they are the ones that are widened on the SM (int8.cuh), and 192 tokens because
// that is what two accumulators leave room for.
//  * Warp 0 loads weights (16 KB per 128 k), warp 2 tokens, warp 3 the scales of the
//    next tile, warps 4-11 widen half a row of weights per thread, one lane of warp 1 of
//    the even CTA issues tcgen05.mma.cta_group::2 with A in tensor memory, warps 12-19 run
//    the epilogue, with registers that the others hand over.
//  * The epilogue: a thread holds a feature's sums; a warp turns a 32 x 32 piece over
//    through its 4 KB of shared memory, after which a thread has eight neighbouring
//    features of a token: scales, bias, activation and residual in fp32, one
//    16-byte store.
//  * kGated: of a warp's 32 rows of weights 16 are features of Wg and 16 the same of
//    Wu, so both projections of a hidden unit meet in one piece; the hidden units go
//    out in fp32 (int8_small.cu says why).
//  * Weights are loaded before the kernel ahead on the stream is done, as in
//    int8_small.cu.
// Bound by the tensor pipe from about 140 tokens in a tile (0.0024 us per token and 128 k),
// below that by the hand-over from the loads through the converters to the MMA (0.3 us).
// 8192 x 4096 x 14336 takes 490 to 520 us (494 at cuBLAS's measured fp16 rate).  On the same
// box: four warps for the even blocks and four for the odd, whole rows each, 524 for 504;
// three or four places behind narrower accumulators 516 for 490; MMAs issued by a lane under
// `if (lane == 0)` 613 for 543, as their descriptors are put together by that lane one by one.
// Every wait is bounded (ptx.cuh).
#include <atomic>
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cuda_runtime.h>

#include "int8.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "rowvec.cuh"
#include "tc_tile.cuh"
#include "tmap.cuh"

namespace dg {
namespace {

struct Cfg {
  static constexpr int BM = 256, HM = 128, BK = 128, MAX_NT = 192;
  static constexpr int W_BYTES = HM * BK, W_STAGES = 4;
  static constexpr int T_MAX_STAGES = 8, T_MIN_STAGES = 2;  // at least as many as PLACES
  static constexpr int PLACES = 2, PLACE_COLS = BK / 2;
  static constexpr int ACC_COLS = MAX_NT, TMEM_COLS = 512;
  static_assert(2 * ACC_COLS + PLACES * PLACE_COLS <= TMEM_COLS, "tensor memory of an SM");
  // Warps in fours, which hand registers to each other: weights, MMA, tokens, scales;
  // converters; epilogue.  96 registers each at launch; the sum of what they go to is
  // no more.
  static constexpr int TOKEN_WARP = 2, SCALE_WARP = 3, CONV_WARP = 4, CONV_WARPS = 8, EPI_WARP = 12, EPI_WARPS = 8;
  static constexpr int THREADS = 32 * (EPI_WARP + EPI_WARPS);
  static constexpr int LAUNCH_REGS = 96, LOAD_REGS = 56, CONV_REGS = 80, EPI_REGS = 128;
  static_assert(THREADS * LAUNCH_REGS <= 65536 && 32 * (CONV_WARP * LOAD_REGS + CONV_WARPS * CONV_REGS +
                                                        EPI_WARPS * EPI_REGS) <= THREADS * LAUNCH_REGS,
                "registers of an SM");
  static constexpr int PIECE_BYTES = 32 * 32 * 4;
  static constexpr int EPI_BYTES = EPI_WARPS * PIECE_BYTES;
  // Scales of a tile, for the epilogue: its features' (or bias or second scales behind),
  // and its tokens'; two tiles'.
  static constexpr int SCALE_FLOATS = 2 * HM + MAX_NT;
  // wfull, wempty, ready, tempty, accf[2], acce[2], sfull[2], sempty[2], drain, stall
  static constexpr int NUM_BARS = 2 * W_STAGES + 2 * T_MAX_STAGES + 10;
  static constexpr int TAIL_BYTES = 2 * SCALE_FLOATS * 4 + NUM_BARS * 8 + 16 + 1024;
  static constexpr int FIXED_BYTES = W_STAGES * W_BYTES + EPI_BYTES + TAIL_BYTES;
  static constexpr int BUDGET = 232448 - FIXED_BYTES;
};

// Site codes of the bounded waits.
enum : int {
  kSite7WeightsEmpty = 0xf1,
  kSite7WeightsTail = 0xf2,
  kSite7TokensEmpty = 0xf3,
  kSite7TokensTail = 0xf4,
  kSite7ConvFull = 0xf5,
  kSite7ConvPlace = 0xf6,
  kSite7MmaAccEmpty = 0xf7,
  kSite7MmaReady = 0xf8,
  kSite7MmaDrain = 0xfa,
  kSite7MmaTail = 0xfb,
  kSite7EpiAccFull = 0xfc,
  kSite7EpiScales = 0xfe,
  kSite7ScalesEmpty = 0xff,
  kSite7TestStall = 0xfd,  // DGEMM_TC_TEST_STALL: the MMA thread's test wait ran out
};

struct Maps {
  CUtensorMap w, w2, t;
};

struct Args {
  int M, N, K;
  int act, nt, t_stages, group, stall, early;
  uint32_t idesc;
  const float *t_scale, *w_scale, *w2_scale;
  const void *in0, *bias;
  int64_t ldi0;
  void *out;
  int64_t ldo;
  int *watchdog;
};

// GATED: out is H in fp32, rows of whole vectors; else out and in0 are T.  AL:
// every row of out and in0 is 16-byte aligned.
template <class T, bool GATED, bool AL>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    int8_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  using G = Cfg;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_base);
  const uint32_t t_bytes = (uint32_t)p.nt * 128u;  // this CTA's half of the tokens, 128 k
  const uint32_t t_base = base + G::W_STAGES * G::W_BYTES;
  const uint32_t epi_base = t_base + (uint32_t)p.t_stages * t_bytes;
  const uint32_t bars = epi_base + G::EPI_BYTES + 2 * G::SCALE_FLOATS * 4;
  float *scales = reinterpret_cast<float *>(smem + (epi_base - base) + G::EPI_BYTES);
  auto wfull_bar = [&](int s) { return bars + 8u * s; };
  auto wempty_bar = [&](int s) { return bars + 8u * (G::W_STAGES + s); };
  auto ready_bar = [&](int s) { return bars + 8u * (2 * G::W_STAGES + s); };
  auto tempty_bar = [&](int s) { return bars + 8u * (2 * G::W_STAGES + G::T_MAX_STAGES + s); };
  const uint32_t more = bars + 8u * (2 * G::W_STAGES + 2 * G::T_MAX_STAGES);
  auto accf_bar = [&](int b) { return more + 8u * b; };
  auto acce_bar = [&](int b) { return more + 8u * (2 + b); };
  auto sfull_bar = [&](int b) { return more + 8u * (4 + b); };
  auto sempty_bar = [&](int b) { return more + 8u * (6 + b); };
  const uint32_t drain_bar = more + 8u * 8;
  const uint32_t stall_bar = more + 8u * 9;  // nothing ever arrives here
  uint8_t *tail = smem + (bars - base) + 8 * G::NUM_BARS;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  auto w_tile = [&](int s) { return base + (uint32_t)(s * G::W_BYTES); };
  auto t_tile = [&](int s) { return t_base + (uint32_t)s * t_bytes; };

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  constexpr int HF = GATED ? G::HM / 2 : G::HM;  // output features of a CTA's share of a tile
  const int tiles_f = (p.N + 2 * HF - 1) / (2 * HF), tiles_t = (p.M + p.nt - 1) / p.nt;
  const int num_tiles = tiles_f * tiles_t;
  const int kblocks = (p.K + G::BK - 1) / G::BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::W_STAGES; ++s) {
      mbar_init(wfull_bar(s), 1);
      mbar_init(wempty_bar(s), G::CONV_WARPS);
    }
    for (int s = 0; s < p.t_stages; ++s) {
      // both CTAs' tokens (one arrival and their bytes) and widened weights
      mbar_init(ready_bar(s), 1 + 2 * G::CONV_WARPS);
      mbar_init(tempty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * G::EPI_WARPS);
      mbar_init(sfull_bar(b), 1);
      mbar_init(sempty_bar(b), G::EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.t);
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
  const uint32_t place0 = tmem_base + 2u * G::ACC_COLS, place1 = place0 + G::PLACE_COLS;
  auto coords = [&](int tile, int &tf, int &tt) {
    tile_coords(tile, tiles_f, tiles_t, p.group, tf, tt);
  };

  if (warp < G::CONV_WARP) {
    setmaxnreg_dec<G::LOAD_REGS>();
    if (warp == 0) {
      // ------------------------------------------------------------- weights
      if (lane == 0) {
        if (!p.early) pdl_wait();
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
          int tf, tt;
          coords(tile, tf, tt);
          const int f0 = (2 * tf + (int)rank) * HF;
          for (int kb = 0; kb < kblocks; ++kb) {
            if (!mbar_try_wait(wempty_bar(s), phase ^ 1u) &&
                (*abort_flag || !mbar_wait(wempty_bar(s), phase ^ 1u))) {
              if (!*abort_flag) watchdog_trip(p.watchdog, kSite7WeightsEmpty, abort_flag);
              ok = false;
              break;
            }
            tma_load_2d(w_tile(s), &maps.w, wfull_bar(s), kb * G::BK, f0);
            if constexpr (GATED)
              tma_load_2d(w_tile(s) + G::W_BYTES / 2, &maps.w2, wfull_bar(s), kb * G::BK, f0);
            mbar_arrive_expect_tx(wfull_bar(s), G::W_BYTES);
            if (++s == G::W_STAGES) s = 0, phase ^= 1u;
          }
        }
        // Tail: no copy is still writing this CTA's shared memory.
        for (int i = 0; i < G::W_STAGES; ++i) {
          if (!mbar_wait(wempty_bar(s), phase ^ 1u)) {
            atomicCAS(p.watchdog, 0, kSite7WeightsTail);
            break;
          }
          if (++s == G::W_STAGES) s = 0, phase ^= 1u;
        }
      }
    } else if (warp == G::TOKEN_WARP) {
      // -------------------------------------------------------------- tokens
      if (lane == 0) {
        pdl_wait();
        const uint32_t fb0 = mapa_shared(ready_bar(0), 0);
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
          int tf, tt;
          coords(tile, tf, tt);
          const int t0 = tt * p.nt + (int)rank * (p.nt / 2);
          for (int kb = 0; kb < kblocks; ++kb) {
            if (!mbar_try_wait(tempty_bar(s), phase ^ 1u) &&
                (*abort_flag || !mbar_wait(tempty_bar(s), phase ^ 1u))) {
              if (!*abort_flag) watchdog_trip(p.watchdog, kSite7TokensEmpty, abort_flag);
              ok = false;
              break;
            }
            tma_load_2d_pair(t_tile(s), &maps.t, fb0 + 8u * (uint32_t)s, kb * G::BK, t0);
            tma_load_2d_pair(t_tile(s) + t_bytes / 2, &maps.t, fb0 + 8u * (uint32_t)s, kb * G::BK + 64, t0);
            if (leader) mbar_arrive_expect_tx(ready_bar(s), 2u * t_bytes);
            if (++s == p.t_stages) s = 0, phase ^= 1u;
          }
        }
        // Tail: every stage-free signal aimed at this CTA has landed, and no
        // copy is still writing its shared memory.
        for (int i = 0; i < p.t_stages; ++i) {
          if (!mbar_wait(tempty_bar(s), phase ^ 1u)) {
            atomicCAS(p.watchdog, 0, kSite7TokensTail);
            break;
          }
          if (++s == p.t_stages) s = 0, phase ^= 1u;
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------- MMA (even CTA only)
      // The whole warp goes through the loop, so that one elected lane issues the MMAs
      // from uniform registers.
      if (leader) {
        int s = 0;
        uint32_t phase = 0, place = place0;
        int acc = 0;
        uint32_t acc_phase = 0;
        // Descriptors of stage 0's tokens; stages and steps of k are added to their
        // address field (a thread's chain through computing them anew for every MMA is
        // as long as the MMA).
        const uint64_t desc0 = smem_desc(t_tile(0), 16u, 1024u);
        const uint32_t stage16 = t_bytes >> 4, box16 = t_bytes >> 5;
        uint64_t desc = desc0;
        bool ok = true;
        if (p.stall && cluster == 0) {  // test hook: a wait that runs out
          warp_wait(stall_bar, 0, lane, p.watchdog, kSite7TestStall, abort_flag);
          ok = false;
        }
        for (int tile = cluster; tile < num_tiles && ok; tile += clusters) {
          if (!warp_wait(acce_bar(acc), acc_phase ^ 1u, lane, p.watchdog, kSite7MmaAccEmpty, abort_flag)) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * G::ACC_COLS);
          for (int kb = 0; kb < kblocks; ++kb) {
            ok = warp_wait(ready_bar(s), phase, lane, p.watchdog, kSite7MmaReady, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < G::BK / 16; ++k)
                umma_f16_ta_pair(d_tmem, place + 8u * k, desc + (k >> 2) * box16 + 2u * (k & 3), p.idesc,
                                 k > 0 ? 1u : kb > 0 ? 1u : 0u);
              umma_commit_pair(tempty_bar(s), 0x3);  // frees the tokens and the place in both CTAs
            }
            __syncwarp();
            place ^= place0 ^ place1;
            desc += stage16;
            if (++s == p.t_stages) s = 0, phase ^= 1u, desc = desc0;
          }
          if (!ok) break;
          if (elect_one()) umma_commit_pair(accf_bar(acc), 0x3);  // accumulator ready in both CTAs
          __syncwarp();
          if (++acc == 2) acc = 0, acc_phase ^= 1u;
        }
        // by the lane that issued the MMAs (elect_one names the same one every time)
        if (elect_one()) umma_commit_pair(drain_bar, 0x1);
        __syncwarp();
        if (!mbar_wait(drain_bar, 0)) atomicCAS(p.watchdog, 0, kSite7MmaDrain);
        // Tail: both accumulators released by both epilogues.
        for (int i = 0; i < 2; ++i) {
          if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u)) {
            atomicCAS(p.watchdog, 0, kSite7MmaTail);
            break;
          }
          if (++acc == 2) acc = 0, acc_phase ^= 1u;
        }
      }
    }
    if (warp == G::SCALE_WARP) {
      // ------------------------------------------------------------ scales
      pdl_wait();
      int b = 0;
      uint32_t phase = 0;
      for (int tile = cluster; tile < num_tiles; tile += clusters) {
        int tf, tt;
        coords(tile, tf, tt);
        if (!warp_wait(sempty_bar(b), phase ^ 1u, lane, p.watchdog, kSite7ScalesEmpty, abort_flag)) break;
        float *to = scales + b * G::SCALE_FLOATS;
        const int f0 = (2 * tf + (int)rank) * HF, t0 = tt * p.nt;
        for (int i = lane; i < HF; i += 32) {
          const bool in = f0 + i < p.N;
          to[i] = in ? p.w_scale[f0 + i] : 0.f;
          float more = 0.f;  // the other projection's scale, or the bias
          if (GATED)
            more = in ? p.w2_scale[f0 + i] : 0.f;
          else if (p.bias != nullptr)
            more = in ? to_f32<T>(static_cast<const T *>(p.bias)[f0 + i]) : 0.f;
          to[G::HM + i] = more;
        }
        for (int i = lane; i < p.nt; i += 32) to[2 * G::HM + i] = t0 + i < p.M ? p.t_scale[t0 + i] : 0.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull_bar(b));
        if (++b == 2) b = 0, phase ^= 1u;
      }
    }
  } else if (warp < G::EPI_WARP) {
    setmaxnreg_dec<G::CONV_REGS>();
    // --------------------------------------------------- widen the weights
    // four warps for each half of a stage's k
    const int quarter = warp & 3, half_k = (warp - G::CONV_WARP) >> 2;
    // gated: of a quarter's 32 lanes 16 features of Wg, then the same of Wu
    const int row = !GATED ? quarter * 32 + lane
                           : (lane < 16 ? quarter * 16 + lane : G::HM / 2 + quarter * 16 + lane - 16);
    const uint32_t lanes = ((uint32_t)(quarter * 32) << 16) + (uint32_t)(32 * half_k);
    const uint32_t ready_leader = mapa_shared(ready_bar(0), 0);
    const int64_t tiles = cluster < num_tiles ? (num_tiles - 1 - cluster) / clusters + 1 : 0;
    const int64_t blocks = tiles * kblocks;
    int s = 0, t = 0, free_t = 0;  // stages of weights and tokens; the tokens of PLACES blocks ago
    uint32_t phase = 0, free_phase = 0, place = place0;
    for (int64_t i = 0; i < blocks; ++i) {
      if (!warp_wait(wfull_bar(s), phase, lane, p.watchdog, kSite7ConvFull, abort_flag)) break;
      const uint8_t *w = smem + (w_tile(s) - base) + row * G::BK;
      uint32_t r[32];
      widen64(w, 4 * half_k, row & 7, r);
      // The stage is given back once the values are here: an arrival that is only issued
      // after the loads can be seen before they have read, and the next copy then lands
      // under them.
      const bool here = warp_has(r);
      if (lane == 0 && here) mbar_arrive(wempty_bar(s));
      if (++s == G::W_STAGES) s = 0, phase ^= 1u;
      if (i >= G::PLACES) {  // the MMAs that read this place PLACES blocks ago are done
        if (!warp_wait(tempty_bar(free_t), free_phase, lane, p.watchdog, kSite7ConvPlace, abort_flag)) break;
        if (++free_t == p.t_stages) free_t = 0, free_phase ^= 1u;
        tc_fence_after();
      }
      tmem_st_32x32b_x32(place + lanes, r);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_tmem(ready_leader + 8u * (uint32_t)t);
      if (++t == p.t_stages) t = 0;
      place ^= place0 ^ place1;
    }
  } else {
    setmaxnreg_inc<G::EPI_REGS>();
    // ------------------------------------------------------------ epilogue
    pdl_wait();
    const int quarter = warp & 3;
    float *piece = reinterpret_cast<float *>(smem + (epi_base - base) + (warp - G::EPI_WARP) * G::PIECE_BYTES);
    const uint32_t acce_leader0 = mapa_shared(acce_bar(0), 0);
    const uint32_t acce_leader1 = mapa_shared(acce_bar(1), 0);
    constexpr int Q = GATED ? 2 : 4;            // threads per token, eight features each
    constexpr int ROUNDS = Q, STEP = 32 / Q;    // a thread's tokens of a piece: STEP apart
    const int chunk = lane % Q, token = lane / Q;
    int acc = 0;
    uint32_t acc_phase = 0;
    const int half = (warp - G::EPI_WARP) >> 2;  // which of the two warps of the quarter
    const bool has_in0 = !GATED && p.in0 != nullptr;
    for (int tile = cluster; tile < num_tiles; tile += clusters) {
      int tf, tt;
      coords(tile, tf, tt);
      const int t0 = tt * p.nt, live = min(p.nt, p.M - t0);
      const int f = quarter * (HF / 4) + 8 * chunk, col = (2 * tf + (int)rank) * HF + f;
      if (!warp_wait(sfull_bar(acc), acc_phase, lane, p.watchdog, kSite7EpiScales, abort_flag)) break;
      const float *sc = scales + acc * G::SCALE_FLOATS;
      float ws[8], more[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = *reinterpret_cast<const float4 *>(sc + f + 4 * h);
        const float4 y = *reinterpret_cast<const float4 *>(sc + G::HM + f + 4 * h);
        ws[4 * h] = x.x, ws[4 * h + 1] = x.y, ws[4 * h + 2] = x.z, ws[4 * h + 3] = x.w;
        more[4 * h] = y.x, more[4 * h + 1] = y.y, more[4 * h + 2] = y.z, more[4 * h + 3] = y.w;
      }
      if (!warp_wait(accf_bar(acc), acc_phase, lane, p.watchdog, kSite7EpiAccFull, abort_flag)) break;
      tc_fence_after();
      const uint32_t t_row =
          tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * G::ACC_COLS);
#pragma unroll 1
      for (int c0 = 32 * half; c0 < live; c0 += 64) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_row + (uint32_t)c0, r);
        const T *res_row = static_cast<const T *>(p.in0) + (int64_t)(t0 + c0 + token) * p.ldi0;
        RowBlocks res[GATED ? 1 : ROUNDS];
        if (has_in0) {
#pragma unroll
          for (int i = 0; i < ROUNDS; ++i)
            res[GATED ? 0 : i] = fetch_row16<T, AL>(res_row + i * STEP * p.ldi0, col,
                                                    c0 + token + i * STEP < live ? p.N : 0);
        }
        tmem_wait_ld();
        __syncwarp();  // the piece before has been read
#pragma unroll
        for (int j = 0; j < 32; ++j) piece[j * 32 + lane] = __uint_as_float(r[j]);
        __syncwarp();
        const float *ts = sc + 2 * G::HM + c0 + token;
        const int left = col < p.N ? live - c0 - token : 0;  // of this thread's tokens, STEP apart
        char *out = static_cast<char *>(p.out) +
                    ((int64_t)(t0 + c0 + token) * p.ldo + col) * (GATED ? 4 : (int)sizeof(T));
        const int64_t step_bytes = (int64_t)STEP * p.ldo * (GATED ? 4 : (int)sizeof(T));
        // halves in an order that keeps the eight lanes of a phase on different banks
        const int first = (lane / Q) & 1;
        auto take = [&](int tp, int at, float (&v)[8]) {
          const float4 x = *reinterpret_cast<const float4 *>(piece + tp * 32 + at + 4 * first);
          const float4 y = *reinterpret_cast<const float4 *>(piece + tp * 32 + at + 4 * (first ^ 1));
          v[0] = first ? y.x : x.x, v[1] = first ? y.y : x.y, v[2] = first ? y.z : x.z, v[3] = first ? y.w : x.w;
          v[4] = first ? x.x : y.x, v[5] = first ? x.y : y.y, v[6] = first ? x.z : y.z, v[7] = first ? x.w : y.w;
        };
        with_act(p.act, [&](auto c) {
          constexpr int ACT = decltype(c)::value;
#pragma unroll
          for (int i = 0; i < ROUNDS; ++i) {
            float a[8];
            take(token + i * STEP, 8 * chunk, a);
            const float row_scale = ts[i * STEP];
            if constexpr (GATED) {
              float b[8];
              take(token + i * STEP, 16 + 8 * chunk, b);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                a[j] = act_f32<ACT>(scaled(a[j], row_scale, ws[j])) * scaled(b[j], row_scale, more[j]);
              if (i * STEP < left) {
                float4 *h = reinterpret_cast<float4 *>(out + i * step_bytes);
                h[0] = make_float4(a[0], a[1], a[2], a[3]);
                h[1] = make_float4(a[4], a[5], a[6], a[7]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) a[j] = act_f32<ACT>(scaled(a[j], row_scale, ws[j]) + more[j]);
              if (has_in0) {
                float x[8];
                widen16<T>(take_row16<T, AL>(res[GATED ? 0 : i], res_row + i * STEP * p.ldi0, col, p.N), x);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += x[j];
              }
              const uint4 v[1] = {narrow16<T>(a)};
              if constexpr (AL) {
                if (i * STEP < left) *reinterpret_cast<uint4 *>(out + i * step_bytes) = v[0];
              } else {
                store_row16<T, AL, 1, Q>(static_cast<T *>(p.out) + (int64_t)(t0 + c0 + token + i * STEP) * p.ldo,
                                         i * STEP < left ? col : p.N, p.N, v);
              }
            }
          }
        });
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sempty_bar(acc));
        mbar_arrive_cluster_tmem(acc ? acce_leader1 : acce_leader0);
      }
      if (++acc == 2) acc = 0, acc_phase ^= 1u;
    }
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
template <class T, bool GATED, bool AL>
cudaError_t launch(const Int8Gemm &p, int nt, int *watchdog, cudaStream_t stream) {
  using G = Cfg;
  constexpr int hf = GATED ? G::HM / 2 : G::HM;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  Args a;
  memset(&a, 0, sizeof a);
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  if (p.K < 1 || nt < 32 || nt > G::MAX_NT || nt % 32 != 0 ||
      !make_map(&maps.w, p.W, u8, 1, p.N, p.K, p.ldw, G::BK, hf, swz) ||
      (GATED && !make_map(&maps.w2, p.W2, u8, 1, p.N, p.K, p.ldw2, G::BK, hf, swz)) ||
      !make_map(&maps.t, p.T, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p.M, p.K, p.ldt, 64, nt / 2, swz))
    return cudaErrorInvalidValue;
  a.M = p.M, a.N = p.N, a.K = p.K;
  a.act = p.act, a.nt = nt;
  a.early = p.early;
  a.t_stages = G::BUDGET / (nt * 128);
  if (a.t_stages > G::T_MAX_STAGES) a.t_stages = G::T_MAX_STAGES;
  static_assert(G::BUDGET / (G::MAX_NT * 128) >= G::T_MIN_STAGES, "a place is free when its tokens are");
  a.group = 16;
  a.stall = test_stall();
  a.idesc = (1u << 4) | ((uint32_t)(nt >> 3) << 17) | ((uint32_t)(G::BM >> 4) << 24);
  a.t_scale = p.t_scale, a.w_scale = p.w_scale, a.w2_scale = p.w2_scale;
  a.in0 = p.in0, a.ldi0 = p.ldi0, a.bias = p.bias;
  a.out = p.out, a.ldo = p.ldo;
  a.watchdog = watchdog;
  const int smem = G::FIXED_BYTES + a.t_stages * nt * 128;
  auto kern = int8_pair_kernel<T, GATED, AL>;
  static std::atomic<int> max_clusters[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int maxc = max_clusters[dev].load(std::memory_order_acquire);
  if (maxc == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = 232448;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&maxc, (void *)kern, &cfg);
    if (e != cudaSuccess) return e;
    if (maxc < 1) return cudaErrorInvalidConfiguration;
    max_clusters[dev].store(maxc, std::memory_order_release);
  }
  const int64_t tiles = (int64_t)((p.N + 2 * hf - 1) / (2 * hf)) * ((p.M + nt - 1) / nt);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const int clusters = (int)(tiles < maxc ? tiles : maxc);
  e = launch_kernel(kern, dim3(2 * clusters), dim3(G::THREADS), (size_t)smem, stream, 2u, maps, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class T>
cudaError_t launch_linear(const Int8Gemm &p, int nt, int *watchdog, cudaStream_t stream) {
  const bool vec = p.N % 8 == 0 && rows_aligned(p.in0, p.in0 ? p.ldi0 : 0) && rows_aligned(p.out, p.ldo);
  return vec ? launch<T, false, true>(p, nt, watchdog, stream)
             : launch<T, false, false>(p, nt, watchdog, stream);
}

}  // namespace

cudaError_t launch_int8_pair(const Int8Gemm &p, int nt, int *watchdog, cudaStream_t stream) {
  if (p.gated) return launch<__half, true, true>(p, nt, watchdog, stream);  // H is fp32
  return p.dtype == DGEMM_DTYPE_BF16 ? launch_linear<__nv_bfloat16>(p, nt, watchdog, stream)
                                     : launch_linear<__half>(p, nt, watchdog, stream);
}

}  // namespace dg
