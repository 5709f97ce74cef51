// fused_small.cu -- the fused products of the feed-forward operators for few
// rows or few tiles: single tokens, serving batches, small layers.
//
// Such a product is bound by reading its weights once, so the roles of the
// operands are swapped with respect to a large product: the weights' output
// features are the 128 rows of the MMA and the tokens its columns (16 to 256,
// a multiple of 16), D^T = op(W)^T X^T, and one token costs little more than
// the weights' traffic.  A tile is 128 features x NT tokens; with few tiles its
// K range is split over a thread-block cluster of up to 8 CTAs, so that enough
// SMs pull weights at once.
//  * Warp 0 loads by TMA (weights and tokens of 64 or 128 k per stage), warp 1
//    issues tcgen05.mma, one accumulator of NT columns in tensor memory.  A
//    grid that fits one CTA per SM takes all of the shared memory for its
//    stages; a larger one half of it, two CTAs per SM, while NT <= 128.
//  * Every CTA parks its fp32 partial tile in its own shared memory, token by
//    token, and the cluster's CTAs add the partials through distributed shared
//    memory in part order, each finishing a share of the tile's elements: the
//    epilogue (epilogue.cuh) runs once per element, on 8 neighbouring features
//    of a token per thread, 16 bytes per access also where rows are not
//    aligned (rowvec.cuh).
//  * kGated: the tile's 128 rows are 64 features of Wg and the same 64 of Wu,
//    so one MMA stream gives both projections of a hidden unit in one tile.
//  * Bound by HBM for single tokens: 4096 -> 14336 features in bf16 20.1 us, 5.8
//    TB/s of 6.8, 14336 -> 4096 20.0 us with K split; below that by latency:
//    1024 -> 1024 6.9 us a call in a graph, weights from HBM.
//  * Up to three independent products (a backward pass's) go out as one launch,
//    their tiles one after the other in one grid.
//  * Every wait is bounded (ptx.cuh).
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
#include "rowvec.cuh"
#include "tc_tile.cuh"
#include "tmap.cuh"

// Compiled once per type and kind of epilogue (DGEMM_FUSED_UNIT): 0: bf16
// linear, 1: fp16 linear, 2: bf16 gated, 3: fp16 gated.
#ifndef DGEMM_FUSED_UNIT
#define DGEMM_FUSED_UNIT 0
#endif
#define DG_CAT2(a, b) a##b
#define DG_CAT(a, b) DG_CAT2(a, b)
#define DG_UNIT_LAUNCHER DG_CAT(launch_fused_small_unit_, DGEMM_FUSED_UNIT)

namespace dg {
namespace {

#if DGEMM_FUSED_UNIT & 1
using Elem = __half;
#else
using Elem = __nv_bfloat16;
#endif

struct SmallCfg {
  static constexpr int BOX = 64;              // elements in a 128-byte swizzle row
  static constexpr int TF = 128;              // features (MMA rows) of a tile
  static constexpr int W_CHUNK = TF * 128;    // weights of 64 k
  static constexpr int MAX_STAGES = 8, MAX_SPLITS = 8;
  // bars (full[8], empty[8], accf, stall), TMEM slot, abort flag; 1024 for alignment
  static constexpr int TAIL_BYTES = (2 * MAX_STAGES + 2) * 8 + 16 + 1024;
  static constexpr int BUDGET2 = 113 * 1024 - TAIL_BYTES;  // two CTAs per SM
  static constexpr int BUDGET1 = 226 * 1024 - TAIL_BYTES;  // one
};

// producer, MMA, four drain warps; without a K split two more for the epilogue
template <bool SPLIT>
constexpr int kThreads = SPLIT ? 192 : 256;

// Stages of weights that a CTA sends for before the kernel ahead of it on the
// stream is done: 1 x 4096 x 14336 22.1 -> 21.7 us, gated block 64 x 1024 x 4096
// 16.3 -> 15.4; from 8 on slower than none (23.3 us with 16).
constexpr int kAheadStages = 3;

// Rounds of the epilogue whose inputs are in flight: 256 x 4096 x 4096 with a
// residual 21.6 -> 20.6 us, 1 x 4096 x 14336 21.8 -> 21.4, gated backward 5136 x
// 784 x 3408 218 -> 210 (one round ahead 20.9, 21.4 and 212).
constexpr int kInputsAhead = 2;

// Site codes of the bounded waits.
enum : int {
  kSite4ProducerEmpty = 0xb1,
  kSite4ProducerDrain = 0xb2,
  kSite4MmaFull = 0xb3,
  kSite4MmaDrain = 0xb4,
  kSite4DrainAccFull = 0xb5,
  kSite4TestStall = 0xb6,  // DGEMM_TC_TEST_STALL: the MMA thread's test wait ran out
};

struct SmallMaps {
  CUtensorMap w, x, w2, x2;
};

struct SmallArgs {
  int M, N, K;
  int dual, act;
  int wt, xt;  // weights stored N x K (read K-major); tokens stored K x M (MN-major)
  int nt, kd, stages;
  uint32_t idesc;
  uint32_t tmem_cols;
  const void *in0, *in1, *bias;
  int64_t ldi0, ldi1;
  void *out[3];
  int64_t ldo[3];
  int *watchdog;
};

// NP products of one launch: their maps and arguments, the first tile of each.
template <int NP>
struct SmallBatch {
  SmallMaps maps[NP];
  SmallArgs p[NP];
  int first[NP + 1];
  int splits, stall;
};

// Descriptor of the k-th 16-element K slice of an operand tile (tc_tile.cuh's
// operand_desc with the layout as an argument): MN-major tiles advance two
// groups of 8 K rows, K-major ones 32 bytes within a 128-byte row; box is the
// distance between 128-byte blocks of M or N, or between 64-element blocks of K.
__device__ __forceinline__ uint64_t slice_desc(uint32_t tile, int k, uint32_t box, bool mn) {
  return smem_desc(tile + (mn ? (uint32_t)k * 2048u : (uint32_t)(k >> 2) * box + (uint32_t)(k & 3) * 32u),
                   mn ? box : 16u, 1024u);
}

// SPLIT: a tile's K range is shared by a cluster.  AL: every row of every
// output and input of the epilogue is 16-byte aligned.  (Template arguments
// because a short kernel's time is partly that of fetching its instructions:
// one kernel for all four took 0.3 us longer for 1 x 1024 x 1024.)
// LAYOUT: 0: tokens M x K, weights K x N; 1: weights N x K; 2: tokens K x M,
// weights K x N; 3: as the arguments say (for several products; the descriptors
// cost the MMA thread instructions then, 0.3 us at 64 x 4096 x 1024).
template <class T, Epi EPI, bool SPLIT, bool AL, int NP, int LAYOUT>
__global__ void __launch_bounds__(kThreads<SPLIT>, 2)
    fused_small_kernel(const __grid_constant__ SmallBatch<NP> batch) {
  using G = SmallCfg;
  constexpr int THREADS = kThreads<SPLIT>;
  const int splits = SPLIT ? batch.splits : 1;
  pdl_launch_dependents();
  const int part = SPLIT ? blockIdx.x % splits : 0;
  int unit = SPLIT ? blockIdx.x / splits : blockIdx.x;
  int job = 0;
#pragma unroll
  for (int j = 1; j < NP; ++j)
    if (unit >= batch.first[j]) job = j;
  const SmallArgs &p = batch.p[job];
  const SmallMaps &maps = batch.maps[job];
  unit -= batch.first[job];
  const bool wt = LAYOUT == 3 ? p.wt != 0 : LAYOUT == 1, xt = LAYOUT == 3 ? p.xt != 0 : LAYOUT == 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_base);
  const int bk = p.kd * G::BOX;
  const uint32_t w_bytes = (uint32_t)(G::W_CHUNK * p.kd), x_bytes = (uint32_t)(p.nt * 128 * p.kd);
  const uint32_t stage_bytes = w_bytes + x_bytes;
  const uint32_t bars = base + (uint32_t)p.stages * stage_bytes;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (G::MAX_STAGES + s); };
  const uint32_t accf_bar = bars + 8u * (2 * G::MAX_STAGES);
  const uint32_t stall_bar = bars + 8u * (2 * G::MAX_STAGES + 1);  // nothing ever arrives here
  uint8_t *tail = smem + (bars - base) + 8 * (2 * G::MAX_STAGES + 2);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  auto w_tile = [&](int s) { return base + (uint32_t)s * stage_bytes; };
  auto x_tile = [&](int s) { return base + (uint32_t)s * stage_bytes + w_bytes; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int TF = EPI == Epi::kGated ? G::TF / 2 : G::TF;  // output features of a tile
  const int tiles_t = (p.M + p.nt - 1) / p.nt, tiles_f = (p.N + TF - 1) / TF;
  const int tiles1 = tiles_t * tiles_f;
  const bool second = unit >= tiles1;  // kPair: a tile of the second product
  const int tile = second ? unit - tiles1 : unit;
  const int f0 = (tile / tiles_t) * TF, t0 = (tile % tiles_t) * p.nt;
  const bool sum = EPI == Epi::kLinear && p.dual == (int)Dual::kSum;
  const int kb1 = (p.K + bk - 1) / bk;
  const int kblocks = sum ? 2 * kb1 : kb1;
  const int per = (kblocks + splits - 1) / splits;
  const int kb_begin = min(kblocks, part * per), kb_end = min(kblocks, part * per + per);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accf_bar, 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0 && p.K > 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x);
    // The first weights towards L2 while the kernel before this one on the
    // stream is still at work.
    const int ahead = min(kb_end, kb_begin + kAheadStages);
    for (int kb = kb_begin; kb < ahead; ++kb) {
      const bool set2 = second || kb >= kb1;
      const int k0 = (kb >= kb1 ? kb - kb1 : kb) * bk;
      const CUtensorMap *mw = set2 ? &maps.w2 : &maps.w;
      if (wt) {
        for (int c = 0; c < p.kd; ++c) {
          tma_prefetch_2d(mw, k0 + c * G::BOX, f0);
          if constexpr (EPI == Epi::kGated) tma_prefetch_2d(&maps.w2, k0 + c * G::BOX, f0);
        }
      } else {
        tma_prefetch_2d(mw, f0, k0);
        if constexpr (EPI == Epi::kGated)
          tma_prefetch_2d(&maps.w2, f0, k0);
        else
          tma_prefetch_2d(mw, f0 + G::BOX, k0);
      }
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // set-up done; the previous kernel on the stream has completed

  // The epilogue's inputs (residual; G and U) are read kInputsAhead rounds
  // ahead, the first of them during the main loop.
  constexpr int Q = TF / 8;  // threads per token
  const int live = min(p.nt, p.M - t0), feats = min(TF, p.N - f0);
  const int n = live * Q, end = f0 + feats, round = splits * THREADS;
  const int e0 = part * THREADS + threadIdx.x;
  const int f = 8 * (e0 % Q), col = f0 + f;  // the same in every round
  const T *in0 = static_cast<const T *>(p.in0), *in1 = static_cast<const T *>(p.in1);
  const bool has_in0 = EPI != Epi::kGated && in0 != nullptr;
  struct Inputs {
    RowBlocks x0, x1;
  } ahead[kInputsAhead];
  auto fetch = [&](int e) {
    const int t = e / Q;
    const int cols = t < live && f < feats ? end : 0;
    const int64_t row = t0 + t;
    Inputs r = {};
    if (has_in0) r.x0 = fetch_row16<T, AL>(in0 + row * p.ldi0, col, cols);
    if (EPI == Epi::kGatedBwd) r.x1 = fetch_row16<T, AL>(in1 + row * p.ldi1, col, cols);
    return r;
  };
  auto fetch_first = [&] {
#pragma unroll
    for (int k = 0; k < kInputsAhead; ++k) ahead[k] = fetch(e0 + k * round);
  };
  if (warp != 0) fetch_first();

  bool all_sent = false;  // this thread is the producer and has sent for every stage
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!mbar_try_wait(empty_bar(stage), phase ^ 1u) &&
            (*abort_flag || !mbar_wait(empty_bar(stage), phase ^ 1u))) {
          if (!*abort_flag) watchdog_trip(p.watchdog, kSite4ProducerEmpty, abort_flag);
          ok = false;
          break;
        }
        const bool set2 = second || kb >= kb1;
        const int k0 = (kb >= kb1 ? kb - kb1 : kb) * bk;
        const CUtensorMap *mw = set2 ? &maps.w2 : &maps.w, *mx = set2 ? &maps.x2 : &maps.x;
        const uint32_t fb = full_bar(stage);
        if (wt) {  // K-major: 64 k x features per box
          for (int c = 0; c < p.kd; ++c) {
            const uint32_t dst = w_tile(stage) + (uint32_t)(c * G::W_CHUNK);
            tma_load_2d(dst, mw, fb, k0 + c * G::BOX, f0);
            if constexpr (EPI == Epi::kGated)
              tma_load_2d(dst + G::W_CHUNK / 2, &maps.w2, fb, k0 + c * G::BOX, f0);
          }
        } else {  // MN-major: 64 features x bk k per box
          tma_load_2d(w_tile(stage), mw, fb, f0, k0);
          if constexpr (EPI == Epi::kGated)
            tma_load_2d(w_tile(stage) + w_bytes / 2, &maps.w2, fb, f0, k0);
          else
            tma_load_2d(w_tile(stage) + w_bytes / 2, mw, fb, f0 + G::BOX, k0);
        }
        if (xt) {
          for (int c = 0; c < p.nt / G::BOX; ++c)
            tma_load_2d(x_tile(stage) + (uint32_t)(c * bk * 128), mx, fb, t0 + c * G::BOX, k0);
        } else {
          for (int c = 0; c < p.kd; ++c)
            tma_load_2d(x_tile(stage) + (uint32_t)(c * p.nt * 128), mx, fb, k0 + c * G::BOX, t0);
        }
        mbar_arrive_expect_tx(fb, stage_bytes);  // announced after the copies are issued
        ++issued;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      all_sent = ok;
      if (!ok) {  // no TMA write lands after this CTA has left
        int s = stage;
        uint32_t ph = phase;
        const int n = issued < p.stages ? issued : p.stages;
        for (int i = 0; i < n; ++i) {
          if (--s < 0) {
            s = p.stages - 1;
            ph ^= 1u;
          }
          if (!mbar_wait(full_bar(s), ph)) atomicCAS(p.watchdog, 0, kSite4ProducerDrain);
        }
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      const uint32_t w_box = wt ? (uint32_t)G::W_CHUNK : w_bytes / 2;
      const uint32_t x_box = xt ? (uint32_t)(bk * 128) : (uint32_t)(p.nt * 128);
      bool ok = true;
      if (batch.stall && blockIdx.x == 0) {  // test hook: a wait that runs out
        if (!mbar_wait(stall_bar, 0)) watchdog_trip(p.watchdog, kSite4TestStall, abort_flag);
        ok = false;
      }
      for (int kb = kb_begin; kb < kb_end && ok; ++kb) {
        if (!mbar_try_wait(full_bar(stage), phase) &&
            (*abort_flag || !mbar_wait(full_bar(stage), phase))) {
          if (!*abort_flag) watchdog_trip(p.watchdog, kSite4MmaFull, abort_flag);
          break;
        }
        tc_fence_after();
        for (int h = 0; h < p.kd; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = 4 * h + q;
            umma_f16(tmem_base, slice_desc(w_tile(stage), k, w_box, !wt),
                     slice_desc(x_tile(stage), k, x_box, xt), p.idesc,
                     (kb > kb_begin || k > 0) ? 1u : 0u);
          }
        umma_commit(empty_bar(stage));
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      umma_commit(accf_bar);  // every MMA issued above has completed
      if (!mbar_wait(accf_bar, 0)) atomicCAS(p.watchdog, 0, kSite4MmaDrain);
    }
  } else if (warp < 6) {
    // ------------------------------- drain: partial tile to shared memory
    const int quarter = warp & 3;
    const bool ok = !*abort_flag && mbar_wait(accf_bar, 0);
    if (!ok && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite4DrainAccFull, abort_flag);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      // Every MMA has completed, so the stage area is idle: partial[t][f]
      float *col = reinterpret_cast<float *>(smem) + quarter * 32 + lane;
      const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16);
      for (int c0 = 0; c0 < live; c0 += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(t_row + (uint32_t)c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          col[(c0 + j) * G::TF] = kb_end > kb_begin ? __uint_as_float(r[j]) : 0.f;
      }
      tc_fence_before();
    }
  }

  if (warp == 0) {
    __syncwarp();
    fetch_first();
  }
  // ------------------------------------------ join the parts, finish, store
  // Every thread of every CTA of the cluster gets here, also after a bounded
  // wait gave up.
  __syncthreads();
  bool aborted = false;
  uint32_t at[G::MAX_SPLITS];
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();
#pragma unroll
    for (int s = 0; s < G::MAX_SPLITS; ++s)
      at[s] = s < splits ? mapa_shared(base, (uint32_t)s) : 0u;
    // looked at before anything is stored, so that these loads and those of the
    // partials are in flight together
    const uint32_t flag = smem_u32(const_cast<int *>(abort_flag)) - base;
#pragma unroll
    for (int s = 0; s < G::MAX_SPLITS; ++s)
      if (s < splits) aborted |= ld_cluster_s32(at[s] + flag) != 0;
  } else {
    aborted = *abort_flag != 0;
  }
  {
    auto sum4 = [&](uint32_t off) {  // parts added in K order
      if constexpr (SPLIT) {
        float4 v[G::MAX_SPLITS];
#pragma unroll
        for (int s = 0; s < G::MAX_SPLITS; ++s)
          if (s < splits) v[s] = ld_cluster_f4(at[s] + off);
        float4 r = v[0];
#pragma unroll
        for (int s = 1; s < G::MAX_SPLITS; ++s)
          if (s < splits) r.x += v[s].x, r.y += v[s].y, r.z += v[s].z, r.w += v[s].w;
        return r;
      } else {
        return *reinterpret_cast<const float4 *>(smem + off);
      }
    };
    constexpr int kOuts = EPI == Epi::kLinear ? 2 : 3;
    const bool pair_out = EPI == Epi::kLinear && p.dual == (int)Dual::kPair;
    auto output = [&](int o, int *slot) {  // which output array result o goes to; false: none
      *slot = pair_out ? (second ? 1 : 0) : o;
      return !(pair_out && o) && p.out[*slot] != nullptr;
    };
    const T *bias = static_cast<const T *>(p.bias);
    const bool kept = !pair_out && p.out[1] != nullptr;
    // whole warps go round together: their stores put blocks together
#pragma unroll 1
    for (int e = e0; e - lane < n; e += round) {
      const int t = e / Q;
      const bool in = t < live && f < feats;
      const int64_t row = t0 + t;
      float a[8], b[8];
      uint32_t i0[4], i1[4], w[3][4];
      auto unpack = [&](uint4 x, uint32_t (&v)[4]) { v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w; };
      const Inputs now = ahead[0];
#pragma unroll
      for (int k = 0; k + 1 < kInputsAhead; ++k) ahead[k] = ahead[k + 1];
      ahead[kInputsAhead - 1] = fetch(e + kInputsAhead * round);
      if (in) {
        if (has_in0) unpack(take_row16<T, AL>(now.x0, in0 + row * p.ldi0, col, end), i0);
        if (EPI == Epi::kGatedBwd)
          unpack(take_row16<T, AL>(now.x1, in1 + row * p.ldi1, col, end), i1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v = sum4((uint32_t)((t * G::TF + f + 4 * h) * 4));
          a[4 * h] = v.x, a[4 * h + 1] = v.y, a[4 * h + 2] = v.z, a[4 * h + 3] = v.w;
          if constexpr (EPI == Epi::kGated) {
            const float4 u = sum4((uint32_t)((t * G::TF + TF + f + 4 * h) * 4));
            b[4 * h] = u.x, b[4 * h + 1] = u.y, b[4 * h + 2] = u.z, b[4 * h + 3] = u.w;
          }
        }
        if (EPI == Epi::kLinear && bias != nullptr) {
          uint32_t v[4];
          unpack(load_row16<T, AL>(bias, col, end), v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 c = unpack2<T>(v[j]);
            a[2 * j] += c.x, a[2 * j + 1] += c.y;
          }
        }
        epilogue_row<EPI, T, 4>(p.act, has_in0, kept, a, b, i0, i1, w[0], w[1], w[2]);
      }
      if (aborted) break;  // the same for the whole cluster
#pragma unroll
      for (int o = 0; o < kOuts; ++o) {
        int slot;
        if (output(o, &slot)) {
          const uint4 v[1] = {make_uint4(w[o][0], w[o][1], w[o][2], w[o][3])};
          store_row16<T, AL, 1, Q>(static_cast<T *>(p.out[slot]) + row * p.ldo[slot],
                                   in ? col : end, end, v);
        }
      }
    }
  }
  if (aborted && all_sent) {  // nor where another thread's wait gave up
    const int sent = kb_end - kb_begin;
    for (int i = max(0, sent - p.stages); i < sent; ++i)
      if (!mbar_wait(full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u))
        atomicCAS(p.watchdog, 0, kSite4ProducerDrain);
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while a peer may still read its partial
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// ------------------------------------------------------------- host side
// Maps of the weights (boxes of 64 k x `w_rows` features, or 64 features x bk
// k) and the tokens.
bool small_maps(CUtensorMap *tw, CUtensorMap *tx, CUtensorMapDataType dt, const FusedGemm &p,
                const void *X, int64_t ldx, const void *W, int64_t ldw, int nt, int bk, int w_rows) {
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  const bool w = p.b_t ? make_map(tw, W, dt, 2, p.N, p.K, ldw, 64, w_rows, swz)
                       : make_map(tw, W, dt, 2, p.K, p.N, ldw, 64, bk, swz);
  const bool x = p.a_t ? make_map(tx, X, dt, 2, p.K, p.M, ldx, 64, bk, swz)
                       : make_map(tx, X, dt, 2, p.M, p.K, ldx, 64, nt, swz);
  return w && x;
}

// Launch one instance, opted in to all of the shared memory once per device.
template <auto KERNEL, class B>
cudaError_t launch_one(unsigned grid, bool split, int smem, cudaStream_t stream, unsigned cluster,
                       const B &batch) {
  using G = SmallCfg;
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             G::BUDGET1 + G::TAIL_BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  e = launch_kernel(KERNEL, dim3(grid), dim3(split ? kThreads<true> : kThreads<false>),
                    (size_t)smem, stream, cluster, batch);
  if (e == cudaSuccess) count_launch();
  return e;
}

// `n` products (n <= NP) in one launch; their plans agree in splits and per_sm.
template <Epi EPI, int NP, int LAYOUT>
cudaError_t launch_small(const FusedGemm *ps, const SmallPlan *plans, int n, int *watchdog,
                         cudaStream_t stream) {
  using G = SmallCfg;
  using T = Elem;
  SmallBatch<NP> batch;
  memset(&batch, 0, sizeof batch);
  const CUtensorMapDataType dt = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
  constexpr int tf = EPI == Epi::kGated ? G::TF / 2 : G::TF;
  const int splits = plans[0].splits;
  int smem = 0;
  int64_t tiles = 0;
  bool vec = true;
  for (int j = 0; j < n; ++j) {
    const FusedGemm &p = ps[j];
    const SmallPlan &plan = plans[j];
    SmallMaps &maps = batch.maps[j];
    SmallArgs &a = batch.p[j];
    if (plan.splits != splits || plan.per_sm != plans[0].per_sm) return cudaErrorInvalidValue;
    a.nt = plan.nt, a.kd = plan.kd;
    a.wt = p.b_t, a.xt = p.a_t;
    const int bk = 64 * plan.kd;
    if (p.K > 0) {
      if (!small_maps(&maps.w, &maps.x, dt, p, p.A, p.lda, p.B, p.ldb, plan.nt, bk, tf))
        return cudaErrorInvalidValue;
      if (p.dual != Dual::kNone) {
        const bool gated = p.dual == Dual::kGated;
        if (!small_maps(&maps.w2, &maps.x2, dt, p, gated ? p.A : p.A2, gated ? p.lda : p.lda2, p.B2,
                        p.ldb2, plan.nt, bk, tf))
          return cudaErrorInvalidValue;
      }
    }
    const int stage_bytes = (G::W_CHUNK + plan.nt * 128) * plan.kd;
    a.stages = small_stages(plan);
    // the parked partial tile takes the stages' place
    if (a.stages < 2 || a.stages * stage_bytes < plan.nt * G::TF * 4) return cudaErrorInvalidValue;
    const int bytes = a.stages * stage_bytes + G::TAIL_BYTES;
    smem = smem > bytes ? smem : bytes;
    a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p.b_t ? 0u : 1u) << 15) |
              ((p.a_t ? 1u : 0u) << 16) | ((uint32_t)(plan.nt >> 3) << 17) |
              ((uint32_t)(G::TF >> 4) << 24);
    a.tmem_cols = 32;
    while ((int)a.tmem_cols < plan.nt) a.tmem_cols *= 2;
    a.M = p.M, a.N = p.N, a.K = p.K;
    a.dual = (int)p.dual, a.act = p.act;
    a.in0 = p.in0, a.in1 = p.in1, a.bias = p.bias;
    a.ldi0 = p.ldi0, a.ldi1 = p.ldi1;
    a.out[0] = p.out0, a.out[1] = p.out1, a.out[2] = p.out2;
    a.ldo[0] = p.ldo0, a.ldo[1] = p.ldo1, a.ldo[2] = p.ldo2;
    vec = vec && p.N % 8 == 0 && rows_aligned(p.in0, p.in0 ? p.ldi0 : 0) &&
          rows_aligned(p.in1, p.in1 ? p.ldi1 : 0) && rows_aligned(p.bias, 0);
    for (int i = 0; i < 3; ++i) vec = vec && rows_aligned(a.out[i], a.out[i] ? a.ldo[i] : 0);
    a.watchdog = watchdog;
    batch.first[j] = (int)tiles;
    tiles += (int64_t)((p.M + plan.nt - 1) / plan.nt) * ((p.N + tf - 1) / tf) *
             (p.dual == Dual::kPair ? 2 : 1);
    if (tiles * splits > 0x3fffffff) return cudaErrorInvalidValue;
  }
  for (int j = n; j <= NP; ++j) batch.first[j] = (int)tiles;
  batch.splits = splits;
  batch.stall = test_stall();
  const unsigned grid = (unsigned)(tiles * splits), cluster = (unsigned)splits;
  if (splits > 1)
    return vec ? launch_one<fused_small_kernel<T, EPI, true, true, NP, LAYOUT>>(grid, true, smem, stream,
                                                                        cluster, batch)
               : launch_one<fused_small_kernel<T, EPI, true, false, NP, LAYOUT>>(grid, true, smem, stream,
                                                                         cluster, batch);
  return vec ? launch_one<fused_small_kernel<T, EPI, false, true, NP, LAYOUT>>(grid, false, smem, stream,
                                                                       1u, batch)
             : launch_one<fused_small_kernel<T, EPI, false, false, NP, LAYOUT>>(grid, false, smem, stream,
                                                                        1u, batch);
}

}  // namespace

cudaError_t DG_UNIT_LAUNCHER(const FusedGemm *p, const SmallPlan *plan, int n, int *watchdog,
                             cudaStream_t stream) {
#if DGEMM_FUSED_UNIT < 2
  if (n > 1) return launch_small<Epi::kLinear, kMaxBatch, 3>(p, plan, n, watchdog, stream);
  if (p->a_t) return launch_small<Epi::kLinear, 1, 2>(p, plan, n, watchdog, stream);
  return p->b_t ? launch_small<Epi::kLinear, 1, 1>(p, plan, n, watchdog, stream)
                : launch_small<Epi::kLinear, 1, 0>(p, plan, n, watchdog, stream);
#else  // the gated epilogues' tokens are activations, M x K
  if (p->epi == Epi::kGated)
    return p->b_t ? launch_small<Epi::kGated, 1, 1>(p, plan, n, watchdog, stream)
                  : launch_small<Epi::kGated, 1, 0>(p, plan, n, watchdog, stream);
  return p->b_t ? launch_small<Epi::kGatedBwd, 1, 1>(p, plan, n, watchdog, stream)
                : launch_small<Epi::kGatedBwd, 1, 0>(p, plan, n, watchdog, stream);
#endif
}

#if DGEMM_FUSED_UNIT == 0
int small_stages(const SmallPlan &plan) {
  using G = SmallCfg;
  const int n = (plan.per_sm == 2 ? G::BUDGET2 : G::BUDGET1) / ((G::W_CHUNK + plan.nt * 128) * plan.kd);
  return n < G::MAX_STAGES ? n : G::MAX_STAGES;
}

// By the occupancy query, once per device and cluster size (every instance of
// the kernel has the same block and bounds; a cluster has to fit in one GPC,
// which holds a few SMs more than a multiple of its size).  The query counts a
// kernel that allocates tensor memory as one CTA per SM whatever its shared
// memory, but two run: with half an SM's memory each, 152 pairs of CTAs were seen
// at work on one SM at the same time.  So clusters of s with two CTAs per SM are
// taken to be as many as clusters of s / 2 with one.  For a kernel of the same
// size without tensor memory the query says 152, 97, 74, 46 and 36 clusters of 2,
// 3, 4, 6 and 8; this gives 152, 92, 76, 46 and 36.  (1 x 4096 x 14336 in 32
// clusters of 8: 20.1 us; in 32 of 4: 21.5.)
int64_t small_resident(const SmallPlan &plan, int num_sms) {
  using G = SmallCfg;
  if (plan.splits == 1) return (int64_t)plan.per_sm * num_sms;
  if (plan.per_sm == 2) {
    const bool even = plan.splits % 2 == 0;
    const int64_t one = small_resident({plan.nt, plan.kd, even ? plan.splits / 2 : plan.splits, 1}, num_sms);
    return even ? one : 2 * one;
  }
  static std::atomic<int> cache[64][G::MAX_SPLITS + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms / plan.splits;
  std::atomic<int> &slot = cache[dev][plan.splits];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    auto kern = fused_small_kernel<Elem, Epi::kLinear, true, true, 1, 0>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.splits);
    cfg.blockDim = dim3(kThreads<true>);
    cfg.dynamicSmemBytes = G::BUDGET1 + G::TAIL_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             G::BUDGET1 + G::TAIL_BYTES) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();  // not sticky; an estimate will do
      n = num_sms / plan.splits;
    }
    slot.store(n, std::memory_order_relaxed);
  }
  return n;
}
#endif

}  // namespace dg
