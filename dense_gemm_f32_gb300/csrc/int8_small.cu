// int8_small.cu -- products with 8-bit weights for few tokens: single tokens and
// serving batches, and small layers.
//
// Bound by reading the weights, so they are the rows of the MMA and the tokens
// its columns, as in fused_small.cu: D^T = W T^T over tiles of 128 features x NT
// tokens (16 to 128), the K range of a tile split over a cluster of up to 8 CTAs
// where there are few tiles, partial tiles joined through distributed shared
// memory in part order.  T holds the tokens' integers in fp16 (quant.cu).
//  * Warp 0 loads stages of 128 k by TMA (16 KB of weights, the tokens' 256
//    bytes each); warps 2-9 widen the weights into one of two places in tensor
//    memory (int8.cuh), half a row each; warp 1 issues tcgen05.mma with A from there.
//  * The first stages of weights are loaded before the kernel ahead on the
//    stream, which quantises the tokens, is done: it signals only after its own
//    wait, so whatever wrote the weights is done by then.  (Not where that kernel also
//    copies weights to rows that TMA can read.)
//  * kGated: rows 0-63 are features of Wg, 64-127 the same of Wu; the hidden
//    units go out in fp32, as the next step quantises them against the largest
//    of their row: rounded to 16 bits before that, one in a hundred would become
//    another integer.
// 64 tokens x 14336 -> 4096 in 19.5 us (floor 9.1: 61 MB): the weights stream at 6 TB/s for 10
// of them, widening and MMAs hidden (without either 17.6); before that the tokens' kernel (3)
// and the first loads (2), after it the join through distributed shared memory and the
// cluster's barriers (4).  More places in tensor memory, or four converter warps for
// every other block, changed nothing.
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
  static constexpr int TF = 128, BK = 128;    // rows of weights and k of a stage
  static constexpr int W_BYTES = TF * BK;
  static constexpr int MAX_STAGES = 10, MAX_SPLITS = 8;
  static constexpr int A_COLS = 64;           // tensor memory of widened weights of 128 k
  static constexpr int CONV_WARPS = 8, THREADS = 32 * (2 + CONV_WARPS);
  // bars (full, empty, conv[2], accf, stall), TMEM slot, abort flag; 1024 for alignment
  static constexpr int NUM_BARS = 2 * MAX_STAGES + 4;
  static constexpr int TAIL_BYTES = NUM_BARS * 8 + 16 + 1024;
  static constexpr int BUDGET2 = 113 * 1024 - TAIL_BYTES;  // two CTAs per SM
  static constexpr int BUDGET1 = 226 * 1024 - TAIL_BYTES;  // one
};

// Site codes of the bounded waits.
enum : int {
  kSite5ProducerEmpty = 0xd1,
  kSite5ProducerDrain = 0xd2,
  kSite5ConvFull = 0xd3,
  kSite5ConvSlot = 0xd4,
  kSite5MmaConv = 0xd5,
  kSite5MmaDrain = 0xd6,
  kSite5DrainAccFull = 0xd7,
  kSite5TestStall = 0xd8,  // DGEMM_TC_TEST_STALL: the MMA thread's test wait ran out
};

struct Maps {
  CUtensorMap w, w2, t;
};

struct Args {
  int M, N, K;
  int act, nt, stages, splits, stall, early;
  uint32_t idesc, tmem_cols;
  const float *t_scale, *w_scale, *w2_scale;
  const void *in0, *bias;
  int64_t ldi0;
  void *out;
  int64_t ldo;
  int *watchdog;
};

// GATED: out is H in fp32, rows of whole vectors; else out and in0 are T.  AL:
// every row of out and in0 is 16-byte aligned.
template <class T, bool GATED, bool SPLIT, bool AL>
__global__ void __launch_bounds__(Cfg::THREADS, 2)
    int8_small_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  using G = Cfg;
  pdl_launch_dependents();
  const int splits = SPLIT ? p.splits : 1;
  const int part = SPLIT ? blockIdx.x % splits : 0, tile = SPLIT ? blockIdx.x / splits : blockIdx.x;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_base);
  const uint32_t t_bytes = (uint32_t)p.nt * 256u, stage_bytes = (uint32_t)G::W_BYTES + t_bytes;
  const uint32_t bars = base + (uint32_t)p.stages * stage_bytes;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (G::MAX_STAGES + s); };
  auto conv_bar = [&](int b) { return bars + 8u * (2 * G::MAX_STAGES + b); };
  const uint32_t accf_bar = bars + 8u * (2 * G::MAX_STAGES + 2);
  const uint32_t stall_bar = bars + 8u * (2 * G::MAX_STAGES + 3);  // nothing ever arrives here
  uint8_t *tail = smem + (bars - base) + 8 * G::NUM_BARS;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  auto w_tile = [&](int s) { return base + (uint32_t)s * stage_bytes; };
  auto t_tile = [&](int s) { return base + (uint32_t)s * stage_bytes + (uint32_t)G::W_BYTES; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int TF = GATED ? G::TF / 2 : G::TF;  // output features of a tile
  const int tiles_t = (p.M + p.nt - 1) / p.nt;
  const int f0 = (tile / tiles_t) * TF, t0 = (tile % tiles_t) * p.nt;
  const int kblocks = (p.K + G::BK - 1) / G::BK;
  const int per = (kblocks + splits - 1) / splits;
  const int kb_begin = min(kblocks, part * per), blocks = min(kblocks, part * per + per) - kb_begin;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(conv_bar(b), G::CONV_WARPS);
    mbar_init(accf_bar, 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0 && p.K > 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.t);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t a_tmem = tmem_base + (p.tmem_cols - 2u * G::A_COLS);  // behind the accumulator

  // What the epilogue needs of a thread's features, and of its first token, is read
  // now.
  constexpr int Q = TF / 8;  // threads per token
  const int live = min(p.nt, p.M - t0), feats = min(TF, p.N - f0), end = f0 + feats;
  const int n = live * Q, round = splits * G::THREADS, e0 = part * G::THREADS + threadIdx.x;
  static_assert(G::THREADS % Q == 0, "a thread keeps its features from round to round");
  const int f = 8 * (e0 % Q), col = f0 + f;
  float ws[8], ws2[8], bias[8];
  struct Inputs {
    float ts;
    RowBlocks res;
  } ahead;
  const T *in0 = static_cast<const T *>(p.in0);
  auto fetch = [&](int e) {
    const int t = e / Q;
    const bool in = t < live && f < feats;
    const int64_t row = t0 + t;
    Inputs x = {};
    x.ts = in ? p.t_scale[row] : 0.f;
    if (!GATED && in0 != nullptr) x.res = fetch_row16<T, AL>(in0 + row * p.ldi0, col, in ? end : 0);
    return x;
  };
  auto fetch_first = [&] {
    const bool mine = e0 < n;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = mine && f + j < feats;
      ws[j] = in ? p.w_scale[col + j] : 0.f;
      ws2[j] = GATED && in ? p.w2_scale[col + j] : 0.f;
      bias[j] = !GATED && in && p.bias != nullptr ? to_f32<T>(static_cast<const T *>(p.bias)[col + j]) : 0.f;
    }
    ahead = fetch(e0);
  };

  bool all_sent = false;  // this thread is the producer and has sent for every stage
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      auto weights = [&](int s, int k0) {
        tma_load_2d(w_tile(s), &maps.w, full_bar(s), k0, f0);
        if constexpr (GATED) tma_load_2d(w_tile(s) + G::W_BYTES / 2, &maps.w2, full_bar(s), k0, f0);
      };
      const int early = p.early ? min(blocks, p.stages) : 0;
      for (int i = 0; i < early; ++i) weights(i, (kb_begin + i) * G::BK);
      pdl_wait();  // the tokens are there
      int issued = 0, s = 0;
      uint32_t phase = 1;  // a fresh barrier's phase before is complete
      bool ok = true;
      for (int i = 0; i < blocks; ++i) {
        const int k0 = (kb_begin + i) * G::BK;
        if (!mbar_try_wait(empty_bar(s), phase) && (*abort_flag || !mbar_wait(empty_bar(s), phase))) {
          if (!*abort_flag) watchdog_trip(p.watchdog, kSite5ProducerEmpty, abort_flag);
          ok = false;
          break;
        }
        if (i >= early) weights(s, k0);
        tma_load_2d(t_tile(s), &maps.t, full_bar(s), k0, t0);
        tma_load_2d(t_tile(s) + t_bytes / 2, &maps.t, full_bar(s), k0 + 64, t0);
        mbar_arrive_expect_tx(full_bar(s), stage_bytes);  // announced after the copies are issued
        ++issued;
        if (++s == p.stages) s = 0, phase ^= 1u;
      }
      all_sent = ok;
      if (!ok) {  // no TMA write lands after this CTA has left
        for (int i = max(0, issued - p.stages); i < issued; ++i)
          if (!mbar_wait(full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u))
            atomicCAS(p.watchdog, 0, kSite5ProducerDrain);
      }
    } else {
      pdl_wait();
    }
    __syncwarp();
    fetch_first();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    // (the whole warp in the loop, descriptors by addition: as in int8_pair.cu)
    pdl_wait();
    fetch_first();
    bool ok = true;
    if (p.stall && blockIdx.x == 0) {  // test hook: a wait that runs out
      warp_wait(stall_bar, 0, lane, p.watchdog, kSite5TestStall, abort_flag);
      ok = false;
    }
    int s = 0;
    uint32_t phase = 0;
    const uint64_t desc0 = smem_desc(t_tile(0), 16u, 1024u);
    const uint32_t stage16 = stage_bytes >> 4, box16 = t_bytes >> 5;
    uint64_t desc = desc0;
    for (int i = 0; i < blocks && ok; ++i) {
      // the converters have seen the stage full; so does this warp, for the tokens
      ok = warp_wait(full_bar(s), phase, lane, p.watchdog, kSite5MmaConv, abort_flag) &&
           warp_wait(conv_bar(i & 1), (uint32_t)(i >> 1) & 1u, lane, p.watchdog, kSite5MmaConv, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t a = a_tmem + (uint32_t)((i & 1) * G::A_COLS);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < G::BK / 16; ++k)
          umma_f16_ta(tmem_base, a + 8u * k, desc + (k >> 2) * box16 + 2u * (k & 3), p.idesc,
                      k > 0 ? 1u : i > 0 ? 1u : 0u);
        umma_commit(empty_bar(s));
      }
      __syncwarp();
      desc += stage16;
      if (++s == p.stages) s = 0, phase ^= 1u, desc = desc0;
    }
    if (elect_one()) umma_commit(accf_bar);  // every MMA issued above has completed
    __syncwarp();
    if (!mbar_wait(accf_bar, 0)) atomicCAS(p.watchdog, 0, kSite5MmaDrain);
  } else {
    // ---------------------------- widen the weights, then drain the accumulator
    pdl_wait();
    fetch_first();
    // four warps for each half of a stage's k
    const int quarter = warp & 3, half = (warp - 2) >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    int s = 0, free_s = 0;
    uint32_t phase = 0, free_phase = 0;
    for (int i = 0; i < blocks; ++i) {
      if (!warp_wait(full_bar(s), phase, lane, p.watchdog, kSite5ConvFull, abort_flag)) break;
      const uint8_t *w = smem + (w_tile(s) - base) + row * G::BK;
      uint32_t r[32];
      widen64(w, 4 * half, row & 7, r);
      if (i >= 2) {  // the MMAs that read this place two blocks ago are done
        if (!warp_wait(empty_bar(free_s), free_phase, lane, p.watchdog, kSite5ConvSlot, abort_flag)) break;
        if (++free_s == p.stages) free_s = 0, free_phase ^= 1u;
        tc_fence_after();
      }
      tmem_st_32x32b_x32(a_tmem + lanes + (uint32_t)((i & 1) * G::A_COLS + 32 * half), r);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(conv_bar(i & 1));
      if (++s == p.stages) s = 0, phase ^= 1u;
    }
    if (warp_wait(accf_bar, 0, lane, p.watchdog, kSite5DrainAccFull, abort_flag) && !*abort_flag) {
      tc_fence_after();
      // Every MMA has completed, so the stage area is idle: partial[t][f]
      float *col = reinterpret_cast<float *>(smem) + row;
      for (int c0 = 16 * half; c0 < live; c0 += 32) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem_base + lanes + (uint32_t)c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) col[(c0 + j) * G::TF] = blocks > 0 ? __uint_as_float(r[j]) : 0.f;
      }
      tc_fence_before();
    }
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
    auto sum8 = [&](int t, int f, float (&a)[8]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = sum4((uint32_t)((t * G::TF + f + 4 * h) * 4));
        a[4 * h] = v.x, a[4 * h + 1] = v.y, a[4 * h + 2] = v.z, a[4 * h + 3] = v.w;
      }
    };
    // whole warps go round together: their stores put blocks together
#pragma unroll 1
    for (int e = e0; e - lane < n; e += round) {
      const int t = e / Q;
      const bool in = t < live && f < feats;
      const int64_t row = t0 + t;
      float a[8], b[8];
      uint32_t i0[4], w0[4], w1[4], w2[4];
      const Inputs now = ahead;
      ahead = fetch(e + round);
      if (in) {
        const float ts = now.ts;
        sum8(t, f, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = scaled(a[j], ts, ws[j]) + bias[j];
        if constexpr (GATED) {
          sum8(t, TF + f, b);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = scaled(b[j], ts, ws2[j]);
        }
      }
      if constexpr (GATED) {
        if (in) {
          with_act(p.act, [&](auto c) {
            constexpr int ACT = decltype(c)::value;
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = act_f32<ACT>(a[j]) * b[j];
          });
          float4 *h = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * p.ldo + col);
          if (aborted) break;  // the same for the whole cluster
          h[0] = make_float4(a[0], a[1], a[2], a[3]);
          h[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
      } else {
        const bool has_in0 = in0 != nullptr;
        if (in) {
          if (has_in0) {
            const uint4 x = take_row16<T, AL>(now.res, in0 + row * p.ldi0, col, end);
            i0[0] = x.x, i0[1] = x.y, i0[2] = x.z, i0[3] = x.w;
          }
          epilogue_row<Epi::kLinear, T, 4>(p.act, has_in0, false, a, a, i0, i0, w0, w1, w2);
        }
        if (aborted) break;
        const uint4 v[1] = {make_uint4(w0[0], w0[1], w0[2], w0[3])};
        store_row16<T, AL, 1, Q>(static_cast<T *>(p.out) + row * p.ldo, in ? col : end, end, v);
      }
    }
  }
  if (aborted && all_sent) {  // no TMA write lands after this CTA has left
    for (int i = max(0, blocks - p.stages); i < blocks; ++i)
      if (!mbar_wait(full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u))
        atomicCAS(p.watchdog, 0, kSite5ProducerDrain);
  }
  if constexpr (SPLIT) {  // no CTA leaves while a peer may still read its partial
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();
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
int stages_of(const Int8Plan &plan) {
  const int n = (plan.per_sm == 2 ? Cfg::BUDGET2 : Cfg::BUDGET1) / (Cfg::W_BYTES + plan.nt * 256);
  return n < Cfg::MAX_STAGES ? n : Cfg::MAX_STAGES;
}

template <auto KERNEL>
cudaError_t launch_one(unsigned grid, size_t smem, cudaStream_t stream, unsigned cluster,
                       const Maps &maps, const Args &a) {
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::BUDGET1 + Cfg::TAIL_BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  e = launch_kernel(KERNEL, dim3(grid), dim3(Cfg::THREADS), smem, stream, cluster, maps, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class T, bool GATED>
cudaError_t launch_small(const Int8Gemm &p, const Int8Plan &plan, int *watchdog,
                         cudaStream_t stream) {
  using G = Cfg;
  constexpr int tf = GATED ? G::TF / 2 : G::TF;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  Args a;
  memset(&a, 0, sizeof a);
  if (p.K > 0) {
    const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!make_map(&maps.w, p.W, u8, 1, p.N, p.K, p.ldw, G::BK, tf, swz) ||
        (GATED && !make_map(&maps.w2, p.W2, u8, 1, p.N, p.K, p.ldw2, G::BK, tf, swz)) ||
        !make_map(&maps.t, p.T, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p.M, p.K, p.ldt, 64, plan.nt, swz))
      return cudaErrorInvalidValue;
  }
  a.M = p.M, a.N = p.N, a.K = p.K;
  a.act = p.act, a.nt = plan.nt, a.splits = plan.splits;
  a.early = p.early;
  a.stages = stages_of(plan);
  a.stall = test_stall();
  // fp16 operands, both K-major, fp32 accumulator
  a.idesc = (1u << 4) | ((uint32_t)(plan.nt >> 3) << 17) | ((uint32_t)(G::TF >> 4) << 24);
  a.tmem_cols = 256;  // accumulator of up to 128 columns, widened weights behind it
  a.t_scale = p.t_scale, a.w_scale = p.w_scale, a.w2_scale = p.w2_scale;
  a.in0 = p.in0, a.ldi0 = p.ldi0, a.bias = p.bias;
  a.out = p.out, a.ldo = p.ldo;
  a.watchdog = watchdog;
  const int stage_bytes = G::W_BYTES + plan.nt * 256;
  // the parked partial tile takes the stages' place
  if (plan.nt > 128 || a.stages < 2 || a.stages * stage_bytes < plan.nt * G::TF * 4)
    return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((p.M + plan.nt - 1) / plan.nt) * ((p.N + tf - 1) / tf);
  if (tiles * plan.splits > 0x3fffffff) return cudaErrorInvalidValue;
  const bool vec = GATED || (p.N % 8 == 0 && rows_aligned(p.in0, p.in0 ? p.ldi0 : 0) &&
                             rows_aligned(p.out, p.ldo));
  const size_t smem = (size_t)(a.stages * stage_bytes + G::TAIL_BYTES);
  const unsigned grid = (unsigned)(tiles * plan.splits), cluster = (unsigned)plan.splits;
  if constexpr (GATED) {
    return plan.splits > 1
               ? launch_one<int8_small_kernel<T, true, true, true>>(grid, smem, stream, cluster, maps, a)
               : launch_one<int8_small_kernel<T, true, false, true>>(grid, smem, stream, 1u, maps, a);
  } else {
    if (plan.splits > 1)
      return vec ? launch_one<int8_small_kernel<T, false, true, true>>(grid, smem, stream, cluster, maps, a)
                 : launch_one<int8_small_kernel<T, false, true, false>>(grid, smem, stream, cluster, maps, a);
    return vec ? launch_one<int8_small_kernel<T, false, false, true>>(grid, smem, stream, 1u, maps, a)
               : launch_one<int8_small_kernel<T, false, false, false>>(grid, smem, stream, 1u, maps, a);
  }
}

}  // namespace

int64_t int8_small_resident(int splits, int per_sm, int num_sms) {
  if (splits == 1) return (int64_t)per_sm * num_sms;
  if (per_sm == 2) {
    // The occupancy call counts one CTA of this kernel per SM whatever its shared memory (76 clusters
    // of two at 104 KB a CTA as at 226), so: clusters of half the size with one each, or twice as many.
    const bool even = splits % 2 == 0;
    const int64_t one = int8_small_resident(even ? splits / 2 : splits, 1, num_sms);
    return even ? one : 2 * one;
  }
  auto kern = int8_small_kernel<__half, false, true, true>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)splits);
  cfg.blockDim = dim3(Cfg::THREADS);
  cfg.dynamicSmemBytes = Cfg::BUDGET1 + Cfg::TAIL_BYTES;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::BUDGET1 + Cfg::TAIL_BYTES) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();  // not sticky; an estimate will do
    n = num_sms / splits;
  }
  return n;
}

cudaError_t launch_int8_small(const Int8Gemm &p, const Int8Plan &plan, int *watchdog,
                              cudaStream_t stream) {
  if (p.gated) return launch_small<__half, true>(p, plan, watchdog, stream);  // H is fp32
  return p.dtype == DGEMM_DTYPE_BF16 ? launch_small<__nv_bfloat16, false>(p, plan, watchdog, stream)
                                     : launch_small<__half, false>(p, plan, watchdog, stream);
}

}  // namespace dg
