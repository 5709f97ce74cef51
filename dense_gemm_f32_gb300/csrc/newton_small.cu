// newton_small.cu -- the products of a Newton-Schulz iteration on small matrices.
//
// An iteration is a chain of some 16 products, each needing the one before, so with
// few tiles its time is the latency of one product 16 times over.  Tiles here are
// 128 x 128 or, on twice as many SMs, 128 x 64, on one CTA (tcgen05.mma.cta_group::1), one or
// two CTAs per SM, finished by eight warps straight from the accumulator.  Where few tiles have a long K range, it
// is split over a cluster of up to 8 CTAs, whose partial tiles are added through
// distributed shared memory in K order, each CTA finishing a share of the tile's
// rows.  Symmetric results: as in newton_pair.cu only the tiles on and above the diagonal
// are computed, and a CTA writes its share of them to the mirrored place too, turned over
// in shared memory; on the diagonal tiles the elements above the diagonal go to both
// places, so results are symmetric to the last bit.
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
#include "rowvec.cuh"
#include "tc_tile.cuh"
#include "tmap.cuh"

namespace dg {
namespace {

template <int LAYOUT, int TN>  // tiles of 128 x TN
struct Cfg {
  static constexpr bool kAT = LAYOUT == 2, kBT = LAYOUT == 1;
  static constexpr int T = 128, BK = 64, UMMA_K = 16;
  static constexpr int BOX = 64;  // elements in one 128-byte swizzle row
  static constexpr int TILE_BYTES = T * 128, STAGE_BYTES = TILE_BYTES + TN * 128;
  static constexpr int MAX_STAGES = 8;
  static constexpr int PIECES = TN / 64;  // of 32 x 32, a warp's
  static constexpr int BOX_BYTES = BK * 128;  // of an MN-major operand
  static constexpr int THREADS = 256;
  static constexpr int PARKED_BYTES = T * T * 4, TURN_PITCH = T + 8;  // the fp16 rows of a share
  // the parked tile, or the pieces of the epilogue, take the stages' place
  static constexpr int MIN_AREA = PARKED_BYTES + T * TURN_PITCH * 2;
  static constexpr int WARPS = THREADS / 32;
  static constexpr int NUM_BARS = 2 * MAX_STAGES + 2 + WARPS;  // full, empty, accf, stall, inputs
  static constexpr int TAIL_BYTES = NUM_BARS * 8 + 16 + 1024;
  static_assert(2 * (MIN_AREA + TAIL_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
  [[maybe_unused]] static constexpr uint32_t MN_LAYOUT = 2u, MN_SBO = 1024u;
  static constexpr uint32_t IDESC = (1u << 4) | ((kAT ? 1u : 0u) << 15) | ((kBT ? 0u : 1u) << 16) |
                                    ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(T >> 4) << 24);
};

constexpr int kMaxSplits = 8;
constexpr int kInputsAhead = 4;  // vectors of in0 that a thread reads during the main loop: all of its share

// Site codes of the bounded waits.
enum : int {
  kSite8ProducerEmpty = 0x91,
  kSite8ProducerDrain = 0x92,
  kSite8MmaFull = 0x93,
  kSite8MmaDrain = 0x94,
  kSite8DrainAccFull = 0x95,
  kSite8EpiWait = 0x97,
  kSite8TestStall = 0x96,  // DGEMM_TC_TEST_STALL: the MMA warp's test wait ran out
};

struct Maps {
  CUtensorMap a, a2, b, b2;  // a2: of A2, or of A_lo; b2: of B_lo
  CUtensorMap o[2], in;  // 32 x 32 boxes
};

// Pieces of 32 x 32 elements in shared memory as TMA lays them out: 16-byte part q of
// row r at q ^ swizzle (64-byte rows in 64-byte swizzle, 128-byte rows in 128).
template <class O>
struct Piece {
  static constexpr int ROW = 32 * (int)sizeof(O), PARTS = ROW / 16, BYTES = 32 * ROW;
  static constexpr CUtensorMapSwizzle SWIZZLE =
      sizeof(O) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  static __device__ __forceinline__ int part(int r, int q) {
    return r * ROW + ((q ^ (sizeof(O) == 2 ? (r >> 1) & 3 : r & 7)) << 4);
  }
  static __device__ __forceinline__ int at(int r, int c) {
    const int b = c * (int)sizeof(O);
    return part(r, b >> 4) + (b & 15);
  }
};

// Tiles on and above the diagonal of a symmetric result.
template <int TN>
__host__ __device__ __forceinline__ int upper_tiles(int M, int tiles_n) {
  const int tiles_m = (M + 127) / 128;
  return tiles_m * tiles_n - 128 / TN * (tiles_m * (tiles_m - 1) / 2);
}

struct Args {
  int M, N, K;
  int splits, products, stall, stages, area;
  int lo;             // B_lo (1), A_lo (2)
  int o_tma, in_tma;  // without a K split: outputs may be written, in0 may be read by TMA
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

// Eight neighbouring elements of a row, from column `cols` on zero / not written.
template <class O, bool AL>
__device__ __forceinline__ void load8(const O *row, int col, int cols, float (&f)[8]) {
  if constexpr (sizeof(O) == 2) {
    widen16<O>(load_row16<O, AL>(row, col, cols), f);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      widen16<O>(load_row16<O, AL>(row, col + 4 * h, cols), f + 4 * h);
  }
}

template <class O, int LAYOUT, int TN, bool SYM, bool SPLIT, bool AL>
__global__ void __launch_bounds__(Cfg<LAYOUT, TN>::THREADS, 2)
    newton_small_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  using G = Cfg<LAYOUT, TN>;
  static_assert(!SPLIT || TN == G::T, "a K split is of square tiles");
  constexpr bool kAT = G::kAT, kBT = G::kBT;
  pdl_launch_dependents();
  const int splits = SPLIT ? p.splits : 1;
  const int part = SPLIT ? blockIdx.x % splits : 0;
  int tile = SPLIT ? blockIdx.x / splits : blockIdx.x;
  const int tiles_n = (p.N + TN - 1) / TN;
  int o = 0, tm, tn;
  if constexpr (SYM) {  // row by row on and above the diagonal
    constexpr int STEP = G::T / TN;
    const int tiles1 = upper_tiles<TN>(p.M, tiles_n);
    if (tile >= tiles1) o = 1, tile -= tiles1;
    tm = 0;
    while (tile >= tiles_n - STEP * tm) tile -= tiles_n - STEP * tm++;
    tn = STEP * tm + tile;
  } else {
    tm = tile / tiles_n, tn = tile % tiles_n;
  }
  const int m0 = tm * G::T, n0 = tn * TN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_base);
  const uint32_t bars = base + (uint32_t)p.area;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (G::MAX_STAGES + s); };
  const uint32_t accf_bar = bars + 8u * (2 * G::MAX_STAGES);
  const uint32_t stall_bar = bars + 8u * (2 * G::MAX_STAGES + 1);  // nothing ever arrives here
  auto in_bar = [&](int w) { return bars + 8u * (2 * G::MAX_STAGES + 2 + w); };
  uint8_t *tail = smem + p.area + 8 * G::NUM_BARS;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + 4);
  auto a_tile = [&](int s) { return base + (uint32_t)(s * G::STAGE_BYTES); };
  auto b_tile = [&](int s) { return base + (uint32_t)(s * G::STAGE_BYTES + G::TILE_BYTES); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kblocks1 = (p.K + G::BK - 1) / G::BK, kblocks = kblocks1 * terms_of(p.lo);
  const int per = (kblocks + splits - 1) / splits;
  const int kb_begin = min(kblocks, part * per), blocks = min(kblocks, part * per + per) - kb_begin;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accf_bar, 1);
    mbar_init(stall_bar, 1);
    for (int w = 0; w < G::WARPS; ++w) mbar_init(in_bar(w), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(o ? &maps.a2 : &maps.a);
    tma_prefetch_desc(&maps.b);
    if (!SPLIT && p.o_tma) tma_prefetch_desc(&maps.o[o]);
    if (!SPLIT && p.in_tma) tma_prefetch_desc(&maps.in);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), TN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // set-up done; the previous kernel on the stream has completed

  // Without a K split a warp finishes one or two pieces of 32 x 32: rows of its quarter of the
  // tensor memory's lanes, columns of one half of the tile.  Those of in0 are sent
  // for now.  (A thread has a row of a piece; global memory is left to TMA, for whose
  // loads and stores the rows need not be neighbours: with the threads' own, 1024^2 took
  // 12 us a product.)
  using P = Piece<O>;
  const bool has_in0 = p.in0 != nullptr && o == 0;
  const O *in0 = static_cast<const O *>(p.in0);
  const int quarter = warp & 3, r_first = m0 + quarter * 32;
  auto piece_col = [&](int h) { return n0 + (TN / 2) * (warp >> 2) + 32 * h; };
  // pieces below the diagonal come from those above it
  auto wanted = [&](int h) { return r_first < p.M && piece_col(h) < p.N && (!SYM || piece_col(h) >= r_first); };
  const uint32_t in_buf = base + (uint32_t)(p.stages * G::STAGE_BYTES + warp * G::PIECES * P::BYTES);
  int in_sent = 0;
  if (!SPLIT && has_in0 && p.in_tma) {
    for (int h = 0; h < G::PIECES; ++h) in_sent += wanted(h) ? 1 : 0;
    if (lane == 0 && in_sent > 0) {
      mbar_arrive_expect_tx(in_bar(warp), (uint32_t)(in_sent * P::BYTES));
      for (int h = 0; h < G::PIECES; ++h)
        if (wanted(h)) tma_load_2d(in_buf + (uint32_t)(h * P::BYTES), &maps.in, in_bar(warp), piece_col(h), r_first);
    }
    __syncwarp();
  }

  // With a K split, this CTA's share of the tile: rows [part R, part R + R), 16 threads
  // per row.
  const int R = G::T / splits, r_begin = part * R;
  const int c = 8 * (threadIdx.x & 15), col = n0 + c;
  float ahead[kInputsAhead][8];
  auto fetch = [&](int r, float (&f)[8]) {
    const int64_t row = m0 + r_begin + r;
    load8<O, AL>(in0 + row * p.ldi0, col, r < R && row < p.M ? p.N : 0, f);
  };
  if (SPLIT && warp != 0 && has_in0) {
#pragma unroll
    for (int k = 0; k < kInputsAhead; ++k) fetch(k * 16 + (threadIdx.x >> 4), ahead[k]);
  }

  bool all_sent = false;  // this thread is the producer and has sent for every stage
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int issued = 0, s = 0;
      uint32_t phase = 1;  // a fresh barrier's phase before is complete
      bool ok = true;
      for (int i = 0; i < blocks; ++i) {
        if (!mbar_try_wait(empty_bar(s), phase) && (*abort_flag || !mbar_wait(empty_bar(s), phase))) {
          if (!*abort_flag) watchdog_trip(p.watchdog, kSite8ProducerEmpty, abort_flag);
          ok = false;
          break;
        }
        const TermBlock at = term_block(kb_begin + i, kblocks1, p.lo);
        const CUtensorMap *map_a = o || at.a_lo ? &maps.a2 : &maps.a, *map_b = at.b_lo ? &maps.b2 : &maps.b;
        const int k0 = at.k * G::BK;
        const uint32_t fb = full_bar(s);
        if (kAT) {  // MN-major: 64 rows of the result x 64 k per box
          for (int j = 0; j < 2; ++j)
            tma_load_2d(a_tile(s) + j * G::BOX_BYTES, map_a, fb, m0 + j * G::BOX, k0);
        } else {
          tma_load_2d(a_tile(s), map_a, fb, k0, m0);
        }
        if (!kBT) {
          for (int j = 0; j < TN / G::BOX; ++j)
            tma_load_2d(b_tile(s) + j * G::BOX_BYTES, map_b, fb, n0 + j * G::BOX, k0);
        } else {
          tma_load_2d(b_tile(s), map_b, fb, k0, n0);
        }
        mbar_arrive_expect_tx(fb, G::STAGE_BYTES);  // announced after the copies are issued
        ++issued;
        if (++s == p.stages) s = 0, phase ^= 1u;
      }
      all_sent = ok;
      if (!ok) {  // no TMA write lands after this CTA has left
        for (int i = max(0, issued - p.stages); i < issued; ++i)
          if (!mbar_wait(full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u))
            atomicCAS(p.watchdog, 0, kSite8ProducerDrain);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    // (the whole warp in the loop, one elected lane issues from uniform registers)
    bool ok = true;
    if (p.stall && blockIdx.x == 0) {  // test hook: a wait that runs out
      if (!mbar_wait(stall_bar, 0) && lane == 0) watchdog_trip(p.watchdog, kSite8TestStall, abort_flag);
      ok = false;
    }
    int s = 0;
    uint32_t phase = 0;
    for (int i = 0; i < blocks && ok; ++i) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(full_bar(s), phase))) {
        ok = !*abort_flag && mbar_wait(full_bar(s), phase);
        if (!ok && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite8MmaFull, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < G::BK / G::UMMA_K; ++k)
          umma_f16(tmem_base, operand_desc<G, kAT>(a_tile(s), k, G::BOX_BYTES),
                   operand_desc<G, !kBT>(b_tile(s), k, G::BOX_BYTES), G::IDESC, (i > 0 || k > 0) ? 1u : 0u);
        umma_commit(empty_bar(s));
      }
      __syncwarp();
      if (++s == p.stages) s = 0, phase ^= 1u;
    }
    if (elect_one()) umma_commit(accf_bar);  // every MMA issued above has completed
    __syncwarp();
    if (!mbar_wait(accf_bar, 0)) atomicCAS(p.watchdog, 0, kSite8MmaDrain);
  } else if (SPLIT && warp < 6) {
    // ------------------------------- drain: partial tile to shared memory
    const int quarter = warp & 3;
    const bool ok = !*abort_flag && mbar_wait(accf_bar, 0);
    if (!ok && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite8DrainAccFull, abort_flag);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      // Every MMA has completed, so the stage area is idle: row r's 16-byte pieces at
      // c ^ (r & 7), or the lanes, which hold rows, would all write to the same banks
      const int r = quarter * 32 + lane;
      uint8_t *row = smem + r * G::T * 4;
      const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < G::T; c0 += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(t_row + (uint32_t)c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 x = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          *reinterpret_cast<uint4 *>(row + (((c0 / 4 + q) ^ (r & 7)) << 4)) =
              blocks > 0 ? x : make_uint4(0u, 0u, 0u, 0u);
        }
      }
      tc_fence_before();
    }
  }
  if (SPLIT && warp == 0) {
    __syncwarp();
    if (has_in0) {
#pragma unroll
      for (int k = 0; k < kInputsAhead; ++k) fetch(k * 16 + (threadIdx.x >> 4), ahead[k]);
    }
  }

  float alpha = p.alpha;
  if (p.factor != nullptr) {
    const float f = *p.factor;
    for (int i = 0; i < p.power; ++i) alpha *= f;
  }
  O *out = static_cast<O *>(p.out[o]);
  const bool diagonal = SYM && tm == tn;
  // ------------------------------ without a K split: from the accumulator
  if constexpr (!SPLIT) {
    __syncwarp();
    bool ok = true;
    auto wait = [&](uint32_t bar) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(bar, 0))) {
        const bool got = !*abort_flag && mbar_wait(bar, 0);
        if (!got && lane == 0 && !*abort_flag) watchdog_trip(p.watchdog, kSite8EpiWait, abort_flag);
        ok = __all_sync(0xffffffffu, got);
      }
    };
    if (has_in0 && !p.in_tma) {  // a row of a piece per instruction
#pragma unroll 1
      for (int h = 0; h < G::PIECES; ++h) {
        if (!wanted(h)) continue;
        const int64_t c0 = piece_col(h) + lane;
        const O *src = in0 + (int64_t)r_first * p.ldi0 + c0;
        const int rows = c0 < p.N ? p.M - r_first : 0;
        uint8_t *dst = smem + (in_buf - base) + h * P::BYTES;
        O x[32];  // all in flight
#pragma unroll
        for (int r = 0; r < 32; ++r) x[r] = r < rows ? src[r * p.ldi0] : from_f32<O>(0.f);
#pragma unroll
        for (int r = 0; r < 32; ++r) *reinterpret_cast<O *>(dst + P::at(r, lane)) = x[r];
      }
      __syncwarp();
    }
    // the stages are done with: a piece for every result, and for its mirrored place
    uint8_t *buf = smem + warp * G::PIECES * (SYM ? 2 : 1) * P::BYTES;
    // A staged piece to rows row0.. and columns col0.. of the result
    auto send = [&](const uint8_t *piece, int row0, int col0) {
      const int valid = min(32, p.out_cols - col0);
      // TMA writes whole 16-byte granules: a piece that ends inside one goes out
      // element by element
      if (p.o_tma && (valid == 32 || p.out_cols * (int)sizeof(O) % 16 == 0)) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_2d(&maps.o[o], smem_u32(piece), col0, row0);
      } else {
        __syncwarp();
        O *dst = out + (int64_t)row0 * p.ldo + col0 + lane;
        const int rows = lane < valid ? p.M - row0 : 0;
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
          if (r < rows) dst[r * p.ldo] = *reinterpret_cast<const O *>(piece + P::at(r, lane));
      }
    };
    if (in_sent > 0) wait(in_bar(warp));
    if (ok) wait(accf_bar);
    ok = ok && !__any_sync(0xffffffffu, *abort_flag != 0);
    tc_fence_after();
#pragma unroll 1
    for (int h = 0; h < G::PIECES; ++h) {
      if (!ok || !wanted(h)) continue;  // the same for the whole warp
      const int col0 = piece_col(h);
      uint32_t x[32];
      tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(col0 - n0), x);
      tmem_wait_ld();
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = alpha * __uint_as_float(x[j]);
      if (has_in0) {
        const uint8_t *in = smem + (in_buf - base) + h * P::BYTES;
#pragma unroll
        for (int q = 0; q < P::PARTS; ++q) {
          float f[kVec<O>];
          widen16<O>(*reinterpret_cast<const uint4 *>(in + P::part(lane, q)), f);
#pragma unroll
          for (int j = 0; j < kVec<O>; ++j) v[kVec<O> * q + j] += p.beta * f[j];
        }
      }
      const bool cross = SYM && col0 == r_first;
      if (cross && o == 0) add_diagonal(v, lane, p.gamma);
      if constexpr (SYM) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack2<O>(v[2 * j], v[2 * j + 1]);
        const uint32_t turned = smem_u32(buf) + P::BYTES;
        piece_store_turned(turned, lane, w);
        if (cross) piece_mirror(turned, lane, w);
        piece_store_row(smem_u32(buf), lane, w);
        send(buf, r_first, col0);
        if (!cross) send(buf + P::BYTES, col0, r_first);
      } else {
#pragma unroll
        for (int q = 0; q < P::PARTS; ++q)
          *reinterpret_cast<uint4 *>(buf + P::part(lane, q)) = narrow16<O>(v + kVec<O> * q);
        send(buf, r_first, col0);
      }
      buf += (SYM ? 2 : 1) * P::BYTES;
    }
    if (lane == 0) {
      bulk_commit_group();
      bulk_wait_group<0>();  // every TMA store of this warp complete
      if (!ok && in_sent > 0) mbar_wait(in_bar(warp), 0);  // after an abort: its input has landed
    }
    __syncwarp();
    tc_fence_before();
  }

  // ------------------------------------------ join the parts, finish, store
  // Every thread of every CTA of the cluster gets here, also after a bounded
  // wait gave up.
  __syncthreads();
  bool aborted = false;
  uint32_t at[kMaxSplits];
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) at[s] = s < splits ? mapa_shared(base, (uint32_t)s) : 0u;
    const uint32_t flag = smem_u32(const_cast<int *>(abort_flag)) - base;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
      if (s < splits) aborted |= ld_cluster_s32(at[s] + flag) != 0;
  } else {
    aborted = *abort_flag != 0;
  }
  if (SPLIT && !aborted) {  // the same for the whole cluster
    __half *turn = reinterpret_cast<__half *>(smem + G::PARKED_BYTES);
#pragma unroll 1
    for (int r0 = 0; r0 < R; r0 += 16) {
      const int r = r0 + (threadIdx.x >> 4), tr = r_begin + r;  // of the share, of the tile
      const int64_t row = m0 + tr;
      const bool in = row < p.M && col < p.out_cols;
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t off = (uint32_t)(tr * G::T * 4 + (((c / 4 + h) ^ (tr & 7)) << 4));
        float4 x;
        float4 y[kMaxSplits];
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s)
          if (s < splits) y[s] = ld_cluster_f4(at[s] + off);
        x = y[0];
#pragma unroll
        for (int s = 1; s < kMaxSplits; ++s)  // parts added in K order
          if (s < splits) x.x += y[s].x, x.y += y[s].y, x.z += y[s].z, x.w += y[s].w;
        v[4 * h] = alpha * x.x, v[4 * h + 1] = alpha * x.y;
        v[4 * h + 2] = alpha * x.z, v[4 * h + 3] = alpha * x.w;
      }
      if (has_in0) {
        static_assert(G::T / 2 <= 16 * kInputsAhead, "a share of half a tile's rows or fewer is all ahead");
        float f[8];
#pragma unroll
        for (int k = 0; k < kInputsAhead; ++k)
          if (r0 == 16 * k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = ahead[k][j];
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += p.beta * f[j];
      }
      if (SYM && diagonal && o == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(p.gamma, c + j == tr ? 1.f : 0.f, v[j]);
      }
      if constexpr (sizeof(O) == 2) {
        const uint4 w[1] = {narrow16<O>(v)};
        if (SYM) *reinterpret_cast<uint4 *>(turn + r * G::TURN_PITCH + c) = w[0];
        if (!diagonal || c >= tr) {  // on the diagonal tile: whole vectors above the diagonal
          if constexpr (SYM) {
            if (in) *reinterpret_cast<uint4 *>(out + row * p.ldo + col) = w[0];
          }
        } else if (c + 8 > tr) {  // the vector that the diagonal crosses
          if (in)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j >= tr) out[row * p.ldo + col + j] = from_f32<O>(v[j]);
        }
        if constexpr (!SYM) store_row16<O, AL, 1, 16>(out + row * p.ldo, in ? col : p.out_cols, p.out_cols, w);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          O *to = out + row * p.ldo + col + 4 * h;
          if (AL && in && col + 4 * h + 4 <= p.out_cols) {
            *reinterpret_cast<uint4 *>(to) = narrow16<O>(v + 4 * h);
          } else if (in) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (col + 4 * h + j < p.out_cols) to[j] = from_f32<O>(v[4 * h + j]);
          }
        }
      }
    }
    if constexpr (SYM) {  // the share once more, column j of it as row n0 + j
      __syncthreads();
      const int chunks = R / 8;
      for (int e = threadIdx.x; e < G::T * chunks; e += G::THREADS) {
        const int j = e % G::T, r = 8 * (e / G::T), tr = r_begin + r;
        const int64_t row = n0 + j;
        const int to = m0 + tr;  // its first column there
        if (row >= p.M || to >= p.out_cols) continue;
        uint32_t w[4];
        const uint16_t *t = reinterpret_cast<const uint16_t *>(turn) + r * G::TURN_PITCH + j;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = (uint32_t)t[2 * q * G::TURN_PITCH] | (uint32_t)t[(2 * q + 1) * G::TURN_PITCH] << 16;
        O *dst = out + row * p.ldo + to;
        if (!diagonal || tr + 7 < j) {
          *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (tr < j) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (tr + q < j) reinterpret_cast<uint16_t *>(dst)[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
        }
      }
    }
  }
  if (aborted && all_sent) {  // no TMA write lands after this CTA has left
    for (int i = max(0, blocks - p.stages); i < blocks; ++i)
      if (!mbar_wait(full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u))
        atomicCAS(p.watchdog, 0, kSite8ProducerDrain);
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
    tmem_dealloc(tmem_base, TN);
  }
}

// ------------------------------------------------------------- host side
template <class O>
constexpr CUtensorMapDataType map_type() {
  return sizeof(O) == 4                       ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : std::is_same<O, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <auto KERNEL, int MOST, int THREADS>
cudaError_t launch_one(unsigned grid, size_t smem, cudaStream_t stream, unsigned cluster, const Maps &maps,
                       const Args &a) {
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  e = launch_kernel(KERNEL, dim3(grid), dim3(THREADS), smem, stream, cluster, maps, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class O, int LAYOUT, int TN, bool SYM>
cudaError_t launch(const NewtonGemm &p, int splits, int num_sms, int *watchdog, cudaStream_t stream) {
  using G = Cfg<LAYOUT, TN>;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  Args a;
  memset(&a, 0, sizeof a);
  const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  auto map_a = [&](CUtensorMap *map, const void *A) {
    return G::kAT ? make_map(map, A, dt, 2, p.K, p.M, p.lda, G::BOX, G::BK, swz)
                  : make_map(map, A, dt, 2, p.M, p.K, p.lda, G::BOX, G::T, swz);
  };
  auto map_b = [&](CUtensorMap *map, const void *B) {
    return G::kBT ? make_map(map, B, dt, 2, p.N, p.K, p.ldb, G::BOX, TN, swz)
                  : make_map(map, B, dt, 2, p.K, p.N, p.ldb, G::BOX, G::BK, swz);
  };
  bool ok = map_a(&maps.a, p.A) && map_b(&maps.b, p.B);
  if (p.A2 != nullptr) ok = ok && SYM && p.A_lo == nullptr && p.B_lo == nullptr && map_a(&maps.a2, p.A2);
  if (p.A_lo != nullptr) ok = ok && map_a(&maps.a2, p.A_lo);
  if (p.B_lo != nullptr) ok = ok && map_b(&maps.b2, p.B_lo);
  a.lo = (p.B_lo != nullptr ? 1 : 0) | (p.A_lo != nullptr ? 2 : 0);
  // symmetric results are workspaces: rows of whole vectors
  const bool out_al = rows_aligned(p.out, p.ldo, sizeof(O)) && rows_aligned(p.out2, p.ldo, sizeof(O));
  if (!ok || p.K < 1 || (SYM && (p.M != p.N || !out_al || p.out_cols % 8 != 0)) ||
      (splits != 1 && (TN != G::T || (splits != 2 && splits != 4 && splits != 8))))
    return cudaErrorInvalidValue;
  a.M = p.M, a.N = p.N, a.K = p.K;
  a.splits = splits, a.products = p.A2 != nullptr ? 2 : 1;
  a.stall = test_stall();
  a.alpha = p.alpha, a.beta = p.beta, a.gamma = p.gamma;
  a.factor = p.factor, a.power = p.power;
  a.in0 = p.in0, a.ldi0 = p.ldi0;
  a.out[0] = p.out, a.out[1] = p.out2;
  a.ldo = p.ldo, a.out_cols = (int)p.out_cols;
  a.watchdog = watchdog;
  const int64_t tm = (p.M + G::T - 1) / G::T, tn = (p.N + TN - 1) / TN;
  if (tm * tn > 0x1fffffff) return cudaErrorInvalidValue;
  const int64_t tiles = SYM ? (int64_t)a.products * upper_tiles<TN>(p.M, (int)tn) : tm * tn;
  if (tiles * splits > 0x3fffffff) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(tiles * splits), cluster = (unsigned)splits;
  // all of an SM's shared memory for one CTA's stages where that holds every CTA at once
  // (or where half of it is too little)
  const int in_bytes = splits == 1 && p.in0 != nullptr ? G::WARPS * G::PIECES * Piece<O>::BYTES : 0;
  // without a K split the results' pieces take the stages' place, with one the parked tile
  const int least = splits == 1 ? G::WARPS * G::PIECES * (SYM ? 2 : 1) * Piece<O>::BYTES : G::MIN_AREA;
  for (int half = grid > (unsigned)num_sms; half >= 0; --half) {
    const int budget = (half ? 113 * 1024 : 232448) - G::TAIL_BYTES;
    a.stages = (budget - in_bytes) / G::STAGE_BYTES;
    if (a.stages > G::MAX_STAGES) a.stages = G::MAX_STAGES;
    a.area = a.stages * G::STAGE_BYTES + in_bytes;
    if (splits > 1 && a.area < least) a.area = least;
    if (a.stages >= 2 && (splits > 1 || a.stages * G::STAGE_BYTES >= least)) break;
  }
  static_assert(2 * G::STAGE_BYTES >= G::WARPS * G::PIECES * 2 * Piece<__half>::BYTES && G::MIN_AREA + G::TAIL_BYTES <= 113 * 1024 &&
                    4 * G::STAGE_BYTES + G::WARPS * G::PIECES * Piece<O>::BYTES + G::TAIL_BYTES <= 232448,
                "what is least always fits");
  if (splits == 1) {
    a.o_tma = out_al;
    for (int i = 0; i < a.products && a.o_tma; ++i)
      a.o_tma = make_map(&maps.o[i], a.out[i], map_type<O>(), sizeof(O), p.M, p.out_cols, p.ldo, 32, 32,
                         Piece<O>::SWIZZLE);
    a.in_tma = p.in0 != nullptr && rows_aligned(p.in0, p.ldi0, sizeof(O)) &&
               make_map(&maps.in, p.in0, map_type<O>(), sizeof(O), p.M, p.N, p.ldi0, 32, 32, Piece<O>::SWIZZLE);
  }
  const size_t smem = (size_t)(a.area + G::TAIL_BYTES);
  constexpr int B = 232448, T = G::THREADS;
  const bool al = SYM || (p.out_cols % (16 / (int)sizeof(O)) == 0 && out_al &&
                          (p.in0 == nullptr || rows_aligned(p.in0, p.ldi0, sizeof(O))));
  if constexpr (TN == G::T) {
    if (splits > 1) {
      if constexpr (SYM)
        return launch_one<newton_small_kernel<O, LAYOUT, TN, true, true, true>, B, T>(grid, smem, stream, cluster, maps, a);
      else
        return al ? launch_one<newton_small_kernel<O, LAYOUT, TN, false, true, true>, B, T>(grid, smem, stream, cluster, maps, a)
                  : launch_one<newton_small_kernel<O, LAYOUT, TN, false, true, false>, B, T>(grid, smem, stream, cluster, maps, a);
    }
  }
  return launch_one<newton_small_kernel<O, LAYOUT, TN, SYM, false, true>, B, T>(grid, smem, stream, 1u, maps, a);
}

template <class O, int LAYOUT, bool SYM>
cudaError_t launch_wide(const NewtonGemm &p, int tn, int splits, int num_sms, int *watchdog, cudaStream_t stream) {
  return tn == 64 ? launch<O, LAYOUT, 64, SYM>(p, splits, num_sms, watchdog, stream)
                  : launch<O, LAYOUT, 128, SYM>(p, splits, num_sms, watchdog, stream);
}
template <class O>
cudaError_t launch_plain(const NewtonGemm &p, int tn, int splits, int num_sms, int *watchdog, cudaStream_t stream) {
  return p.layout == 0 ? launch_wide<O, 0, false>(p, tn, splits, num_sms, watchdog, stream)
                       : launch_wide<O, 1, false>(p, tn, splits, num_sms, watchdog, stream);
}

}  // namespace

cudaError_t launch_newton_small(const NewtonGemm &p, int tn, int splits, int num_sms, int *watchdog,
                                cudaStream_t stream) {
  if (p.symmetric) {
    if (p.dtype != DGEMM_DTYPE_F16 || p.layout == 0) return cudaErrorInvalidValue;
    return p.layout == 1 ? launch_wide<__half, 1, true>(p, tn, splits, num_sms, watchdog, stream)
                         : launch_wide<__half, 2, true>(p, tn, splits, num_sms, watchdog, stream);
  }
  if (p.layout == 2) return cudaErrorInvalidValue;
  switch (p.dtype) {
    case DGEMM_DTYPE_F32: return launch_plain<float>(p, tn, splits, num_sms, watchdog, stream);
    case DGEMM_DTYPE_BF16: return launch_plain<__nv_bfloat16>(p, tn, splits, num_sms, watchdog, stream);
    default: return launch_plain<__half>(p, tn, splits, num_sms, watchdog, stream);
  }
}

}  // namespace dg
