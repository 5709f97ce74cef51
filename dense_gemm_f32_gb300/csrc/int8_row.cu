// int8_row.cu -- products with 8-bit weights for one to four tokens, in one launch.
//
// Bound by reading the weights once, and then by latency: no tensor cores, no
// stages, no tokens written by a kernel before.  A warp takes a row of weights (or,
// for long rows, 2, 4 or 8 warps take a part each), 16 bytes per lane and load, all
// loads of a row and those of the next in flight; the products with the tokens are
// dp4a, four at a time, into 32-bit integers, which hold any sum exactly; the
// warps' sums are kept in shared memory and finished together, a thread per output.
//  * The tokens are quantised by every block for itself (quant.cuh), from L2, while
//    its first rows are on their way.
//  * Rows on any alignment: a lane's aligned 16 bytes are put together with its
//    neighbour's, so weights need no copy.
//  * One token, 4096 -> 14336: 13.3 us (floor 8.8), 15.6 by a tokens' kernel and
//    int8_small.cu; 1000 -> 1000 4.2 and 8.8; four tokens, 4096 -> 14336, 18.9 and 16.4: a
//    token costs every weight another dp4a, so int8_use_row weighs both.
//  * The product after another of this kind (the gated block's second) sends for its
//    weights before the first is done, which signals after its own wait.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "int8.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "quant.cuh"
#include "rowvec.cuh"

namespace dg {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;  // one block per SM
constexpr int kMaxVecs = 8;    // 16-byte loads of a lane for its part of a row
constexpr int kMaxTokens = 4;
constexpr int kChunk = 1024;   // parts of rows whose sums are kept before they are finished

struct Args {
  int M, N, K;
  int act, parts, vecs;  // warps per row, loads per lane
  int early;             // the weights may be read before the kernel ahead is done
  int x_aligned;         // rows of X are, and whole vectors
  int pitch;             // bytes of a token in shared memory
  const void *X;         // the tokens, of type `x_type`, or integers with x_scale
  int64_t ldx;
  const float *x_scale;
  const uint8_t *W, *W2;
  int64_t ldw, ldw2;
  const float *w_scale, *w2_scale;
  const void *bias, *in0;
  int64_t ldi0;
  void *out;
  int64_t ldo;
};

// f(column, elements) for this thread's vectors of a row, four of them in flight.
template <class X, bool AL, class F>
__device__ __forceinline__ void for_vectors(const X *x, int cols, int end, F &&f) {
  constexpr int V = kVec<X>, AHEAD = 4;
  for (int c0 = threadIdx.x * V; c0 < end; c0 += AHEAD * kThreads * V) {
    RowBlocks b[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) b[k] = fetch_row16<X, AL>(x, c0 + k * kThreads * V, cols);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int c = c0 + k * kThreads * V;
      if (c >= end) break;
      float v[V];
      widen16<X>(take_row16<X, AL>(b[k], x, c, cols), v);
      f(c, v);
    }
  }
}

// Rows of tokens in 8 bits in shared memory, zeros behind them; their scales.  Their
// largest first (before the weights are sent for, or the tokens' few bytes come after
// those), then the integers.  A single token on aligned rows is held in between.
template <class X, int MT>
struct Tokens {
  static constexpr int V = kVec<X>, HELD = 8;
  RowBlocks held[HELD];

  __device__ __forceinline__ bool holds(const Args &p) const {
    return MT == 1 && p.x_aligned && p.K <= HELD * kThreads * V;
  }
  __device__ __forceinline__ void send(const Args &p) {
    if (holds(p)) {
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        held[k] = fetch_row16<X, true>(static_cast<const X *>(p.X), min((int)(threadIdx.x + k * kThreads) * V, p.K), p.K);
    }
  }
  __device__ __forceinline__ void largest(const Args &p, uint32_t *tops) {
    for (int m = 0; m < MT; ++m) {
      const X *x = static_cast<const X *>(p.X) + m * p.ldx;
      const int cols = m < p.M ? p.K : 0;
      uint32_t top = 0;
      auto widest = [&](int, const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) top = max(top, abs_bits(v[j]));
      };
      if (holds(p)) {
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
          float v[V];
          widen16<X>(held[k].a, v);  // zeros past the row
          widest(0, v);
        }
      } else if (p.x_aligned) {
        for_vectors<X, true>(x, cols, cols, widest);
      } else {
        for_vectors<X, false>(x, cols, cols, widest);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if ((threadIdx.x & 31) == 0) tops[m * kWarps + (threadIdx.x >> 5)] = top;
    }
  }
  __device__ __forceinline__ void quantise(const Args &p, int8_t *tokens, float *scales, const uint32_t *tops) {
    for (int m = 0; m < MT; ++m) {
      const X *x = static_cast<const X *>(p.X) + m * p.ldx;
      const int cols = m < p.M ? p.K : 0;
      const RowScale r = row_scale(
          __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < kWarps ? tops[m * kWarps + (threadIdx.x & 31)] : 0u));
      if (threadIdx.x == 0) scales[m] = r.scale;
      int8_t *to = tokens + m * p.pitch;
      auto put_one = [&](int c, float (&v)[V]) {
        quantise_vec<V>(v, r);
        put<V>(to + c, v, V, true);
      };
      if (holds(p)) {
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
          const int c = (int)(threadIdx.x + k * kThreads) * V;
          if (c >= p.pitch) break;
          float v[V];
          widen16<X>(held[k].a, v);
          put_one(c, v);
        }
        // what no held vector covers is behind the row
        for (int c = HELD * kThreads * V + (int)threadIdx.x * 4; c < p.pitch; c += kThreads * 4)
          *reinterpret_cast<uint32_t *>(to + c) = 0u;
      } else if (p.x_aligned) {
        for_vectors<X, true>(x, cols, p.pitch, put_one);
      } else {
        for_vectors<X, false>(x, cols, p.pitch, put_one);
      }
    }
  }
};

// X: the tokens' type (int8_t: given as integers); T: the result's; GATED: H = act(g)
// u in fp32.  MT: tokens, 1, 2 or 4.  AL: rows of weights on 16-byte boundaries.
template <class X, class T, bool GATED, int MT, bool AL>
__global__ void __launch_bounds__(kThreads, 1) int8_row_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(16) uint8_t smem[];
  int8_t *tokens = reinterpret_cast<int8_t *>(smem);
  int *sums = reinterpret_cast<int *>(smem + MT * p.pitch);  // [row of the chunk][part][token]
  float *scales = reinterpret_cast<float *>(sums + kChunk * MT);
  uint32_t *tops = reinterpret_cast<uint32_t *>(scales + kMaxTokens);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % p.parts, group = warp / p.parts, groups = kWarps / p.parts;
  constexpr int MATS = GATED ? 2 : 1;
  // this block's features: first, first + step, ...; a group of warps takes every
  // groups-th of them, both matrices' rows in turn
  const int step = gridDim.x, mine = blockIdx.x < p.N ? (p.N - 1 - blockIdx.x) / step + 1 : 0;
  const int first_vec = part * p.vecs * 32 + lane;  // of the row, in 16 bytes
  const int row_vecs = (p.K + 15) / 16;

  struct Row {
    uint4 v[kMaxVecs + (AL ? 0 : 1)];
    int off;
  };
  auto load = [&](int task, Row &r) {  // task: 2 f + matrix, or f
    const int i = task / MATS;
    const bool in = i < mine;
    const int64_t f = blockIdx.x + (int64_t)(in ? i : 0) * step;
    const uint8_t *w = MATS == 2 && (task & 1) ? p.W2 + f * p.ldw2 : p.W + f * p.ldw;
    r.off = AL ? 0 : (int)(reinterpret_cast<uintptr_t>(w) & 15);
    const uint4 *block = reinterpret_cast<const uint4 *>(w - r.off);
    const int blocks = in ? (r.off + p.K + 15) / 16 : 0;
#pragma unroll
    for (int k = 0; k < kMaxVecs; ++k) {
      const int b = first_vec + k * 32;
      r.v[k] = k < p.vecs && b < blocks ? __ldcs(block + b) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (!AL) {  // lane 0 of the part behind, for the last lane
      const int b = (part + 1) * p.vecs * 32;
      r.v[kMaxVecs] = lane == 0 && b < blocks ? __ldcs(block + b) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  Row now, next;
  auto task_of = [&](int k) { return (k / MATS * groups + group) * MATS + k % MATS; };
  if (p.early) load(task_of(0), now);
  pdl_wait();
  pdl_launch_dependents();
  // this thread's first output of the finish below, for which it reads now what it needs
  auto feature_at = [&](int at) { return blockIdx.x + (int64_t)at * step; };
  struct Rest {
    float ws, ws2, bias, res;
  };
  auto rest_of = [&](int at, int m) {
    Rest r = {0.f, 0.f, 0.f, 0.f};
    if (at >= mine || m >= p.M) return r;
    const int64_t f = feature_at(at);
    r.ws = p.w_scale[f];
    if constexpr (GATED) {
      r.ws2 = p.w2_scale[f];
    } else {
      if (p.bias != nullptr) r.bias = to_f32<T>(static_cast<const T *>(p.bias)[f]);
      if (p.in0 != nullptr) r.res = to_f32<T>(static_cast<const T *>(p.in0)[m * p.ldi0 + f]);
    }
    return r;
  };
  const Rest first = rest_of(threadIdx.x / MT, threadIdx.x % MT);
  if constexpr (sizeof(X) == 1) {
    for (int m = 0; m < MT; ++m) {
      const int8_t *x = static_cast<const int8_t *>(p.X) + m * p.ldx;
      for (int c = threadIdx.x; c < p.pitch; c += kThreads)
        tokens[m * p.pitch + c] = m < p.M && c < p.K ? x[c] : (int8_t)0;
      if (threadIdx.x == 0) scales[m] = m < p.M ? p.x_scale[m] : 0.f;
    }
    if (!p.early) load(task_of(0), now);
  } else {
    Tokens<X, MT> t;
    t.send(p);
    if (!t.holds(p)) t.largest(p, tops);
    if (!p.early) load(task_of(0), now);
    if (t.holds(p)) t.largest(p, tops);
    __syncthreads();
    t.quantise(p, tokens, scales, tops);
  }
  load(task_of(1), next);
  __syncthreads();

  const int per_group = (mine + groups - 1) / groups * MATS;  // rounds of the longest group
  const int chunk = kChunk / (p.parts * groups * MATS) * MATS;  // rounds between flushes
  for (int k0 = 0; k0 < per_group; k0 += chunk) {
    const int k1 = min(per_group, k0 + chunk);
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      int acc[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = 0;
#pragma unroll
      for (int v = 0; v < kMaxVecs; ++v) {
        if (v >= p.vecs) break;
        uint32_t w[4] = {now.v[v].x, now.v[v].y, now.v[v].z, now.v[v].w};
        if constexpr (!AL) {
          // the neighbour's block; the last lane's is the first lane's of the next round
          const uint4 after = v + 1 < p.vecs ? now.v[v + 1 < kMaxVecs ? v + 1 : v] : now.v[kMaxVecs];
          const uint32_t own[4] = {lane == 0 ? after.x : w[0], lane == 0 ? after.y : w[1],
                                   lane == 0 ? after.z : w[2], lane == 0 ? after.w : w[3]};
          uint4 n;
          n.x = __shfl_sync(0xffffffffu, own[0], (lane + 1) & 31);
          n.y = __shfl_sync(0xffffffffu, own[1], (lane + 1) & 31);
          n.z = __shfl_sync(0xffffffffu, own[2], (lane + 1) & 31);
          n.w = __shfl_sync(0xffffffffu, own[3], (lane + 1) & 31);
          const uint4 s = shift16<uint8_t>(now.v[v], n, now.off);
          w[0] = s.x, w[1] = s.y, w[2] = s.z, w[3] = s.w;
        }
        const int b = first_vec + v * 32;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 t = *reinterpret_cast<const uint4 *>(tokens + m * p.pitch + min(b, row_vecs) * 16);
          acc[m] = __dp4a((int)w[0], (int)t.x, acc[m]);
          acc[m] = __dp4a((int)w[1], (int)t.y, acc[m]);
          acc[m] = __dp4a((int)w[2], (int)t.z, acc[m]);
          acc[m] = __dp4a((int)w[3], (int)t.w, acc[m]);
        }
      }
      now = next;
      load(task_of(k + 2), next);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = __reduce_add_sync(0xffffffffu, acc[m]);
      if (lane < MT) {
        int x = acc[0];
#pragma unroll
        for (int m = 1; m < MT; ++m) x = lane == m ? acc[m] : x;
        sums[(((k - k0) * groups + group) * p.parts + part) * MT + lane] = x;
      }
    }
    __syncthreads();
    // a thread per feature and token of the chunk
    const int features = (k1 - k0) / MATS * groups;
    for (int e = threadIdx.x; e < features * MT; e += kThreads) {
      const int m = e % MT, i = e / MT, round = i / groups, g = i % groups;
      const int at = k0 / MATS * groups + i;
      if (at >= mine || m >= p.M) continue;
      const int64_t f = feature_at(at);
      auto sum = [&](int mat) {
        int s = 0;  // any order gives the same integer
        for (int q = 0; q < p.parts; ++q)
          s += sums[(((round * MATS + mat) * groups + g) * p.parts + q) * MT + m];
        return (float)s;
      };
      const Rest r = e == (int)threadIdx.x && k0 == 0 ? first : rest_of(at, m);
      float z = scaled(sum(0), scales[m], r.ws) + r.bias;
      const float u = GATED ? scaled(sum(1), scales[m], r.ws2) : 0.f;
      with_act(p.act, [&](auto c) { z = act_f32<decltype(c)::value>(z); });
      if constexpr (GATED)
        static_cast<float *>(p.out)[m * p.ldo + f] = z * u;
      else
        static_cast<T *>(p.out)[m * p.ldo + f] = from_f32<T>(z + r.res);
    }
    __syncthreads();
  }
}

// Warps per row: the fewest whose lanes hold their parts in kMaxVecs loads.
int parts_of(int K) {
  int parts = 1;
  while (parts < kWarps && (K + 15) / 16 > parts * 32 * kMaxVecs) parts *= 2;
  return parts;
}

template <class X, class T, bool GATED, int MT, bool AL>
cudaError_t launch_one(const Args &a, int num_sms, cudaStream_t stream) {
  auto kern = int8_row_kernel<X, T, GATED, MT, AL>;
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 190 * 1024);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const size_t smem = (size_t)MT * a.pitch + kChunk * MT * 4 + kMaxTokens * 4 + kMaxTokens * kWarps * 4;
  // one block per SM, each with the same number of rounds where there are many
  const int groups = kWarps / a.parts, most = num_sms;
  int64_t grid = ((int64_t)a.N + groups - 1) / groups;
  if (grid > most) {
    const int64_t rounds = ((int64_t)a.N + (int64_t)most * groups - 1) / ((int64_t)most * groups);
    grid = ((int64_t)a.N + rounds * groups - 1) / (rounds * groups);
  }
  e = launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), smem, stream, 1u, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <class X, class T, bool GATED, int MT>
cudaError_t launch_mt(const Args &a, int num_sms, cudaStream_t stream) {
  const bool al = reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && a.ldw % 16 == 0 &&
                  (!GATED || (reinterpret_cast<uintptr_t>(a.W2) % 16 == 0 && a.ldw2 % 16 == 0));
  return al ? launch_one<X, T, GATED, MT, true>(a, num_sms, stream)
            : launch_one<X, T, GATED, MT, false>(a, num_sms, stream);
}

template <class X, class T, bool GATED>
cudaError_t launch_x(const Args &a, int num_sms, cudaStream_t stream) {
  if (a.M == 1) return launch_mt<X, T, GATED, 1>(a, num_sms, stream);
  return a.M == 2 ? launch_mt<X, T, GATED, 2>(a, num_sms, stream) : launch_mt<X, T, GATED, 4>(a, num_sms, stream);
}

}  // namespace

// Whether it can, and its time (microseconds, fitted like those of int8.cu): the
// weights', and for each token the shared memory's and the integer units'.
double int8_row_time(const Int8Gemm &p) {
  const bool aligned = rows_aligned(p.W, p.ldw, 1) && (!p.gated || rows_aligned(p.W2, p.ldw2, 1));
  const double weights = (double)p.N * p.K * (p.gated ? 2 : 1) / 6.6e6;
  return 2.8 + weights * (0.95 + 0.22 * p.M) * (aligned ? 1.0 : 1.8);
}

bool int8_row_takes(int M, int K) {
  const int64_t pitch = ((int64_t)K + 15) / 16 * 16 + 16;
  return M >= 1 && M <= kMaxTokens && K >= 1 && (K + 15) / 16 <= kWarps * 32 * kMaxVecs &&
         (M == 3 ? 4 : M) * pitch <= 160 * 1024;
}

cudaError_t launch_int8_row(const Int8Gemm &p, const void *X, int64_t ldx, int x_type, bool early, int num_sms,
                            cudaStream_t stream) {
  if (!int8_row_takes(p.M, p.K)) return cudaErrorInvalidValue;
  Args a = {};
  a.M = p.M, a.N = p.N, a.K = p.K, a.act = p.act;
  a.parts = parts_of(p.K);
  a.vecs = ((p.K + 15) / 16 + a.parts * 32 - 1) / (a.parts * 32);
  a.early = early;
  a.pitch = (p.K + 15) / 16 * 16 + 16;  // a vector of zeros behind
  a.X = X, a.ldx = ldx, a.x_scale = p.t_scale;
  const int xs = x_type == DGEMM_DTYPE_F32 ? 4 : 2;
  a.x_aligned = rows_aligned(X, ldx, xs) && p.K % (16 / xs) == 0;
  a.W = static_cast<const uint8_t *>(p.W), a.W2 = static_cast<const uint8_t *>(p.W2);
  a.ldw = p.ldw, a.ldw2 = p.ldw2, a.w_scale = p.w_scale, a.w2_scale = p.w2_scale;
  a.bias = p.bias, a.in0 = p.in0, a.ldi0 = p.ldi0, a.out = p.out, a.ldo = p.ldo;
  const bool half = p.dtype == DGEMM_DTYPE_F16;
  if (p.gated)  // H, from 16-bit tokens
    return half ? launch_x<__half, __half, true>(a, num_sms, stream)
                : launch_x<__nv_bfloat16, __nv_bfloat16, true>(a, num_sms, stream);
  if (p.t_scale != nullptr)  // integers
    return half ? launch_x<int8_t, __half, false>(a, num_sms, stream)
                : launch_x<int8_t, __nv_bfloat16, false>(a, num_sms, stream);
  if (x_type == DGEMM_DTYPE_F32)  // H
    return half ? launch_x<float, __half, false>(a, num_sms, stream)
                : launch_x<float, __nv_bfloat16, false>(a, num_sms, stream);
  return half ? launch_x<__half, __half, false>(a, num_sms, stream)
              : launch_x<__nv_bfloat16, __nv_bfloat16, false>(a, num_sms, stream);
}

}  // namespace dg
