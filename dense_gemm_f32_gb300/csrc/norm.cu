// norm.cu -- layer norm over the rows of a matrix, forward and backward.
//
//   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps)
//   y = (x - mu) rstd w + b
//   with xh = (x - mu) rstd and p = dy w:
//   dx = rstd (p - mean(p) - xh mean(p xh)) [+ dr]
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: forward one read and one write of the matrix, backward two
// (three) reads and one write.  A row is held in registers by the threads that
// share it, so it is read once and the variance is that of the centred values
// (two passes over registers).  What the SMs issue is the other bound: a row
// costs a thread about 190 instructions besides the 9 to 12 per element, so a
// thread takes 32 elements (16 in the backward pass, which has to hold column
// sums too) and a row as few threads as that leaves: a warp up to 1024
// elements, without a block barrier, then 64 to 512 threads.  The
// backward kernel is persistent: a ring of rows per block is filled ahead by
// bulk copies, and a thread keeps the same columns for every row, so the
// column sums of dw and db stay in its registers and each block writes one
// partial sum, which a second launch adds up in a fixed order.
//
// Not made fast: backward rows of 8193 to 16384 16-bit elements, whose 64 column
// sums per thread spill (4096 x 16384 bf16 149 us, its bytes 59); rows beyond 16384
// elements (backward: 32 KB), which go an element per load through one block per
// row, several passes from L2 and the column sums from both whole matrices once more
// (2048 x 32768 bf16 105 us forward, its bytes 40, 277 backward, 59; 4096 x 16384
// fp32 backward 269, 119); and backward with fewer rows than SMs, where each row
// writes its own fp32 partial sums (128 x 8192 bf16 22 us, its bytes 1).
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace dg {
namespace {

// A row's share of a thread: CH vectors.  GROUP threads share a row, each warp
// of them CH * 32 neighbouring vectors, 32 at a time; a block holds BLOCK /
// GROUP rows.  The share does not depend on the rows' alignment, so neither do the
// sums.
template <class T_, bool ALIGNED_, int CH_, int GROUP_>
struct Shape {
  using T = T_;
  static constexpr bool ALIGNED = ALIGNED_;
  static constexpr int V = kVec<T_>, CH = CH_, GROUP = GROUP_;
  static constexpr int BLOCK = GROUP == 32 ? 128 : GROUP, ROWS = BLOCK / GROUP;
  static constexpr int CAPACITY = GROUP * CH * V;
  // column of vector c of thread t of the group
  static __device__ __forceinline__ int col(int c, int t) {
    return ((t / 32 * CH + c) * 32 + t % 32) * V;
  }
  // backward: a row's values stay in registers between its two passes, else
  // they are read again from the ring
  static constexpr bool KEEP = CH * V <= 16;
  // backward: one block of 512 threads per SM, so that there are few partial
  // column sums to write and join (1000 x 1013 bf16: 22 us with blocks of 64
  // threads and eight per SM, 10.5 us)
  static constexpr int BWD_BLOCK = 512, BWD_ROWS = BWD_BLOCK / GROUP;
};

constexpr int kMaxStages = 8;

// Site code of the bounded wait for a row's copy.
enum : int { kSiteNormRow = 0xc1 };

// Sums of N values over the threads of a row; every thread gets them.  `red`
// alternates between two buffers, so one barrier per sum is enough (barrier 1 +
// sub, which only the row's threads use).
template <class S, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[32], int sub = 0) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (S::GROUP > 32) {
    constexpr int W = S::GROUP / 32;
    const int warp = threadIdx.x % S::GROUP >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i][warp] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "n"(S::GROUP) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = lane < W ? red[i][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (o < W) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[i] = __shfl_sync(0xffffffffu, s, 0);
    }
  }
}

template <class S>
__global__ void __launch_bounds__(S::BLOCK)
    ln_fwd_kernel(int rows, int cols, float inv, float eps, const typename S::T *X, int64_t ldx,
                  const typename S::T *w, const typename S::T *b, typename S::T *Y, int64_t ldy,
                  float *mean, float *rstd) {
  using T = typename S::T;
  constexpr int V = S::V, CH = S::CH, GROUP = S::GROUP;
  __shared__ float red[2][1][32];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % GROUP;
  const int64_t row = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / GROUP;
  if (GROUP == 32 && row >= rows) return;
  const T *x = X + row * ldx;
  float v[CH][V], s[1] = {0.f};
  RowBlocks raw[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) raw[c] = fetch_row16<T, S::ALIGNED>(x, S::col(c, t), cols);
#pragma unroll
  for (int c = 0; c < CH; ++c)
    widen16<T>(take_row16<T, S::ALIGNED>(raw[c], x, S::col(c, t), cols), v[c]);
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) s[0] += v[c][j];
  row_sum<S>(s, red[0]);
  const float mu = s[0] / cols;  // by 1 / cols a constant row's mean is not its value, and y not b
  s[0] = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[c][j] -= mu;
      if (S::col(c, t) + (S::ALIGNED ? 0 : j) < cols) s[0] += v[c][j] * v[c][j];
    }
  row_sum<S>(s, red[1]);
  const float r = rsqrtf(s[0] * inv + eps);
  uint4 out[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = S::col(c, t);
    float g[V], h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = 1.f, h[j] = 0.f;
    if (w) widen16<T>(load_row16<T, S::ALIGNED>(w, col, cols), g);
    if (b) widen16<T>(load_row16<T, S::ALIGNED>(b, col, cols), h);
#pragma unroll
    for (int j = 0; j < V; ++j) v[c][j] = v[c][j] * r * g[j] + h[j];
    out[c] = narrow16<T>(v[c]);
  }
  store_row16<T, S::ALIGNED, CH>(Y + row * ldy, S::col(0, t), cols, out);
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

// A ring of rows in shared memory, filled ahead by bulk copies: one per group
// of threads that shares rows.  A stage holds NIN matrices' rows, each copied
// as the whole 16-byte blocks it lies in; a row starts `offset` bytes into its
// place.  Every wait is bounded; a group whose wait gave up records it, stops
// copying and waiting and finishes with incomplete results.
template <class S, int NIN>
struct Ring {
  using T = typename S::T;
  const T *src[NIN];
  int64_t ld[NIN];
  uint32_t data, bars;   // shared-memory addresses
  uint8_t *base;         // data, as a pointer
  int place, stages, cols;
  bool leader, dead;
  int *watchdog;

  // Bytes of one matrix's row in a stage.
  static __host__ __device__ int place_bytes(int cols) {
    return (cols * (int)sizeof(T) + (S::ALIGNED ? 15 : 29)) / 16 * 16;
  }
  static __host__ __device__ size_t group_bytes(int cols, int stages) {
    return (size_t)stages * NIN * place_bytes(cols);
  }

  __device__ void init(uint8_t *smem, uint64_t *bar, int group, bool lead, int st, int c, int *wd) {
    cols = c, stages = st, place = place_bytes(c), leader = lead, dead = false, watchdog = wd;
    base = smem + (size_t)group * stages * NIN * place;
    data = smem_u32(base);
    bars = smem_u32(bar) + 8u * (uint32_t)(group * stages);
    if (leader) {
      for (int s = 0; s < stages; ++s) mbar_init(bars + 8u * s, 1);
      fence_mbar_init();
    }
  }
  // Leader: start the copies of `row` into `stage`.
  __device__ void fill(int stage, int64_t row) {
    const uint32_t bar = bars + 8u * (uint32_t)stage;
    uint32_t bytes[NIN], total = 0;
    const uint8_t *from[NIN];
#pragma unroll
    for (int i = 0; i < NIN; ++i) {
      bytes[i] = 0;
      if (src[i] == nullptr) continue;
      const uintptr_t p = reinterpret_cast<uintptr_t>(src[i] + row * ld[i]);
      from[i] = reinterpret_cast<const uint8_t *>(p & ~(uintptr_t)15);
      bytes[i] = ((uint32_t)(p & 15) + (uint32_t)cols * (uint32_t)sizeof(T) + 15u) & ~15u;
      total += bytes[i];
    }
    mbar_arrive_expect_tx(bar, total);
#pragma unroll
    for (int i = 0; i < NIN; ++i)
      if (bytes[i]) bulk_load(data + (uint32_t)((stage * NIN + i) * place), from[i], bytes[i], bar);
  }
  // False when this wait is the one that gave up.
  __device__ bool wait(int stage, uint32_t parity) {
    if (dead || mbar_wait(bars + 8u * (uint32_t)stage, parity)) return true;
    dead = true;
    if (leader) atomicCAS(watchdog, 0, kSiteNormRow);
    return false;
  }
  // Matrix i's copy of `row` in `stage`.
  __device__ const T *row_at(int stage, int i, int64_t row) const {
    const uintptr_t off = reinterpret_cast<uintptr_t>(src[i] + row * ld[i]) & 15;
    return reinterpret_cast<const T *>(base + (stage * NIN + i) * place + (S::ALIGNED ? 0 : off));
  }
};

// dX, and this block's partial sums of dw and db: partial[block][0][col] and
// partial[block][1][col] (or dw and db themselves when there is one block).  A
// stage of the ring is refilled one row later, when the next row's sums have
// shown that nobody reads it any more.
template <class S>
__global__ void __launch_bounds__(S::BWD_BLOCK, 1)
    ln_bwd_kernel(int rows, int cols, float inv, const typename S::T *dY, int64_t lddy,
                  const typename S::T *X, int64_t ldx, const typename S::T *w, const float *mean,
                  const float *rstd, const typename S::T *dR, int64_t lddr, typename S::T *dX,
                  int64_t lddx, float *partial, typename S::T *dw, typename S::T *db, int stages,
                  int stall, int *watchdog) {
  using T = typename S::T;
  constexpr int V = S::V, CH = S::CH, GROUP = S::GROUP, ROWS = S::BWD_ROWS;
  __shared__ float red[GROUP > 32 ? ROWS : 1][2][2][32];
  __shared__ uint64_t bars[ROWS * kMaxStages];
  struct GaveUp {
    int64_t row;
    int stage, stages;
    uint32_t phase;
  };
  __shared__ GaveUp gave_up[ROWS];  // where a ring's wait gave up (in registers it cost spills)
  extern __shared__ __align__(16) uint8_t rows_smem[];
  pdl_launch_dependents();
  const int t = threadIdx.x % GROUP, sub = threadIdx.x / GROUP;
  Ring<S, 3> ring;
  ring.src[0] = dY, ring.ld[0] = lddy;
  ring.src[1] = X, ring.ld[1] = ldx;
  ring.src[2] = dR, ring.ld[2] = lddr;
  ring.init(rows_smem, bars, sub, t == 0, stages, cols, watchdog);
  __syncthreads();
  pdl_wait();
  const bool grads = partial != nullptr || dw != nullptr || db != nullptr;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t row = (int64_t)blockIdx.x * ROWS + sub;
  if (t == 0)
    for (int s = stall && blockIdx.x == 0 && sub == 0 ? 1 : 0;  // test hook: a copy never begun
         s < stages && row + s * step < rows; ++s)
      ring.fill(s, row + s * step);
  float sw[CH][V], sb[CH][V];
  uint4 wr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < V; ++j) sw[c][j] = sb[c][j] = 0.f;
    wr[c] = load_row16<T, S::ALIGNED>(w, S::col(c, t), w ? cols : 0);
  }
  auto weights = [&](int c, float(&g)[V]) {
    if (w) {
      widen16<T>(wr[c], g);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = 1.f;
    }
  };
  float mu_next = 0.f, r_next = 0.f;
  if (row < rows) mu_next = mean[row], r_next = rstd[row];
  int buf = 0, stage = 0, last = -1;
  uint32_t phase = 0;
  for (; row < rows; row += step) {
    const float mu = mu_next, r = r_next;
    if (row + step < rows) mu_next = mean[row + step], r_next = rstd[row + step];
    if (!ring.wait(stage, phase) && t == 0)  // all stages are full but for the last row's
      gave_up[sub] = {row, stage, stages - (last >= 0 ? 1 : 0), phase};
    const T *dy = ring.row_at(stage, 0, row), *x = ring.row_at(stage, 1, row);
    float p[S::KEEP ? CH : 1][V], xh[S::KEEP ? CH : 1][V], s[2] = {0.f, 0.f};
    // p = dy w and xh of vector c.  Past the row's end p is 0, and so has xh to
    // be: -mu r may be past fp32's range, and 0 times that NaN.  (A vector of an
    // aligned row is all inside or all past; others take a branch that few warps
    // enter, as a select per element cost odd rows 3%.)
    auto read = [&](int c, float(&d)[V], float(&pc)[V], float(&hc)[V]) {
      float g[V];
      widen16<T>(load_row16<T, S::ALIGNED>(dy, S::col(c, t), cols), d);
      widen16<T>(load_row16<T, S::ALIGNED>(x, S::col(c, t), cols), hc);
      weights(c, g);
      const float rc = !S::ALIGNED || S::col(c, t) < cols ? r : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        hc[j] = (hc[j] - mu) * rc;
        pc[j] = d[j] * g[j];
      }
      if (!S::ALIGNED && S::col(c, t) + V > cols) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (S::col(c, t) + j >= cols) hc[j] = 0.f;
      }
    };
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float d[V];
      float(&pc)[V] = p[S::KEEP ? c : 0], (&hc)[V] = xh[S::KEEP ? c : 0];
      read(c, d, pc, hc);
#pragma unroll
      for (int j = 0; j < V; ++j) {  // past the row's end d is 0, and with it every term
        s[0] += pc[j];
        s[1] += pc[j] * hc[j];
        sw[c][j] += d[j] * hc[j];
        sb[c][j] += d[j];
      }
    }
    row_sum<S>(s, red[GROUP > 32 ? sub : 0][buf], sub);
    buf ^= 1;
    if (GROUP == 32) __syncwarp();
    if (t == 0 && !ring.dead && last >= 0 && row + (stages - 1) * step < rows)
      ring.fill(last, row + (stages - 1) * step);
    last = stage;
    const float m1 = s[0] * inv, m2 = s[1] * inv;
    uint4 out[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float e[V], d[V];
      float(&pc)[V] = p[S::KEEP ? c : 0], (&hc)[V] = xh[S::KEEP ? c : 0];
      if constexpr (!S::KEEP) read(c, d, pc, hc);
      if (dR) {
        widen16<T>(load_row16<T, S::ALIGNED>(ring.row_at(stage, 2, row), S::col(c, t), cols), e);
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] += r * (pc[j] - m1 - hc[j] * m2);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = r * (pc[j] - m1 - hc[j] * m2);
      }
      out[c] = narrow16<T>(e);
    }
    store_row16<T, S::ALIGNED, CH>(dX + row * lddx, S::col(0, t), cols, out);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (ring.dead && t == 0) {
    // No copy was begun after the wait that gave up; those begun before it land
    // (a bounded wait each) before the block leaves or puts its memory to other use.
    const GaveUp g = gave_up[sub];
    for (int k = 0; k < g.stages && g.row + k * step < rows; ++k) {
      const bool wrap = g.stage + k >= stages;
      mbar_wait(ring.bars + 8u * (uint32_t)(wrap ? g.stage + k - stages : g.stage + k),
                g.phase ^ (wrap ? 1u : 0u));
    }
  }
  if (!grads) return;
  // the block's rows side by side, added in their order (the ring is idle now)
  float *fold = reinterpret_cast<float *>(rows_smem);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float(&sum)[CH][V] = k ? sb : sw;
    T *out = k ? db : dw;
    float *part = partial ? partial + ((int64_t)blockIdx.x * 2 + k) * cols : nullptr;
    if constexpr (ROWS > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) fold[sub * S::CAPACITY + S::col(c, t) + j] = sum[c][j];
      __syncthreads();
      for (int col = threadIdx.x; col < cols; col += S::BWD_BLOCK) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) v += fold[i * S::CAPACITY + col];
        if (part)
          part[col] = v;
        else if (out)
          out[col] = from_f32<T>(v);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int col = S::col(c, t) + j;
          if (col >= cols) continue;
          if (part)
            part[col] = sum[c][j];
          else if (out)
            out[col] = from_f32<T>(sum[c][j]);
        }
    }
  }
}

// ---------------------------------------------- rows too long for registers
template <class T>
struct LongShape {
  static constexpr int GROUP = 1024;
};

template <class T>
__global__ void __launch_bounds__(1024)
    ln_fwd_long_kernel(int cols, float eps, const T *X, int64_t ldx, const T *w, const T *b, T *Y,
                       int64_t ldy, float *mean, float *rstd) {
  __shared__ float red[2][1][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T *x = X + row * ldx;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < cols; c += 1024) s[0] += to_f32<T>(x[c]);
  row_sum<LongShape<T>>(s, red[0]);
  const float mu = s[0] / cols;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < cols; c += 1024) {
    const float d = to_f32<T>(x[c]) - mu;
    s[0] += d * d;
  }
  row_sum<LongShape<T>>(s, red[1]);
  const float r = rsqrtf(s[0] / cols + eps);
  for (int c = threadIdx.x; c < cols; c += 1024)
    Y[row * ldy + c] = from_f32<T>((to_f32<T>(x[c]) - mu) * r * (w ? to_f32<T>(w[c]) : 1.f) +
                                   (b ? to_f32<T>(b[c]) : 0.f));
  if (threadIdx.x == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

template <class T>
__global__ void __launch_bounds__(1024)
    ln_dx_long_kernel(int cols, const T *dY, int64_t lddy, const T *X, int64_t ldx, const T *w,
                      const float *mean, const float *rstd, const T *dR, int64_t lddr, T *dX,
                      int64_t lddx) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const float mu = mean[row], r = rstd[row];
  float s[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < cols; c += 1024) {
    const float p = to_f32<T>(dY[row * lddy + c]) * (w ? to_f32<T>(w[c]) : 1.f);
    s[0] += p;
    s[1] += p * (to_f32<T>(X[row * ldx + c]) - mu) * r;
  }
  row_sum<LongShape<T>>(s, red);
  const float m1 = s[0] / cols, m2 = s[1] / cols;
  for (int c = threadIdx.x; c < cols; c += 1024) {
    const float p = to_f32<T>(dY[row * lddy + c]) * (w ? to_f32<T>(w[c]) : 1.f);
    const float xh = (to_f32<T>(X[row * ldx + c]) - mu) * r;
    const float d = r * (p - m1 - xh * m2);
    dX[row * lddx + c] = from_f32<T>(dR ? d + to_f32<T>(dR[row * lddr + c]) : d);
  }
}

// Partial sums of dw and db over the rows of one part, a column per thread.
template <class T>
__global__ void __launch_bounds__(256)
    ln_dw_long_kernel(int rows, int cols, const T *dY, int64_t lddy, const T *X, int64_t ldx,
                      const float *mean, const float *rstd, float *partial) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * 256 + threadIdx.x, parts = gridDim.y, part = blockIdx.y;
  if (c >= cols) return;
  float sw = 0.f, sb = 0.f;
  for (int64_t i = part; i < rows; i += parts) {
    const float d = to_f32<T>(dY[i * lddy + c]);
    sw += d * (to_f32<T>(X[i * ldx + c]) - mean[i]) * rstd[i];
    sb += d;
  }
  partial[((int64_t)part * 2) * cols + c] = sw;
  partial[((int64_t)part * 2 + 1) * cols + c] = sb;
}

// ------------------------------------------------------------- host side
constexpr int kMaxRegisterCols = 16384;
constexpr int kMaxRingBytes = 32768;  // of a row in the backward ring: two stages of three rows fit
constexpr int kLongParts = 16;        // row shares of the column sums of longer rows

// f(shape) for the shape a row of `cols` elements is held in: at most 32
// elements per thread forward, 16 (for rows beyond 8192, 32) backward.
// Measured at 16384 x 4096 bf16, forward: 128 threads to a row 45.3 us (5.93
// TB/s), 256 threads 54.8 us; 65536 x 1024: a warp 44.3 us.  Backward with dR:
// 86.3 us (6.22 TB/s); one row ahead in registers instead of the ring 115 us.
template <class T, bool ALIGNED, bool BWD, class F>
cudaError_t with_shape(int cols, F &&f) {
  constexpr int K = 8 / kVec<T>;  // vectors in 8 elements
  constexpr int W = BWD ? 2 : 1;  // threads, relative to forward
  if (cols <= 256) return f(Shape<T, ALIGNED, K, 32>{});
  if (cols <= 512) return f(Shape<T, ALIGNED, 2 * K, 32>{});
  if (cols <= 1024) return f(Shape<T, ALIGNED, 4 * K / W, 32 * W>{});
  if (cols <= 2048) return f(Shape<T, ALIGNED, 4 * K / W, 64 * W>{});
  if (cols <= 4096) return f(Shape<T, ALIGNED, 4 * K / W, 128 * W>{});
  if (cols <= 8192) return f(Shape<T, ALIGNED, 4 * K / W, 256 * W>{});
  if constexpr (!BWD || sizeof(T) == 2) return f(Shape<T, ALIGNED, 4 * K, 512>{});
  static_assert(kMaxRingBytes <= 8192 * 4, "backward, no fp32 row gets here");
  return cudaErrorInvalidValue;
}
template <class T, bool BWD, class F>
cudaError_t with_shape(int cols, bool aligned, F &&f) {
  return aligned ? with_shape<T, true, BWD>(cols, f) : with_shape<T, false, BWD>(cols, f);
}

// Stages of the backward kernel's rings, and its dynamic shared memory: the
// rings, and the fold of the column sums in their place.
template <class S, int NIN>
int ring_stages(int cols, bool fold, size_t *smem) {
  const size_t one = Ring<S, NIN>::group_bytes(cols, 1) * S::BWD_ROWS;
  const size_t budget = 212 * 1024;  // static shared memory and the system's share aside
  int stages = (int)(budget / one);
  stages = stages < 2 ? 2 : stages > kMaxStages ? kMaxStages : stages;
  *smem = one * stages;
  const size_t sums = fold && S::BWD_ROWS > 1 ? (size_t)S::BWD_ROWS * S::CAPACITY * sizeof(float) : 0;
  if (*smem < sums) *smem = sums;
  return stages;
}

// Opt in to `smem` bytes of dynamic shared memory, once per kernel and device
// (the largest any call needs: 220 KB).
template <auto KERNEL>
cudaError_t allow_smem() {
  static std::atomic<bool> set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return e;
}

template <class T>
cudaError_t fwd(int rows, int cols, float eps, const void *X, int64_t ldx, const void *weight,
                const void *bias, void *Y, int64_t ldy, float *mean, float *rstd,
                cudaStream_t stream) {
  const T *x = static_cast<const T *>(X), *w = static_cast<const T *>(weight);
  const T *b = static_cast<const T *>(bias);
  T *y = static_cast<T *>(Y);
  cudaError_t e;
  if (cols > kMaxRegisterCols) {
    e = launch_kernel(ln_fwd_long_kernel<T>, dim3((unsigned)rows), dim3(1024), 0, stream, 1u, cols,
                      eps, x, ldx, w, b, y, ldy, mean, rstd);
  } else {
    constexpr int es = sizeof(T);
    const bool vec = rows_aligned(X, ldx, es) && rows_aligned(Y, ldy, es) &&
                     rows_aligned(w, 0, es) && rows_aligned(b, 0, es) && cols * es % 16 == 0;
    e = with_shape<T, false>(cols, vec, [&](auto shape) {
      using S = decltype(shape);
      const int64_t blocks = ((int64_t)rows + S::ROWS - 1) / S::ROWS;
      return launch_kernel(ln_fwd_kernel<S>, dim3((unsigned)blocks), dim3(S::BLOCK), 0, stream, 1u,
                           rows, cols, 1.f / cols, eps, x, ldx, w, b, y, ldy, mean, rstd);
    });
  }
  if (e == cudaSuccess) count_launch();
  return e;
}

// Blocks of the backward kernel, each one partial sum.
int bwd_parts(int rows, int rows_per_block, int num_sms) {
  const int64_t need = ((int64_t)rows + rows_per_block - 1) / rows_per_block;
  return (int)(need < 1 ? 1 : need < num_sms ? need : num_sms);
}

template <class T>
cudaError_t bwd(int dtype, int rows, int cols, const void *dY, int64_t lddy, const void *X,
                int64_t ldx, const void *weight, const float *mean, const float *rstd,
                const void *dR, int64_t lddr, void *dX, int64_t lddx, void *dweight, void *dbias,
                float *partial, int num_sms, cudaStream_t stream) {
  const T *dy = static_cast<const T *>(dY), *x = static_cast<const T *>(X);
  const T *w = static_cast<const T *>(weight), *dr = static_cast<const T *>(dR);
  T *dx = static_cast<T *>(dX), *dw = static_cast<T *>(dweight), *db = static_cast<T *>(dbias);
  const bool grads = dw != nullptr || db != nullptr;
  cudaError_t e = cudaSuccess;
  int parts = 1;
  if (cols > kMaxRingBytes / (int)sizeof(T)) {
    if (rows > 0) {
      e = launch_kernel(ln_dx_long_kernel<T>, dim3((unsigned)rows), dim3(1024), 0, stream, 1u, cols,
                        dy, lddy, x, ldx, w, mean, rstd, dr, lddr, dx, lddx);
      if (e != cudaSuccess) return e;
      count_launch();
    }
    if (!grads) return e;
    const unsigned gx = (unsigned)((cols + 255) / 256);
    parts = rows < kLongParts ? (rows < 1 ? 1 : rows) : kLongParts;
    e = launch_kernel(ln_dw_long_kernel<T>, dim3(gx, (unsigned)parts), dim3(256), 0, stream, 1u,
                      rows, cols, dy, lddy, x, ldx, mean, rstd, partial);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_column_sums(dtype, partial, parts, cols, dw, db, stream);
  }
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  constexpr int es = sizeof(T);
  const bool vec = rows_aligned(dY, lddy, es) && rows_aligned(X, ldx, es) &&
                   rows_aligned(w, 0, es) && rows_aligned(dr, dr ? lddr : 0, es) &&
                   rows_aligned(dX, lddx, es) && cols * es % 16 == 0;
  e = with_shape<T, true>(cols, vec, [&](auto shape) {
    using S = decltype(shape);
    parts = bwd_parts(rows, S::BWD_ROWS, num_sms);
    size_t smem = 0;
    const int stages = ring_stages<S, 3>(cols, grads, &smem);
    const cudaError_t ea = allow_smem<ln_bwd_kernel<S>>();
    if (ea != cudaSuccess) return ea;
    return launch_kernel(ln_bwd_kernel<S>, dim3((unsigned)parts), dim3(S::BWD_BLOCK), smem, stream, 1u,
                         rows, cols, 1.f / cols, dy, lddy, x, ldx, w, mean, rstd, dr, lddr, dx,
                         lddx, grads && parts > 1 ? partial : nullptr, dw, db, stages,
                         test_stall(), wd);
  });
  if (e != cudaSuccess) return e;
  count_launch();
  return grads && parts > 1 ? launch_column_sums(dtype, partial, parts, cols, dw, db, stream) : e;
}

}  // namespace

cudaError_t launch_layer_norm(int dtype, int rows, int cols, float eps, const void *X, int64_t ldx,
                              const void *weight, const void *bias, void *Y, int64_t ldy,
                              float *mean, float *rstd, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return fwd<__nv_bfloat16>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
    case DGEMM_DTYPE_F16:
      return fwd<__half>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
    default:
      return fwd<float>(rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd, stream);
  }
}

size_t layer_norm_scratch(int rows, int cols, bool with_grads, int num_sms) {
  if (!with_grads) return 0;
  const int ring = bwd_parts(rows, 1, num_sms);
  const int parts = ring > kLongParts ? ring : kLongParts;
  return (size_t)parts * 2 * cols * sizeof(float);
}

cudaError_t launch_layer_norm_backward(int dtype, int rows, int cols, const void *dY, int64_t lddy,
                                       const void *X, int64_t ldx, const void *weight,
                                       const float *mean, const float *rstd, const void *dR,
                                       int64_t lddr, void *dX, int64_t lddx, void *dweight,
                                       void *dbias, float *partial, int num_sms,
                                       cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_BF16:
      return bwd<__nv_bfloat16>(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr,
                                dX, lddx, dweight, dbias, partial, num_sms, stream);
    case DGEMM_DTYPE_F16:
      return bwd<__half>(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX,
                         lddx, dweight, dbias, partial, num_sms, stream);
    default:
      return bwd<float>(dtype, rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dR, lddr, dX,
                        lddx, dweight, dbias, partial, num_sms, stream);
  }
}

}  // namespace dg
