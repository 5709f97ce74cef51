// quant.cu -- rows in 8-bit integers with one scale each, and the forms of them
// that the integer products read.
//
// Bound by memory: a row is read once and held in registers up to 16384 elements
// (longer rows are read again, from L2 mostly).  Three
// kinds of output: the integers, for a user; the integers in fp16, which hold
// them exactly, for the products (int8_small.cu, int8_pair.cu multiply in fp16);
// and columns instead of rows, transposed on the way, for weights stored in x
// out.  8192 x 4096 bf16 rows take 27 us (floor 15), 8192 x 14336 fp32 rows 110 (88): a
// row's loads, maximum and stores follow one another.  Columns, which a program quantises once for each
// weight, take 167 us for 4096 x 14336 bf16 (floor 26), read twice, an element per load.
//
// Weights on rows that TMA cannot read are copied by blocks of the same launch (in one of its
// own a product of 1000 x 997 x 1013 took 14.1 us for 12.3, of 64 x 4095 x 14335 43.1 for 35.9).
//
// A kernel here signals its dependents only after its own wait, unlike the
// library's other kernels: a product that follows may then read its weights
// before this kernel is done, since all that came before it is.
#include <cstdint>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "quant.cuh"
#include "rowvec.cuh"

namespace dg {
namespace {

// The copies' share of block `block` of `blocks`: 16 bytes per thread and round, four rounds'
// loads in flight.
__device__ __forceinline__ void copy_bytes(const ByteCopies &copies, int64_t block, int64_t blocks) {
  constexpr int AHEAD = 4;
  const int64_t first = block * blockDim.x + threadIdx.x, step = blocks * blockDim.x;
  for (int n = 0; n < copies.n; ++n) {
    const ByteCopies::Job &j = copies.job[n];
    const int vecs = (j.cols + 15) / 16;
    const int64_t all = (int64_t)j.rows * vecs;
    for (int64_t i0 = first; i0 < all; i0 += AHEAD * step) {
      RowBlocks b[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int64_t i = i0 + k * step, row = i / vecs;
        b[k] = fetch_row16<uint8_t, false>(j.src + row * j.lds, (int)(i - row * vecs) * 16, i < all ? j.cols : 0);
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int64_t i = i0 + k * step, row = i / vecs;
        if (i >= all) break;
        const uint8_t *src = j.src + row * j.lds;
        // (what is behind the row's end is read by nothing)
        *reinterpret_cast<uint4 *>(j.dst + row * j.ldd + (i - row * vecs) * 16) =
            shift16<uint8_t>(b[k].a, b[k].b, (int)(reinterpret_cast<uintptr_t>(src) & 15));
      }
    }
  }
}
// Blocks for them, besides those of the tokens.
int copy_blocks(const ByteCopies &copies, int threads, int num_sms) {
  int64_t vecs = 0;
  for (int n = 0; n < copies.n; ++n) vecs += (int64_t)copies.job[n].rows * ((copies.job[n].cols + 15) / 16);
  const int64_t want = (vecs + 4 * threads - 1) / (4 * threads), most = (int64_t)num_sms * (2048 / threads);
  return (int)(want < most ? want : most);
}

// One row per block, whose threads hold HELD vectors of it each; the blocks behind copy bytes.
template <class T, class O, bool ALIGNED, int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    quantize_rows_kernel(int rows, int cols, const T *X, int64_t ldx, O *Q, int64_t ldq, float *scale,
                         bool vec, const __grid_constant__ ByteCopies copies) {
  constexpr int V = kVec<T>;
  __shared__ uint32_t tops[THREADS / 32];
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= (unsigned)rows) {
    copy_bytes(copies, blockIdx.x - rows, gridDim.x - rows);
    return;
  }
  const int64_t row = blockIdx.x;
  const T *x = X + row * ldx;
  O *out = Q + row * ldq;
  RowBlocks b[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    b[k] = fetch_row16<T, ALIGNED>(x, min((int)(threadIdx.x + k * THREADS), cols) * V, cols);
  uint4 held[HELD];
  uint32_t top = 0;
  auto widest = [&](const float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) top = max(top, abs_bits(v[j]));
  };
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const int col = min((int)(threadIdx.x + k * THREADS), cols) * V;
    if (col < cols) {
      float v[V];
      held[k] = take_row16<T, ALIGNED>(b[k], x, col, cols);
      widen16<T>(held[k], v);
      widest(v);
    }
  }
  for (int64_t c = (int64_t)(threadIdx.x + HELD * THREADS) * V; c < cols; c += THREADS * V) {
    float v[V];
    widen16<T>(load_row16<T, ALIGNED>(x, (int)c, cols), v);
    widest(v);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < THREADS / 32 ? tops[threadIdx.x & 31] : 0u);
  const RowScale r = row_scale(top);
  if (threadIdx.x == 0) scale[row] = r.scale;
  auto finish = [&](float (&v)[V], int col) {
    quantise_vec<V>(v, r);
    put<V>(out + col, v, cols - col, vec);
  };
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const int col = min((int)(threadIdx.x + k * THREADS), cols) * V;
    if (col < cols) {
      float v[V];
      widen16<T>(held[k], v);
      finish(v, col);
    }
  }
  for (int64_t c = (int64_t)(threadIdx.x + HELD * THREADS) * V; c < cols; c += THREADS * V) {
    float v[V];
    widen16<T>(load_row16<T, ALIGNED>(x, (int)c, cols), v);
    finish(v, (int)c);
  }
}

template <class T, class O>
cudaError_t launch_rows(int rows, int cols, const void *X, int64_t ldx, O *Q, int64_t ldq,
                        float *scale, const ByteCopies &copies, int num_sms, cudaStream_t stream) {
  const bool al = rows_aligned(X, ldx, sizeof(T)) && cols % kVec<T> == 0;
  const bool vec = reinterpret_cast<uintptr_t>(Q) % kVec<T> == 0 && ldq % kVec<T> == 0;
  // Few rows, as in a decoding step: as many threads as hold one or two vectors each, for the
  // shortest chain (64 rows of 4096 fp32 in 1.8 us, 2.1 with eight held); else threads that
  // hold 32 elements.
  const int vecs = (cols + kVec<T> - 1) / kVec<T>;
  const bool few = rows <= 2 * num_sms;
  auto go = [&](auto kern, int threads) {
    const unsigned grid = (unsigned)rows + (unsigned)copy_blocks(copies, threads, num_sms);
    const cudaError_t e = launch_kernel(kern, dim3(grid), dim3(threads), 0, stream, 1u, rows, cols,
                                        static_cast<const T *>(X), ldx, Q, ldq, scale, vec, copies);
    if (e == cudaSuccess) count_launch();
    return e;
  };
#define DG_ROWS(threads, held)                                                \
  (al ? go(quantize_rows_kernel<T, O, true, threads, held>, threads)        \
      : go(quantize_rows_kernel<T, O, false, threads, held>, threads))
  constexpr int MANY = 32 / kVec<T>;
  if (few) {
    if (vecs <= 128) return DG_ROWS(128, 1);
    if (vecs <= 512 * 2) return DG_ROWS(512, 2);
    return DG_ROWS(1024, MANY / 2);
  }
  return vecs <= 128 * MANY ? DG_ROWS(128, MANY) : DG_ROWS(512, MANY);
#undef DG_ROWS
}

// The integers of X (int8) in fp16.
constexpr int kExpandThreads = 256;
__global__ void __launch_bounds__(kExpandThreads)
    expand_rows_kernel(int rows, int cols, const int8_t *X, int64_t ldx, __half *T, int64_t ldt,
                       bool vec, int blocks, const __grid_constant__ ByteCopies copies) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= (unsigned)blocks) {
    copy_bytes(copies, blockIdx.x - blocks, gridDim.x - blocks);
    return;
  }
  const int vecs = (cols + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * kExpandThreads + threadIdx.x; i < (int64_t)rows * vecs;
       i += (int64_t)blocks * kExpandThreads) {
    const int64_t row = i / vecs;
    const int col = (int)(i - row * vecs) * 8;
    const int8_t *x = X + row * ldx + col;
    int8_t b[8] = {};
    if (vec && col + 8 <= cols) {
      const uint2 w = *reinterpret_cast<const uint2 *>(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = (int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < cols) b[j] = x[j];
    }
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (float)b[j];
    put<8>(T + row * ldt + col, q, 8, true);
  }
}

// ------------------------------------------------------- columns, transposed
// tops[c] = the largest |X[r][c]| over the rows, as bits (zero before).
template <class T>
__global__ void __launch_bounds__(256)
    column_tops_kernel(int rows, int cols, const T *X, int64_t ldx, uint32_t *tops) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  if (col >= cols) return;
  uint32_t top = 0;
#pragma unroll 8
  for (int64_t r = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.y * 4)
    top = max(top, abs_bits(to_f32<T>(X[r * ldx + col])));
  atomicMax(tops + col, top);  // of whole numbers: the same in any order
}

__global__ void clear_kernel(int n, uint32_t *p) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0;
}

// Q[c][r] = X[r][c] in column c's scale; tiles of 64 x 64.
template <class T>
__global__ void __launch_bounds__(256)
    quantize_columns_kernel(int rows, int cols, const T *X, int64_t ldx, int8_t *Q, int64_t ldq,
                            const uint32_t *tops, float *scale, bool vec) {
  __shared__ int8_t tile[64][68];  // [column][row]
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c0 = (int64_t)blockIdx.x * 64;
  const int64_t col = c0 + (threadIdx.x & 63);
  const bool in = col < cols;
  const RowScale s = row_scale(in ? tops[col] : 0u);
  if (in && blockIdx.y == 0 && threadIdx.x < 64) scale[col] = s.scale;
  for (int64_t r0 = (int64_t)blockIdx.y * 64; r0 < rows; r0 += (int64_t)gridDim.y * 64) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t r = r0 + (threadIdx.x >> 6) * 16 + i;
      x[i] = in && r < rows ? to_f32<T>(X[r * ldx + col]) : 0.f;
    }
    __syncthreads();  // the tile before has been stored
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) w |= ((uint32_t)(int)quantised(x[i + k], s) & 0xFFu) << (8 * k);
      *reinterpret_cast<uint32_t *>(&tile[threadIdx.x & 63][(threadIdx.x >> 6) * 16 + i]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = (threadIdx.x >> 4) + 16 * i, r = (threadIdx.x & 15) * 4;
      if (c0 + c >= cols) continue;
      int8_t *out = Q + (c0 + c) * ldq + r0 + r;
      if (vec && r0 + r + 4 <= rows) {
        *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<const uint32_t *>(&tile[c][r]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r0 + r + k < rows) out[k] = tile[c][r + k];
      }
    }
  }
}

template <class T>
cudaError_t launch_columns(int rows, int cols, const void *X, int64_t ldx, int8_t *Q, int64_t ldq,
                           float *scale, uint32_t *tops, int num_sms, cudaStream_t stream) {
  const unsigned gx = (unsigned)((cols + 63LL) / 64);
  // about eight blocks per SM, each with rows of its own
  const int64_t want = (8LL * num_sms + gx - 1) / gx, most = (rows + 63LL) / 64;
  const unsigned gy = (unsigned)(want < most ? want : most < 1 ? 1 : most);
  const unsigned gc = (unsigned)((cols + 1023LL) / 1024);
  cudaError_t e = launch_kernel(clear_kernel, dim3(gc < 1024 ? gc : 1024), dim3(256), 0, stream, 1u,
                                cols, tops);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_kernel(column_tops_kernel<T>, dim3(gx, gy), dim3(256), 0, stream, 1u, rows, cols,
                    static_cast<const T *>(X), ldx, tops);
  if (e != cudaSuccess) return e;
  count_launch();
  const bool vec = reinterpret_cast<uintptr_t>(Q) % 4 == 0 && ldq % 4 == 0;
  e = launch_kernel(quantize_columns_kernel<T>, dim3(gx, gy), dim3(256), 0, stream, 1u, rows, cols,
                    static_cast<const T *>(X), ldx, Q, ldq, static_cast<const uint32_t *>(tops), scale,
                    vec);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_quantize_rows(int dtype, int rows, int cols, const void *X, int64_t ldx,
                                 int8_t *Q, int64_t ldq, float *scale, int num_sms,
                                 cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_F32: return launch_rows<float>(rows, cols, X, ldx, Q, ldq, scale, {}, num_sms, stream);
    case DGEMM_DTYPE_BF16: return launch_rows<__nv_bfloat16>(rows, cols, X, ldx, Q, ldq, scale, {}, num_sms, stream);
    default: return launch_rows<__half>(rows, cols, X, ldx, Q, ldq, scale, {}, num_sms, stream);
  }
}

cudaError_t launch_quantize_tokens(int dtype, int rows, int cols, const void *X, int64_t ldx,
                                   void *T, int64_t ldt, float *scale, const ByteCopies &copies,
                                   int num_sms, cudaStream_t stream) {
  __half *t = static_cast<__half *>(T);
  switch (dtype) {
    case DGEMM_DTYPE_F32: return launch_rows<float>(rows, cols, X, ldx, t, ldt, scale, copies, num_sms, stream);
    case DGEMM_DTYPE_BF16: return launch_rows<__nv_bfloat16>(rows, cols, X, ldx, t, ldt, scale, copies, num_sms, stream);
    default: return launch_rows<__half>(rows, cols, X, ldx, t, ldt, scale, copies, num_sms, stream);
  }
}

cudaError_t launch_expand_tokens(int rows, int cols, const int8_t *X, int64_t ldx, void *T,
                                 int64_t ldt, const ByteCopies &copies, int num_sms,
                                 cudaStream_t stream) {
  const int64_t vecs = (int64_t)rows * ((cols + 7) / 8), want = (vecs + kExpandThreads - 1) / kExpandThreads;
  const int most = 8 * num_sms, blocks = want < most ? (int)want : most;
  const bool vec = reinterpret_cast<uintptr_t>(X) % 8 == 0 && ldx % 8 == 0;
  const cudaError_t e = launch_kernel(
      expand_rows_kernel, dim3((unsigned)(blocks + copy_blocks(copies, kExpandThreads, num_sms))),
      dim3(kExpandThreads), 0, stream, 1u, rows, cols, X, ldx, static_cast<__half *>(T), ldt, vec, blocks, copies);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_quantize_columns(int dtype, int rows, int cols, const void *X, int64_t ldx,
                                    int8_t *Q, int64_t ldq, float *scale, uint32_t *tops,
                                    int num_sms, cudaStream_t stream) {
  switch (dtype) {
    case DGEMM_DTYPE_F32:
      return launch_columns<float>(rows, cols, X, ldx, Q, ldq, scale, tops, num_sms, stream);
    case DGEMM_DTYPE_BF16:
      return launch_columns<__nv_bfloat16>(rows, cols, X, ldx, Q, ldq, scale, tops, num_sms, stream);
    default:
      return launch_columns<__half>(rows, cols, X, ldx, Q, ldq, scale, tops, num_sms, stream);
  }
}

}  // namespace dg
