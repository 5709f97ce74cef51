// api_common.h -- what the files of exported entry points (api.cu,
// ops_api.cu) share: errors, device facts and pointer checks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace dg {

constexpr int kMaxDevices = 64;

// Keep the CUDA error text for dgemm_last_cuda_error; returns DGEMM_ERR_CUDA.
int cuda_fail(cudaError_t e, const char *where);

// Current device and its SM count; DGEMM_ERR_ARCH unless it is compute
// capability 10.3.  Device facts are looked up once.
int current_device(int *dev, int *num_sms);

// DGEMM_ERR_INVALID_POINTER unless p is memory that `dev`'s kernels can
// address directly.
int check_device_pointer(const void *p, int dev);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte range [lo, hi) spanned by a rows x cols row-major matrix.
struct Span {
  uintptr_t lo, hi;
};
inline Span span(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (rows <= 0 || cols <= 0) return {lo, lo};
  return {lo, lo + static_cast<uintptr_t>(((rows - 1) * ld + cols) * es)};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// TMA needs 16-byte aligned bases and row pitches that are multiples of 16 B.
inline bool tma_ok(const void *p, int64_t ld, int es) { return aligned(p, 16) && (ld * es) % 16 == 0; }

}  // namespace dg
