// fused.cu -- the fused products of the feed-forward operators: operands that
// TMA cannot read are staged first, then one kernel runs.
#include <cstdint>
#include <cuda_runtime.h>

#include "api_common.h"
#include "kernels.h"
#include "ops.h"

namespace dg {
namespace {

// Re-pitched copies of operands whose rows do not start on 16-byte
// boundaries, in stream-ordered scratch that lives until the product has run.
// An operand given twice is staged once.
struct Staging {
  struct Item {
    const void **p;
    int64_t *ld;
    int rows, cols;
  };
  Item items[4];
  int n = 0;

  void want(const void *&p, int64_t &ld, int rows, int cols) {
    if (p == nullptr || rows == 0 || cols == 0 || tma_ok(p, ld, 2)) return;
    items[n++] = {&p, &ld, rows, cols};
  }

  cudaError_t run(void **scratch, int num_sms, cudaStream_t stream) {
    *scratch = nullptr;
    if (n == 0) return cudaSuccess;
    int owner[4];
    size_t at[4], total = 0;
    for (int i = 0; i < n; ++i) {
      owner[i] = i;
      for (int j = 0; j < i; ++j)
        if (*items[j].p == *items[i].p && *items[j].ld == *items[i].ld) owner[i] = j;
      at[i] = total;
      if (owner[i] == i)
        total += (size_t)((int64_t)items[i].rows * pitch(items[i].cols) * 2 + 255) / 256 * 256;
    }
    cudaError_t e = scratch_alloc(scratch, total, stream);
    if (e != cudaSuccess) return e;
    char *s = static_cast<char *>(*scratch);
    StageJob jobs[4];
    int njobs = 0;
    for (int i = 0; i < n; ++i)
      if (owner[i] == i)
        jobs[njobs++] = {*items[i].p, *items[i].ld, s + at[i], pitch(items[i].cols),
                         items[i].rows, items[i].cols, false};
    for (int j = 0; j < njobs && e == cudaSuccess; j += 2)
      e = launch_stage(jobs + j, njobs - j < 2 ? njobs - j : 2, 2, num_sms, stream);
    for (int i = 0; i < n; ++i) {
      *items[i].p = s + at[owner[i]];
      *items[i].ld = pitch(items[i].cols);
    }
    return e;
  }

  static int64_t pitch(int cols) { return (cols + 7) / 8 * 8; }
};

}  // namespace

cudaError_t launch_fused(const FusedGemm &p0, int num_sms, cudaStream_t stream) {
  FusedGemm p = p0;
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  Staging st;
  const int ar = p.a_t ? p.K : p.M, ac = p.a_t ? p.M : p.K;
  const int br = p.b_t ? p.N : p.K, bc = p.b_t ? p.K : p.N;
  st.want(p.A, p.lda, ar, ac);
  st.want(p.B, p.ldb, br, bc);
  if (p.dual == Dual::kSum || p.dual == Dual::kPair) st.want(p.A2, p.lda2, ar, ac);
  if (p.dual != Dual::kNone) st.want(p.B2, p.ldb2, br, bc);
  void *scratch = nullptr;
  cudaError_t e = st.run(&scratch, num_sms, stream);
  if (e == cudaSuccess) {
    if (p.a_t)
      e = p.b_t ? cudaErrorInvalidValue : launch_fused_pair_unit_2(p, wd, stream);
    else
      e = p.b_t ? launch_fused_pair_unit_1(p, wd, stream) : launch_fused_pair_unit_0(p, wd, stream);
  }
  if (scratch != nullptr) {
    const cudaError_t e2 = scratch_free(scratch, stream);
    if (e == cudaSuccess) e = e2;
  }
  return e;
}

}  // namespace dg
