// int8.cu -- which kernel runs a product with 8-bit weights, and how it is cut.
#include <cstdint>
#include <cstdlib>
#include <cuda_runtime.h>

#include "../../include/dgemm.h"
#include "kernels.h"
#include "ops.h"

namespace dg {
namespace {

// DGEMM_INT8_*: an environment variable's value in lo .. hi, or -1 (read at
// every launch, for tests and tuning).
int knob(const char *name, int lo, int hi) {
  const char *e = getenv(name);
  if (e == nullptr || e[0] < '0' || e[0] > '9') return -1;
  const int v = atoi(e);
  return v >= lo && v <= hi ? v : -1;
}

Int8Plan small_plan(const Int8Gemm &p, int num_sms) {
  const int f_nt = knob("DGEMM_INT8_NT", 16, 128), f_splits = knob("DGEMM_INT8_SPLITS", 1, 8);
  const int all = p.M >= 128 ? 128 : (p.M + 15) / 16 * 16;
  Int8Plan plan = {f_nt >= 0 ? (f_nt + 15) / 16 * 16 : all, 1, 1};
  const int tf = p.gated ? 64 : 128;
  const int64_t tiles = (int64_t)((p.N + tf - 1) / tf) * ((p.M + plan.nt - 1) / plan.nt);
  const int64_t kblocks = (p.K + 127) / 128;
  for (int s : {2, 3, 4, 6, 8}) {
    if (s > kblocks) break;
    if (tiles * s <= small_resident({plan.nt, 1, s, 2}, num_sms) * s) plan.splits = s;
  }
  if (f_splits >= 0) plan.splits = f_splits;
  if (tiles > small_resident({plan.nt, 1, plan.splits, 1}, num_sms)) plan.per_sm = 2;
  return plan;
}

}  // namespace

cudaError_t launch_int8(const Int8Gemm &p, int num_sms, cudaStream_t stream) {
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  const int force = p.K > 0 ? knob("DGEMM_INT8_PAIR", 0, 1) : 0;
  if (force < 0 ? p.M > 128 : force == 1) {
    const int f_nt = knob("DGEMM_INT8_NT", 32, 192);
    const int all = p.M >= 192 ? 192 : (p.M + 31) / 32 * 32;
    return launch_int8_pair(p, f_nt >= 0 ? (f_nt + 31) / 32 * 32 : all, wd, stream);
  }
  return launch_int8_small(p, small_plan(p, num_sms), wd, stream);
}

}  // namespace dg
