// fused.cu -- the fused products of the feed-forward operators: operands that
// TMA cannot read are staged first, then one kernel runs.
#include <cstdint>
#include <cstdlib>
#include <cuda_runtime.h>

#include "api_common.h"
#include "kernels.h"
#include "ops.h"

namespace dg {
namespace {

// DGEMM_FUSED_*: an environment variable's value in lo .. hi, or -1 (read at
// every launch, for tests and tuning).
int knob(const char *name, int lo, int hi) {
  const char *e = getenv(name);
  if (e == nullptr || e[0] < '0' || e[0] > '9') return -1;
  const int v = atoi(e);
  return v >= lo && v <= hi ? v : -1;
}

// Whether a product runs on CTA pairs: once its 256-row tiles occupy a quarter
// of the SMs and more than one 256-column tile of tokens is there to fill
// them.  DGEMM_FUSED_PAIR=0 / =1 forces the choice.
bool use_pair(const FusedGemm &p, int num_sms) {
  if (p.K == 0) return false;  // the small kernel takes an empty sum
  const int force = knob("DGEMM_FUSED_PAIR", 0, 1);
  if (force >= 0) return force == 1;
  if (p.M <= 256) return false;
  const int tn = p.epi == Epi::kGated ? 128 : 256;
  const int64_t tiles = (int64_t)((p.M + 255) / 256) * ((p.N + tn - 1) / tn) *
                        (p.dual == Dual::kPair ? 2 : 1);
  return tiles * 4 >= num_sms;
}

// DGEMM_FUSED_NT / _KD / _SPLITS override the parts of the plan.
SmallPlan small_plan(const FusedGemm &p, int num_sms) {
  SmallPlan plan;
  const int step = p.a_t ? 64 : 16;
  plan.nt = p.M <= 256 ? (p.M + step - 1) / step * step : 128;
  const int nt = knob("DGEMM_FUSED_NT", 16, 256);
  if (nt >= 0) plan.nt = (nt + step - 1) / step * step;
  const int tf = p.epi == Epi::kGated ? 64 : 128;
  const int64_t tiles = (int64_t)((p.M + plan.nt - 1) / plan.nt) * ((p.N + tf - 1) / tf) *
                        (p.dual == Dual::kPair ? 2 : 1);
  plan.kd = plan.nt <= 32 && p.K > 64 ? 2 : 1;
  const int kd = knob("DGEMM_FUSED_KD", 1, 2);
  if (kd >= 0 && (kd == 1 || plan.nt <= 64)) plan.kd = kd;
  const int kblocks = (p.K + 64 * plan.kd - 1) / (64 * plan.kd) * (p.dual == Dual::kSum ? 2 : 1);
  const int64_t slots = (plan.nt <= 128 ? 2 : 1) * (int64_t)num_sms;
  int64_t s = slots / (tiles > 0 ? tiles : 1);
  s = s < 8 ? s : 8;
  s = s < kblocks / 2 ? s : kblocks / 2;
  plan.splits = s < 1 ? 1 : (int)s;
  const int splits = knob("DGEMM_FUSED_SPLITS", 1, 8);
  if (splits >= 0) plan.splits = splits;
  return plan;
}

}  // namespace

cudaError_t launch_fused(const FusedGemm &p0, int num_sms, cudaStream_t stream) {
  FusedGemm p = p0;
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  Stager st(num_sms, stream);
  const int ar = p.a_t ? p.K : p.M, ac = p.a_t ? p.M : p.K;
  const int br = p.b_t ? p.N : p.K, bc = p.b_t ? p.K : p.N;
  st.add(p.A, p.lda, ar, ac);
  st.add(p.B, p.ldb, br, bc);
  if (p.dual == Dual::kSum || p.dual == Dual::kPair) st.add(p.A2, p.lda2, ar, ac);
  if (p.dual != Dual::kNone) st.add(p.B2, p.ldb2, br, bc);
  cudaError_t e = st.run();
  if (e == cudaSuccess) {
    const int unit = p.a_t ? 2 : p.b_t ? 1 : 0;
    if (p.a_t && p.b_t) {
      e = cudaErrorInvalidValue;
    } else if (use_pair(p, num_sms)) {
      e = unit == 0   ? launch_fused_pair_unit_0(p, wd, stream)
          : unit == 1 ? launch_fused_pair_unit_1(p, wd, stream)
                      : launch_fused_pair_unit_2(p, wd, stream);
    } else {
      const SmallPlan plan = small_plan(p, num_sms);
      e = unit == 0   ? launch_fused_small_unit_0(p, plan, wd, stream)
          : unit == 1 ? launch_fused_small_unit_1(p, plan, wd, stream)
                      : launch_fused_small_unit_2(p, plan, wd, stream);
    }
  }
  const cudaError_t e2 = st.release();
  return e == cudaSuccess ? e2 : e;
}

// ------------------------------------------------------------------ Stager
void Stager::add(const void *&p, int64_t &ld, int64_t rows, int64_t cols) {
  if (p == nullptr || rows == 0 || cols == 0 || tma_ok(p, ld, 2) || n_ == kMax) return;
  items_[n_++] = {&p, &ld, rows, cols};
}

cudaError_t Stager::run() {
  if (n_ == 0) return cudaSuccess;
  const int n = n_;
  n_ = 0;
  RepitchJob jobs[kMax];
  int njobs = 0, job_of[kMax];
  size_t at[kMax], total = 0;
  for (int i = 0; i < n; ++i) {
    const Item &x = items_[i];
    int j = 0;
    while (j < njobs && !(jobs[j].src == *x.p && jobs[j].lds == *x.ld && jobs[j].rows == x.rows &&
                          jobs[j].cols == x.cols))
      ++j;
    job_of[i] = j;
    if (j < njobs) continue;  // given twice, staged once
    const int64_t pitch = (x.cols + 7) / 8 * 8;
    jobs[njobs++] = {*x.p, *x.ld, nullptr, pitch, x.rows, x.cols};
    at[j] = total;
    total += (size_t)(x.rows * pitch * 2 + 255) / 256 * 256;
  }
  cudaError_t e = scratch_alloc(&scratch_, total, stream_);
  if (e != cudaSuccess) {
    scratch_ = nullptr;
    return e;
  }
  for (int j = 0; j < njobs; ++j) jobs[j].dst = static_cast<char *>(scratch_) + at[j];
  for (int i = 0; i < n; ++i) {
    *items_[i].p = jobs[job_of[i]].dst;
    *items_[i].ld = jobs[job_of[i]].ldd;
  }
  return launch_repitch(jobs, njobs, num_sms_, stream_);
}

cudaError_t Stager::release() {
  if (scratch_ == nullptr) return cudaSuccess;
  void *s = scratch_;
  scratch_ = nullptr;
  return scratch_free(s, stream_);
}

}  // namespace dg
