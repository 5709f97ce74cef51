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

// Time models (microseconds) of the two kernels, fitted to 50 shapes of one to
// 16384 tokens with every cut of the small kernel on GB300, in a graph with
// operands rotating through more than L2.  Choosing by them is within 2% of
// the best cut on average (1.13 times at worst); 256-row tiles once they fill a
// quarter of the SMs, and 128-token tiles below that, were 30% off on average.
//
// Pair kernel: a wave of 256 x 256 tiles takes 0.31 us per 64 k, or as long as
// writing its outputs.
double pair_time(const FusedGemm &p, int num_sms) {
  const int tn = p.epi == Epi::kGated ? 128 : 256;
  const int64_t products = p.dual == Dual::kPair ? 2 : 1;
  const int64_t tiles = (int64_t)((p.M + 255) / 256) * ((p.N + tn - 1) / tn) * products;
  const int64_t waves = (tiles + num_sms / 2 - 1) / (num_sms / 2);
  const int kblocks = (p.K + 63) / 64 * (p.dual == Dual::kSum ? 2 : 1);
  const int outs = p.dual == Dual::kPair ? 1 : (p.out0 != nullptr) + (p.out1 != nullptr) + (p.out2 != nullptr);
  const double written = 2.0 * (double)p.M * p.N * outs * products;
  const double main = waves * (kblocks * 0.31), out = written / 2.4e6;
  return 6.1 + (main > out ? main : out);
}

// Small kernel: a stage costs a CTA its wait (0.197 us, and 0.959 us shared by
// the stages in flight), its bytes at 96 GB/s, or its share of the SM's 312
// GB/s when two run there; all together at most 17.8 TB/s from L2; a tile's
// drain and epilogue grow with its tokens, and joining the parts of a K split
// costs 1.6 us.
double small_time(int64_t tiles, int64_t kblocks, const SmallPlan &plan, int64_t resident) {
  const double nt = plan.nt, share = plan.per_sm, stage = (128 + nt) * 128 * plan.kd;
  const int64_t parts = (kblocks + plan.splits - 1) / plan.splits;
  const int64_t waves = (tiles + resident - 1) / resident;
  double per = 0.959 / small_stages(plan) + 0.197;
  if (per < stage / 96.2e3) per = stage / 96.2e3;
  if (per < stage * share / 312e3) per = stage * share / 312e3;
  const double loads = waves * (2.18 + parts * per);
  const double l2 = parts * stage * tiles * plan.splits / 17.8e6;
  const double tail = plan.splits > 1 ? 0.0283 * nt + 1.61 : 0.0124 * nt;
  return 1.27 + (loads > l2 ? loads : l2) + waves * (share > 1 ? 1.414 : 1.0) * tail;
}

// The kernel and its cut for a product.  DGEMM_FUSED_PAIR=0 / =1 forces the
// kernel, DGEMM_FUSED_NT / _KD / _SPLITS parts of the small kernel's cut.
struct Choice {
  bool pair;
  SmallPlan plan;
};
Choice choose(const FusedGemm &p, int num_sms) {
  const int force = p.K == 0 ? 0 : knob("DGEMM_FUSED_PAIR", 0, 1);  // an empty sum is the small one's
  Choice c = {force == 1, {}};
  if (c.pair) return c;
  const int f_nt = knob("DGEMM_FUSED_NT", 16, 256), f_kd = knob("DGEMM_FUSED_KD", 1, 2);
  const int f_splits = knob("DGEMM_FUSED_SPLITS", 1, 8);
  const int step = p.a_t ? 64 : 16, tf = p.epi == Epi::kGated ? 64 : 128;
  const int64_t tiles_f = (int64_t)((p.N + tf - 1) / tf) * (p.dual == Dual::kPair ? 2 : 1);
  double best = 0;
  for (int nt : {16, 32, 48, 64, 96, 128, 192, 256}) {
    if (f_nt >= 0) nt = f_nt;
    nt = (nt + step - 1) / step * step;
    const int64_t tiles = tiles_f * ((p.M + nt - 1) / nt);
    // stages of 128 k where two of them fit beside another CTA's
    const int kd = f_kd == 1 || nt > 64 || (f_kd < 0 && p.K <= 64) ? 1 : 2;
    const int64_t kblocks = (int64_t)((p.K + 64 * kd - 1) / (64 * kd)) * (p.dual == Dual::kSum ? 2 : 1);
    for (int s : {1, 2, 3, 4, 6, 8}) {
      if (f_splits >= 0) s = f_splits;
      else if (s > 1 && s > kblocks) break;
      // all of an SM's shared memory for one CTA's stages where that holds every
      // tile at once
      SmallPlan plan = {nt, kd, s, 1};
      int64_t resident = small_resident(plan, num_sms);
      if (tiles > resident && nt <= 128) {
        plan.per_sm = 2;
        resident = small_resident(plan, num_sms);
      }
      const double t = small_time(tiles, kblocks, plan, resident);
      if (best == 0 || t < best) {
        best = t;
        c.plan = plan;
      }
      if (f_splits >= 0) break;
    }
    if (f_nt >= 0 || nt >= p.M) break;
  }
  if (force < 0) c.pair = pair_time(p, num_sms) < best;
  return c;
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
    } else {
      const Choice c = choose(p, num_sms);
      if (c.pair)
        e = unit == 0   ? launch_fused_pair_unit_0(p, wd, stream)
            : unit == 1 ? launch_fused_pair_unit_1(p, wd, stream)
                        : launch_fused_pair_unit_2(p, wd, stream);
      else
        e = unit == 0   ? launch_fused_small_unit_0(p, c.plan, wd, stream)
            : unit == 1 ? launch_fused_small_unit_1(p, c.plan, wd, stream)
                        : launch_fused_small_unit_2(p, c.plan, wd, stream);
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
