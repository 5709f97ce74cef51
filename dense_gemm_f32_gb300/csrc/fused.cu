// fused.cu -- the fused products of the feed-forward operators: operands that
// TMA cannot read are staged first, then one kernel runs.
#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <new>
#include <cuda_runtime.h>

#include "../../include/dgemm.h"
#include "api_common.h"
#include "kernels.h"
#include "ops.h"

namespace dg {

namespace {

// one(splits, per_sm): the tiles of a kernel.
template <class F>
const Residency *made_once(std::atomic<const Residency *> (&made)[64], F &&one) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  const Residency *r = made[dev].load(std::memory_order_acquire);
  if (r == nullptr) {
    Residency *mine = new (std::nothrow) Residency;
    if (mine == nullptr) return nullptr;
    for (int per_sm = 1; per_sm <= 2; ++per_sm)
      for (int s = 1; s <= 8; ++s) mine->tiles[per_sm][s] = one(s, per_sm);
    if (made[dev].compare_exchange_strong(r, mine, std::memory_order_acq_rel))
      r = mine;
    else
      delete mine;
  }
  return r;
}

}  // namespace

const Residency *residency(int num_sms) {
  static std::atomic<const Residency *> made[64] = {};
  return made_once(made, [&](int s, int per_sm) { return small_resident({16, 1, s, per_sm}, num_sms); });
}

const Residency *int8_residency(int num_sms) {
  static std::atomic<const Residency *> made[64] = {};
  return made_once(made, [&](int s, int per_sm) { return int8_small_resident(s, per_sm, num_sms); });
}

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
// writing its outputs; the gate gradient's last epilogue shows, and inputs that
// do not come by TMA cost it 15%.
double pair_time(const FusedGemm &p, int num_sms) {
  const int tn = p.epi == Epi::kGated ? 128 : 256;
  const int64_t products = p.dual == Dual::kPair ? 2 : 1;
  const int64_t tiles = (int64_t)((p.M + 255) / 256) * ((p.N + tn - 1) / tn) * products;
  const int64_t waves = (tiles + num_sms / 2 - 1) / (num_sms / 2);
  const int kblocks = (p.K + 63) / 64 * (p.dual == Dual::kSum ? 2 : 1);
  const int outs = p.dual == Dual::kPair ? 1 : (p.out0 != nullptr) + (p.out1 != nullptr) + (p.out2 != nullptr);
  const double written = 2.0 * (double)p.M * p.N * outs * products;
  const double main = waves * (kblocks * 0.31), out = written / 2.4e6;
  if (p.epi != Epi::kGatedBwd) return 6.1 + (main > out ? main : out);
  const bool in_tma = tma_ok(p.in0, p.ldi0, 2) && tma_ok(p.in1, p.ldi1, 2);
  return (13 + (main > out ? main : out)) * (in_tma ? 1.0 : 1.15);
}

// Small kernel: a stage costs a CTA its wait (0.197 us, and 0.959 us shared by
// the stages in flight), its bytes at 96 GB/s, or its share of the SM's 312
// GB/s when two run there; all together at most 17.8 TB/s from L2; a tile's
// drain and epilogue grow with its tokens, and joining the parts of a K split
// costs 1.6 us, and with two CTAs per SM, whose clusters join at different
// times, 0.05 us more per token (1 x 4096 x 14336: 21.5 us in 4 parts, 20.1 in
// 8; 64 x 4096 x 14336: 24.1 and 26.7).  The gate gradient's epilogue, shared
// by the parts, is three times a linear layer's (5136 x 3408 x 784 on 128-token
// tiles: 69 us, 45 without the term; the pair kernel 55).
// `tiles` of this product among `all` of the launch.
double small_time(const FusedGemm &p, int64_t tiles, int64_t kblocks, const SmallPlan &plan,
                  int64_t resident, int64_t all) {
  const double nt = plan.nt, share = plan.per_sm, stage = (128 + nt) * 128 * plan.kd;
  const int64_t parts = (kblocks + plan.splits - 1) / plan.splits;
  const int64_t waves = (all + resident - 1) / resident;
  double per = 0.959 / small_stages(plan) + 0.197;
  if (per < stage / 96.2e3) per = stage / 96.2e3;
  if (per < stage * share / 312e3) per = stage * share / 312e3;
  const double loads = waves * (2.18 + parts * per);
  const double l2 = parts * stage * (all > tiles ? all : tiles) * plan.splits / 17.8e6;
  double tail = plan.splits > 1 ? 0.0283 * nt + 1.61 : 0.0124 * nt;
  if (plan.splits > 1 && plan.per_sm == 2) tail += 0.05 * (p.M < plan.nt ? p.M : plan.nt);
  if (p.epi == Epi::kGatedBwd) tail += 0.037 * nt / plan.splits;
  return 1.27 + (loads > l2 ? loads : l2) + waves * (share > 1 ? 1.414 : 1.0) * tail;
}

int64_t tiles_of(const FusedGemm &p, int nt) {
  const int tf = p.epi == Epi::kGated ? 64 : 128;
  return (int64_t)((p.N + tf - 1) / tf) * ((p.M + nt - 1) / nt) * (p.dual == Dual::kPair ? 2 : 1);
}
int64_t kblocks_of(const FusedGemm &p, int kd) {
  return (int64_t)((p.K + 64 * kd - 1) / (64 * kd)) * (p.dual == Dual::kSum ? 2 : 1);
}

// The best cut of `n` products as one launch of the small kernel, and its time.
// Token counts tried are the same for all, each product's cut down to its own;
// stages hold 128 k where two of them fit beside another CTA's.
// DGEMM_FUSED_NT / _KD / _SPLITS force parts of the cut.
double small_plan(const FusedGemm *ps, int n, const Residency &res, SmallPlan *best_plans) {
  const int f_nt = knob("DGEMM_FUSED_NT", 16, 256), f_kd = knob("DGEMM_FUSED_KD", 1, 2);
  const int f_splits = knob("DGEMM_FUSED_SPLITS", 1, 8);
  double best = 0;
  for (int cap : {16, 32, 48, 64, 96, 128, 192, 256}) {
    SmallPlan plans[kMaxBatch];
    int64_t tiles = 0, kmax = 0;
    int widest = 0;
    bool last = true;
    for (int j = 0; j < n; ++j) {
      const int step = ps[j].a_t ? 64 : 16, all = (ps[j].M + step - 1) / step * step;
      int nt = ((f_nt >= 0 ? f_nt : cap) + step - 1) / step * step;
      if (f_nt < 0 && nt > all) nt = all;
      last = last && nt >= all;
      const int kd = f_kd == 1 || nt > 64 || (f_kd < 0 && ps[j].K <= 64) ? 1 : 2;
      plans[j] = {nt, kd, 1, 1};
      tiles += tiles_of(ps[j], nt);
      const int64_t kb = kblocks_of(ps[j], kd);
      kmax = kmax > kb ? kmax : kb;
      widest = widest > nt ? widest : nt;
    }
    for (int s : {1, 2, 3, 4, 6, 8}) {
      if (f_splits >= 0) s = f_splits;
      else if (s > 1 && s > kmax) break;
      // all of an SM's shared memory for one CTA's stages where that holds every
      // tile at once
      for (int j = 0; j < n; ++j) plans[j].splits = s, plans[j].per_sm = 1;
      int64_t resident = res.tiles[1][s];
      if (tiles > resident && widest <= 128) {
        for (int j = 0; j < n; ++j) plans[j].per_sm = 2;
        resident = res.tiles[2][s];
      }
      double t = 0;
      for (int j = 0; j < n; ++j) {
        const double tj = small_time(ps[j], tiles_of(ps[j], plans[j].nt),
                                     kblocks_of(ps[j], plans[j].kd), plans[j], resident, tiles);
        t = t > tj ? t : tj;
      }
      if (best == 0 || t < best) {
        best = t;
        for (int j = 0; j < n; ++j) best_plans[j] = plans[j];
      }
      if (f_splits >= 0) break;
    }
    if (f_nt >= 0 || last) break;
  }
  return best;
}

cudaError_t run_pair(const FusedGemm &p, int *wd, cudaStream_t stream) {
  if (p.a_t) return p.b_t ? cudaErrorInvalidValue : launch_fused_pair_unit_2(p, wd, stream);
  return p.b_t ? launch_fused_pair_unit_1(p, wd, stream) : launch_fused_pair_unit_0(p, wd, stream);
}

cudaError_t run_small(const FusedGemm *p, const SmallPlan *plans, int n, int *wd,
                      cudaStream_t stream) {
  const bool half = p->dtype == DGEMM_DTYPE_F16, linear = p->epi == Epi::kLinear;
  return linear ? (half ? launch_fused_small_unit_1(p, plans, n, wd, stream)
                        : launch_fused_small_unit_0(p, plans, n, wd, stream))
                : (half ? launch_fused_small_unit_3(p, plans, n, wd, stream)
                        : launch_fused_small_unit_2(p, plans, n, wd, stream));
}

// DGEMM_FUSED_PAIR=0 / =1 forces the kernel; an empty sum is the small one's.
int forced_kernel(const FusedGemm &p) {
  return p.K == 0 ? 0 : knob("DGEMM_FUSED_PAIR", 0, 1);
}

void stage_operands(Stager &st, FusedGemm &p) {
  const int ar = p.a_t ? p.K : p.M, ac = p.a_t ? p.M : p.K;
  const int br = p.b_t ? p.N : p.K, bc = p.b_t ? p.K : p.N;
  st.add(p.A, p.lda, ar, ac);
  st.add(p.B, p.ldb, br, bc);
  if (p.dual == Dual::kSum || p.dual == Dual::kPair) st.add(p.A2, p.lda2, ar, ac);
  if (p.dual != Dual::kNone) st.add(p.B2, p.ldb2, br, bc);
}

}  // namespace

cudaError_t launch_fused_batch(const FusedGemm *ps, int n, int num_sms, cudaStream_t stream) {
  if (n < 1 || n > kMaxBatch) return n == 0 ? cudaSuccess : cudaErrorInvalidValue;
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  const Residency *table = residency(num_sms);
  if (table == nullptr) return cudaErrorInvalidDevice;
  const Residency &res = *table;
  FusedGemm p[kMaxBatch];
  Stager st(num_sms, stream);
  for (int j = 0; j < n; ++j) {
    p[j] = ps[j];
    stage_operands(st, p[j]);
  }
  cudaError_t e = st.run();
  if (e == cudaSuccess) {
    // each by itself, on the kernel that is quicker for it
    SmallPlan alone[kMaxBatch], together[kMaxBatch];
    bool pair[kMaxBatch];
    double sum = 0;
    for (int j = 0; j < n; ++j) {
      const int force = forced_kernel(p[j]);
      const double small = small_plan(&p[j], 1, res, &alone[j]);
      const double big = pair_time(p[j], num_sms);
      pair[j] = force >= 0 ? force == 1 : big < small;
      sum += pair[j] ? big : small;
    }
    // DGEMM_FUSED_BATCH=0 / =1 forces the choice
    const int force = knob("DGEMM_FUSED_BATCH", 0, 1);
    const bool batch = n > 1 && force != 0 &&
                       (small_plan(p, n, res, together) < sum || force == 1);
    if (batch) {
      e = run_small(p, together, n, wd, stream);
    } else {
      for (int j = 0; j < n && e == cudaSuccess; ++j)
        e = pair[j] ? run_pair(p[j], wd, stream) : run_small(&p[j], &alone[j], 1, wd, stream);
    }
  }
  const cudaError_t e2 = st.release();
  return e == cudaSuccess ? e2 : e;
}

cudaError_t launch_fused(const FusedGemm &p, int num_sms, cudaStream_t stream) {
  return launch_fused_batch(&p, 1, num_sms, stream);
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
