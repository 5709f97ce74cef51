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

// Time models (microseconds), fitted to 250 calls of 1 to 4096 tokens with every cut
// on GB300, in a graph with weights rotating through more than L2.  What they choose
// took 1.03 times the best cut's time on average and 1.21 at worst.
//
// Pair kernel: a block of 128 k takes a wave of tiles its MMAs' time, or that of the
// hand-overs between converters and MMA.
double pair_time(const Int8Gemm &p, int nt, int num_sms) {
  const int tf = p.gated ? 128 : 256;
  const int64_t tiles = (int64_t)((p.N + tf - 1) / tf) * ((p.M + nt - 1) / nt);
  const int64_t waves = (tiles + num_sms / 2 - 1) / (num_sms / 2);
  const double sync = 0.26 + 0.00056 * nt, mma = 0.0024 * nt;
  const double main = (double)waves * ((p.K + 127) / 128 * (sync > mma ? sync : mma) + 0.53);
  const double weights = (double)p.N * p.K * (p.gated ? 2 : 1) / 6.9e6;
  return 5.3 + 0.0056 * nt + (main > weights ? main : weights);
}

// Small kernel: a block takes a CTA its chain of hand-overs, or its bytes' time at
// an SM's 135 GB/s (101 where two CTAs share it); the epilogue 0.054 per token of a tile,
// and joining the parts of a K split 0.72 for each.
double small_time(const Int8Gemm &p, const Int8Plan &plan, const Residency &res, int num_sms) {
  const int tf = p.gated ? 64 : 128;
  const int64_t tiles_t = (p.M + plan.nt - 1) / plan.nt;
  const int64_t ctas = (int64_t)((p.N + tf - 1) / tf) * tiles_t * plan.splits;
  const int64_t slots = res.tiles[plan.per_sm][plan.splits] * plan.splits;
  const int64_t waves = (ctas + slots - 1) / slots;
  const int64_t blocks = ((p.K + 127) / 128 + plan.splits - 1) / plan.splits;
  const bool two = (ctas < slots ? ctas : slots) > num_sms;  // on the fullest SM
  const double bytes = (16384.0 + 256.0 * plan.nt) * (two ? 2 / 101e3 : 1 / 135e3);
  const double stream = (double)(waves * blocks) * (bytes > 0.36 ? bytes : 0.36);
  const double weights = (double)p.N * p.K * (p.gated ? 2 : 1) * (double)tiles_t / 6.9e6;
  return 3.0 + (stream > weights ? stream : weights) + 0.054 * (double)(waves * plan.nt) +
         3.8 * (double)(waves - 1) + (plan.splits > 1 ? 0.72 * plan.splits : 0.);
}

// The best cut of each kernel; DGEMM_INT8_NT / _SPLITS force parts of it.
double small_plan(const Int8Gemm &p, const Residency &res, int num_sms, Int8Plan *best_plan) {
  const int f_nt = knob("DGEMM_INT8_NT", 16, 128), f_splits = knob("DGEMM_INT8_SPLITS", 1, 8);
  const int64_t kblocks = (p.K + 127) / 128;
  double best = 0;
  for (int cap : {16, 32, 48, 64, 96, 128}) {
    const int all = (p.M + 15) / 16 * 16;
    Int8Plan plan = {f_nt >= 0 ? (f_nt + 15) / 16 * 16 : cap < all ? cap : all, 1, 1};
    for (int s : {1, 2, 3, 4, 6, 8}) {
      if (f_splits >= 0) s = f_splits;
      else if (s > 1 && s > kblocks) break;
      plan.splits = s;
      const int tf = p.gated ? 64 : 128;
      const int64_t tiles = (int64_t)((p.N + tf - 1) / tf) * ((p.M + plan.nt - 1) / plan.nt);
      // all of an SM's shared memory for one CTA's stages where that holds every tile at once
      plan.per_sm = tiles > res.tiles[1][s] ? 2 : 1;
      const double t = small_time(p, plan, res, num_sms);
      if (best == 0 || t < best) best = t, *best_plan = plan;
      if (f_splits >= 0) break;
    }
    if (f_nt >= 0 || cap >= all) break;
  }
  return best;
}

double pair_plan(const Int8Gemm &p, int num_sms, int *best_nt) {
  const int f_nt = knob("DGEMM_INT8_NT", 32, 192);
  double best = 0;
  for (int nt = 32; nt <= 192; nt += 32) {
    if (f_nt >= 0) nt = (f_nt + 31) / 32 * 32;
    const double t = pair_time(p, nt, num_sms);
    if (best == 0 || t < best) best = t, *best_nt = nt;
    if (f_nt >= 0) break;
  }
  return best;
}

}  // namespace

bool int8_use_row(const Int8Gemm *p, int n, int num_sms) {
  const int force = knob("DGEMM_INT8_ROW", 0, 1);
  for (int i = 0; i < n; ++i)
    if (!int8_row_takes(p[i].M, p[i].K)) return false;
  const Residency *res = int8_residency(num_sms);
  if (force == 0 || res == nullptr) return false;
  double row = 0, other = 0;
  for (int i = 0; i < n; ++i) {
    row += int8_row_time(p[i]);
    Int8Plan plan;
    other += small_plan(p[i], *res, num_sms, &plan) + 3.0;  // the tokens' kernel
    // the copy of weights on other than 16-byte boundaries
    const int mats = p[i].gated ? 2 : 1;
    if (!rows_aligned(p[i].W, p[i].ldw, 1)) other += 1.0 + (double)p[i].N * p[i].K * mats / 3.5e6;
  }
  return force == 1 || row < other;
}

cudaError_t launch_int8(const Int8Gemm &p, int num_sms, cudaStream_t stream) {
  int *wd = watchdog_address();
  if (wd == nullptr) return cudaErrorInvalidSymbol;
  const Residency *res = int8_residency(num_sms);
  if (res == nullptr) return cudaErrorInvalidDevice;
  Int8Plan plan;
  int nt = 0;
  const double small = small_plan(p, *res, num_sms, &plan), pair = pair_plan(p, num_sms, &nt);
  // DGEMM_INT8_PAIR=0 / =1 forces the kernel; an empty sum is the small one's
  const int force = p.K > 0 ? knob("DGEMM_INT8_PAIR", 0, 1) : 0;
  return (force >= 0 ? force == 1 : pair < small) ? launch_int8_pair(p, nt, wd, stream)
                                                  : launch_int8_small(p, plan, wd, stream);
}

}  // namespace dg
