// ops_api.cu -- the exported feed-forward operators: argument validation and
// the launches each call is made of.
//
// The order of checks is that of the GEMM entry points (api.cu):
//   1. element type, activation, weight layout        -> DGEMM_ERR_UNSUPPORTED
//   2. sizes, leading dimensions, eps                 -> DGEMM_ERR_INVALID_VALUE
//   3. nothing to write                               -> DGEMM_OK, nothing launched
//   4. NULL for a matrix that is not optional         -> DGEMM_ERR_NULL_POINTER
//   5. pointer alignment to the element size          -> DGEMM_ERR_MISALIGNED
//   6. an output overlapping another argument         -> DGEMM_ERR_ALIAS
//   7. current device is compute capability 10.3      -> DGEMM_ERR_ARCH / DGEMM_ERR_CUDA
//   8. every pointer is device memory of this device  -> DGEMM_ERR_INVALID_POINTER
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <cuda_runtime.h>

#include "../../include/dgemm.h"
#include "api_common.h"
#include "kernels.h"
#include "ops.h"

namespace {

using namespace dg;

// One matrix (or vector, rows = 1) argument of a call.
struct Arg {
  const void *p;
  int64_t rows, cols, ld;
  int es;
  bool out;
  bool optional;
};

// A vector of n elements.
Arg vec(const void *p, int n, int es, bool out) {
  return {p, 1, n, n > 1 ? n : 1, es, out, true};
}

bool ok_dtype(int dtype, bool f32) {
  return dtype == DGEMM_DTYPE_BF16 || dtype == DGEMM_DTYPE_F16 || (f32 && dtype == DGEMM_DTYPE_F32);
}
bool ok_act(int act) { return act >= DGEMM_ACT_NONE && act <= DGEMM_ACT_SILU; }
bool ok_op(int op) { return op == DGEMM_OP_N || op == DGEMM_OP_T; }
int elem_bytes(int dtype) { return dtype == DGEMM_DTYPE_F32 ? 4 : 2; }

// Step 2 for the sizes that the kernels count in 32 bits: a round-up to whole
// tiles or vectors, and a step past the end, stay below 2^31.
bool ok_counts(std::initializer_list<int> sizes) {
  for (int n : sizes)
    if (n > DGEMM_OPS_MAX_SIZE) return false;
  return true;
}

// Step 2 for the matrices (an absent optional one is not looked at).
bool ok_sizes(const Arg *a, int n) {
  for (int i = 0; i < n; ++i) {
    if (a[i].rows < 0 || a[i].cols < 0) return false;
    if (a[i].p == nullptr && a[i].optional) continue;
    if (a[i].ld < (a[i].cols > 1 ? a[i].cols : 1)) return false;
  }
  return true;
}

// Steps 4-8.  Output number in_place_out may coincide exactly (same address and
// leading dimension) with input number in_place_in; -1, -1 for none.
int check_args(const Arg *a, int n, int in_place_out, int in_place_in, int *dev, int *num_sms) {
  auto empty = [&](int i) { return a[i].rows == 0 || a[i].cols == 0; };
  for (int i = 0; i < n; ++i)
    if (a[i].p == nullptr && !a[i].optional && !empty(i)) return DGEMM_ERR_NULL_POINTER;
  for (int i = 0; i < n; ++i)
    if (a[i].p != nullptr && !empty(i) && !aligned(a[i].p, a[i].es)) return DGEMM_ERR_MISALIGNED;
  auto sp = [&](int i) { return span(a[i].p, a[i].rows, a[i].cols, a[i].ld, a[i].es); };
  for (int i = 0; i < n; ++i) {
    if (!a[i].out || a[i].p == nullptr) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || a[j].p == nullptr) continue;
      if (i == in_place_out && j == in_place_in && a[i].p == a[j].p && a[i].ld == a[j].ld) continue;
      if (overlap(sp(i), sp(j))) return DGEMM_ERR_ALIAS;
    }
  }
  int st = current_device(dev, num_sms);
  if (st != DGEMM_OK) return st;
  for (int i = 0; i < n; ++i)
    if (a[i].p != nullptr && !empty(i) && (st = check_device_pointer(a[i].p, *dev)) != DGEMM_OK)
      return st;
  return DGEMM_OK;
}

int done(cudaError_t e, const char *what) { return e == cudaSuccess ? DGEMM_OK : cuda_fail(e, what); }

// fp32 scratch around a launch: f(scratch) enqueues the work.
template <class F>
int with_scratch(size_t bytes, cudaStream_t stream, const char *what, F &&f) {
  void *s = nullptr;
  if (bytes) {
    const cudaError_t e = scratch_alloc(&s, bytes, stream);
    if (e != cudaSuccess) return cuda_fail(e, "scratch allocation (column sums)");
  }
  const int st = done(f(static_cast<float *>(s)), what);
  if (s != nullptr) {
    const cudaError_t e = scratch_free(s, stream);
    if (st == DGEMM_OK && e != cudaSuccess) return cuda_fail(e, "scratch release");
  }
  return st;
}

// The end of a call that staged operands.
int release(Stager &stage, int st) {
  const cudaError_t e = stage.release();
  return st == DGEMM_OK ? done(e, "scratch release") : st;
}

}  // namespace

extern "C" {

int dgemm_layer_norm(int dtype, int rows, int cols, float eps, const void *X, int ldx,
                     const void *weight, const void *bias, void *Y, int ldy, float *mean,
                     float *rstd, cudaStream_t stream) {
  if (!ok_dtype(dtype, true)) return DGEMM_ERR_UNSUPPORTED;
  const int es = elem_bytes(dtype);
  const Arg a[] = {{X, rows, cols, ldx, es, false, false}, vec(weight, cols, es, false),
                   vec(bias, cols, es, false),   {Y, rows, cols, ldy, es, true, false},
                   vec(mean, rows, 4, true),     vec(rstd, rows, 4, true)};
  if (!ok_counts({cols}) || !ok_sizes(a, 4) || !(eps >= 0.f) || std::isinf(eps))
    return DGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return DGEMM_OK;
  int dev = 0, sms = 0;
  const int st = check_args(a, 6, -1, -1, &dev, &sms);
  if (st != DGEMM_OK) return st;
  return done(launch_layer_norm(dtype, rows, cols, eps, X, ldx, weight, bias, Y, ldy, mean, rstd,
                                stream),
              "layer norm launch");
}

int dgemm_layer_norm_backward(int dtype, int rows, int cols, const void *dY, int lddy,
                              const void *X, int ldx, const void *weight, const float *mean,
                              const float *rstd, const void *dR, int lddr, void *dX, int lddx,
                              void *dweight, void *dbias, cudaStream_t stream) {
  if (!ok_dtype(dtype, true)) return DGEMM_ERR_UNSUPPORTED;
  const int es = elem_bytes(dtype);
  const Arg a[] = {{dY, rows, cols, lddy, es, false, false}, {X, rows, cols, ldx, es, false, false},
                   vec(weight, cols, es, false), {mean, 1, rows, rows, 4, false, false},
                   {rstd, 1, rows, rows, 4, false, false},   {dR, rows, cols, lddr, es, false, true},
                   {dX, rows, cols, lddx, es, true, false},  vec(dweight, cols, es, true),
                   vec(dbias, cols, es, true)};
  if (!ok_counts({cols})) return DGEMM_ERR_INVALID_VALUE;
  for (int i : {0, 1, 2, 5, 6, 7, 8})
    if (!ok_sizes(a + i, 1)) return DGEMM_ERR_INVALID_VALUE;
  if (cols == 0 || (rows == 0 && !dweight && !dbias)) return DGEMM_OK;
  int dev = 0, sms = 0;
  const int st = check_args(a, 9, -1, -1, &dev, &sms);
  if (st != DGEMM_OK) return st;
  return with_scratch(layer_norm_scratch(rows, cols, dweight || dbias, sms), stream,
                      "layer norm backward launch", [&](float *partial) {
                        return launch_layer_norm_backward(dtype, rows, cols, dY, lddy, X, ldx,
                                                          weight, mean, rstd, dR, lddr, dX, lddx,
                                                          dweight, dbias, partial, sms, stream);
                      });
}

int dgemm_linear(int dtype, int activation, int op_w, int M, int N, int K, const void *X, int ldx,
                 const void *W, int ldw, const void *bias, const void *R, int ldr, void *D,
                 int ldd, void *Z, int ldz, cudaStream_t stream) {
  if (!ok_dtype(dtype, false) || !ok_act(activation) || !ok_op(op_w)) return DGEMM_ERR_UNSUPPORTED;
  const bool t = op_w == DGEMM_OP_T;
  const int es = 2;
  const Arg a[] = {{X, M, K, ldx, es, false, false},
                   {W, t ? N : K, t ? K : N, ldw, es, false, false},
                   vec(bias, N, es, false),
                   {R, M, N, ldr, es, false, true},
                   {D, M, N, ldd, es, true, false},
                   {Z, M, N, ldz, es, true, true}};
  if (!ok_counts({M, N, K})) return DGEMM_ERR_INVALID_VALUE;
  for (int i : {0, 1, 3, 4, 5})
    if (!ok_sizes(a + i, 1)) return DGEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return DGEMM_OK;
  int dev = 0, sms = 0;
  const int st = check_args(a, 6, 4, 3, &dev, &sms);  // D may be R itself
  if (st != DGEMM_OK) return st;
  FusedGemm p;
  p.dtype = dtype, p.act = activation;
  p.M = M, p.N = N, p.K = K;
  p.A = X, p.lda = ldx, p.B = W, p.ldb = ldw, p.b_t = t;
  p.bias = bias, p.in0 = R, p.ldi0 = ldr;
  p.out0 = D, p.ldo0 = ldd, p.out1 = Z, p.ldo1 = ldz;
  return done(launch_fused(p, sms, stream), "linear launch");
}

int dgemm_linear_backward(int dtype, int activation, int op_w, int M, int N, int K, const void *dD,
                          int lddd, const void *X, int ldx, const void *W, int ldw, const void *Z,
                          int ldz, void *dZ, int lddz, void *dX, int lddx, void *dW, int lddw,
                          void *dbias, cudaStream_t stream) {
  if (!ok_dtype(dtype, false) || !ok_act(activation) || !ok_op(op_w)) return DGEMM_ERR_UNSUPPORTED;
  const bool t = op_w == DGEMM_OP_T, act = activation != DGEMM_ACT_NONE;
  const int es = 2, wr = t ? N : K, wc = t ? K : N;
  const Arg a[] = {{dD, M, N, lddd, es, false, false},
                   {X, M, K, ldx, es, false, dW == nullptr},
                   {W, wr, wc, ldw, es, false, dX == nullptr},
                   {act ? Z : nullptr, M, N, ldz, es, false, !act},
                   {act ? dZ : nullptr, M, N, lddz, es, true, !act},
                   {dX, M, K, lddx, es, true, true},
                   {dW, wr, wc, lddw, es, true, true},
                   vec(dbias, N, es, true)};
  if (!ok_counts({M, N, K})) return DGEMM_ERR_INVALID_VALUE;
  for (int i = 0; i < 7; ++i)
    if (!ok_sizes(a + i, 1)) return DGEMM_ERR_INVALID_VALUE;
  const bool want_dx = dX && M > 0 && K > 0, want_dw = dW && N > 0 && K > 0;
  const bool want_db = dbias && N > 0;
  if (!want_dx && !want_dw && !want_db) return DGEMM_OK;
  int dev = 0, sms = 0;
  int st = check_args(a, 8, -1, -1, &dev, &sms);
  if (st != DGEMM_OK) return st;
  if (N > 0 && (want_db || (act && M > 0))) {
    st = with_scratch(act_grad_scratch(M, N, want_db, sms), stream, "activation gradient launch",
                      [&](float *partial) {
                        return launch_act_grad(dtype, activation, M, N, dD, lddd, Z, ldz, dZ, lddz,
                                               want_db ? dbias : nullptr, partial, sms, stream);
                      });
    if (st != DGEMM_OK) return st;
  }
  // operands that TMA cannot read, all in one launch (dZ by its own product
  // when a caller's workspace is not aligned)
  const void *dz = act ? dZ : dD, *x = X, *w = W;
  int64_t ldz_use = act ? lddz : lddd, ldx_use = ldx, ldw_use = ldw;
  Stager stage(sms, stream);
  if (!act && (want_dx || want_dw)) stage.add(dz, ldz_use, M, N);
  if (want_dw) stage.add(x, ldx_use, M, K);
  if (want_dx) stage.add(w, ldw_use, wr, wc);
  if ((st = done(stage.run(), "operand staging")) != DGEMM_OK) return release(stage, st);
  FusedGemm ps[2];
  int n = 0;
  if (want_dx) {  // dX (M x K) = dZ op(W)^T
    FusedGemm &p = ps[n++];
    p.dtype = dtype;
    p.M = M, p.N = K, p.K = N;
    p.A = dz, p.lda = ldz_use, p.B = w, p.ldb = ldw_use, p.b_t = !t;
    p.out0 = dX, p.ldo0 = lddx;
  }
  if (want_dw) {  // dW as W is stored: X^T dZ, or its transpose dZ^T X
    FusedGemm &p = ps[n++];
    p.dtype = dtype;
    p.M = wr, p.N = wc, p.K = M;
    p.a_t = true;
    p.A = t ? dz : x, p.lda = t ? ldz_use : ldx_use;
    p.B = t ? x : dz, p.ldb = t ? ldx_use : ldz_use;
    p.out0 = dW, p.ldo0 = lddw;
  }
  return release(stage, done(launch_fused_batch(ps, n, sms, stream), "gradient launch"));
}

int dgemm_gated_ffn(int dtype, int activation, int op_w, int M, int D, int F, const void *X,
                    int ldx, const void *Wg, int ldwg, const void *Wu, int ldwu, const void *Wd,
                    int ldwd, const void *R, int ldr, void *H, int ldh, void *G, int ldg, void *U,
                    int ldu, void *Y, int ldy, cudaStream_t stream) {
  if (!ok_dtype(dtype, false) || !ok_act(activation) || !ok_op(op_w)) return DGEMM_ERR_UNSUPPORTED;
  const bool t = op_w == DGEMM_OP_T;
  const int es = 2, ur = t ? F : D, uc = t ? D : F;
  const Arg a[] = {{X, M, D, ldx, es, false, false},   {Wg, ur, uc, ldwg, es, false, false},
                   {Wu, ur, uc, ldwu, es, false, false}, {Wd, uc, ur, ldwd, es, false, false},
                   {R, M, D, ldr, es, false, true},    {H, M, F, ldh, es, true, false},
                   {G, M, F, ldg, es, true, U == nullptr}, {U, M, F, ldu, es, true, G == nullptr},
                   {Y, M, D, ldy, es, true, false}};
  if (!ok_counts({M, D, F}) || !ok_sizes(a, 9)) return DGEMM_ERR_INVALID_VALUE;
  if (M == 0 || (D == 0 && F == 0)) return DGEMM_OK;
  int dev = 0, sms = 0;
  int st = check_args(a, 9, 8, 4, &dev, &sms);  // Y may be R itself
  if (st != DGEMM_OK) return st;
  const void *x = X, *wg = Wg, *wu = Wu, *wd = Wd;
  int64_t lx = ldx, lg = ldwg, lu = ldwu, ld = ldwd;
  Stager stage(sms, stream);  // operands that TMA cannot read, in one launch
  if (F > 0) {
    stage.add(x, lx, M, D);
    stage.add(wg, lg, ur, uc);
    stage.add(wu, lu, ur, uc);
    if (D > 0) stage.add(wd, ld, uc, ur);
  }
  if ((st = done(stage.run(), "operand staging")) != DGEMM_OK) return release(stage, st);
  if (F > 0) {
    FusedGemm p;
    p.epi = Epi::kGated, p.dual = Dual::kGated;
    p.dtype = dtype, p.act = activation;
    p.M = M, p.N = F, p.K = D;
    p.A = x, p.lda = lx, p.b_t = t;
    p.B = wg, p.ldb = lg, p.B2 = wu, p.ldb2 = lu;
    p.out0 = H, p.ldo0 = ldh, p.out1 = G, p.ldo1 = ldg, p.out2 = U, p.ldo2 = ldu;
    st = done(launch_fused(p, sms, stream), "gated product launch");
  }
  if (st == DGEMM_OK && D > 0) {
    FusedGemm p;
    p.dtype = dtype;
    p.M = M, p.N = D, p.K = F;
    p.A = H, p.lda = ldh, p.B = wd, p.ldb = ld, p.b_t = t;
    p.in0 = R, p.ldi0 = ldr, p.out0 = Y, p.ldo0 = ldy;
    st = done(launch_fused(p, sms, stream), "down product launch");
  }
  return release(stage, st);
}

int dgemm_gated_ffn_backward(int dtype, int activation, int op_w, int M, int D, int F,
                             const void *dY, int lddy, const void *X, int ldx, const void *Wg,
                             int ldwg, const void *Wu, int ldwu, const void *Wd, int ldwd,
                             const void *G, int ldg, const void *U, int ldu, void *H, int ldh,
                             void *dG, int lddg, void *dU, int lddu, void *dX, int lddx, void *dWg,
                             int lddwg, void *dWu, int lddwu, void *dWd, int lddwd,
                             cudaStream_t stream) {
  if (!ok_dtype(dtype, false) || !ok_act(activation) || !ok_op(op_w)) return DGEMM_ERR_UNSUPPORTED;
  const bool t = op_w == DGEMM_OP_T;
  const int es = 2, ur = t ? F : D, uc = t ? D : F;
  const Arg a[] = {{dY, M, D, lddy, es, false, false},  {X, M, D, ldx, es, false, false},
                   {Wg, ur, uc, ldwg, es, false, false}, {Wu, ur, uc, ldwu, es, false, false},
                   {Wd, uc, ur, ldwd, es, false, false}, {G, M, F, ldg, es, false, false},
                   {U, M, F, ldu, es, false, false},    {H, M, F, ldh, es, true, false},
                   {dG, M, F, lddg, es, true, false},   {dU, M, F, lddu, es, true, false},
                   {dX, M, D, lddx, es, true, true},    {dWg, ur, uc, lddwg, es, true, dWu == nullptr},
                   {dWu, ur, uc, lddwu, es, true, dWg == nullptr},
                   {dWd, uc, ur, lddwd, es, true, true}};
  if (!ok_counts({M, D, F}) || !ok_sizes(a, 14)) return DGEMM_ERR_INVALID_VALUE;
  const bool want_dx = dX && M > 0, want_up = dWg && F > 0, want_down = dWd && F > 0;
  if (D == 0 || (!want_dx && !want_up && !want_down)) return DGEMM_OK;
  int dev = 0, sms = 0;
  int st = check_args(a, 14, -1, -1, &dev, &sms);
  if (st != DGEMM_OK) return st;
  const void *dy = dY, *x = X, *wg = Wg, *wu = Wu, *wd = Wd;
  int64_t ly = lddy, lx = ldx, lg = ldwg, lu = ldwu, ld = ldwd;
  Stager stage(sms, stream);  // operands that TMA cannot read, in one launch
  if (M > 0 && F > 0) {
    stage.add(dy, ly, M, D);
    stage.add(wd, ld, uc, ur);
    if (want_up) stage.add(x, lx, M, D);
    if (want_dx) {
      stage.add(wg, lg, ur, uc);
      stage.add(wu, lu, ur, uc);
    }
  }
  if ((st = done(stage.run(), "operand staging")) != DGEMM_OK) return release(stage, st);
  if (M > 0 && F > 0) {  // dh = dY op(Wd)^T in the accumulator -> dG, dU, H
    FusedGemm p;
    p.epi = Epi::kGatedBwd;
    p.dtype = dtype, p.act = activation;
    p.M = M, p.N = F, p.K = D;
    p.A = dy, p.lda = ly, p.B = wd, p.ldb = ld, p.b_t = !t;
    p.in0 = G, p.ldi0 = ldg, p.in1 = U, p.ldi1 = ldu;
    p.out0 = dG, p.ldo0 = lddg, p.out1 = dU, p.ldo1 = lddu, p.out2 = H, p.ldo2 = ldh;
    st = done(launch_fused(p, sms, stream), "gate gradient launch");
  }
  if (st != DGEMM_OK) return release(stage, st);
  FusedGemm ps[3];
  int n = 0;
  if (want_dx) {  // dX = dG op(Wg)^T + dU op(Wu)^T
    FusedGemm &p = ps[n++];
    p.dual = Dual::kSum;
    p.dtype = dtype;
    p.M = M, p.N = D, p.K = F;
    p.A = dG, p.lda = lddg, p.A2 = dU, p.lda2 = lddu, p.b_t = !t;
    p.B = wg, p.ldb = lg, p.B2 = wu, p.ldb2 = lu;
    p.out0 = dX, p.ldo0 = lddx;
  }
  if (want_up) {  // dWg, dWu as stored: X^T dG, X^T dU, or transposed
    FusedGemm &p = ps[n++];
    p.dual = Dual::kPair;
    p.dtype = dtype;
    p.M = ur, p.N = uc, p.K = M;
    p.a_t = true;
    p.A = t ? dG : x, p.lda = t ? lddg : lx, p.A2 = t ? dU : x, p.lda2 = t ? lddu : lx;
    p.B = t ? x : dG, p.ldb = t ? lx : lddg, p.B2 = t ? x : dU, p.ldb2 = t ? lx : lddu;
    p.out0 = dWg, p.ldo0 = lddwg, p.out1 = dWu, p.ldo1 = lddwu;
  }
  if (want_down) {  // dWd as stored: H^T dY, or its transpose
    FusedGemm &p = ps[n++];
    p.dtype = dtype;
    p.M = uc, p.N = ur, p.K = M;
    p.a_t = true;
    p.A = t ? dy : H, p.lda = t ? ly : ldh, p.B = t ? H : dy, p.ldb = t ? ldh : ly;
    p.out0 = dWd, p.ldo0 = lddwd;
  }
  return release(stage, done(launch_fused_batch(ps, n, sms, stream), "gradient launch"));
}

}  // extern "C"
