// ops.h -- internal launchers of the feed-forward operators (not exported).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace dg {

// Whether rows at pitch `ld` (elements of `es` bytes) all start on 16-byte
// boundaries; an absent matrix (null, pitch 0) does.
inline bool rows_aligned(const void *p, int64_t ld, int es = 2) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0;
}

// Pitch of a workspace's rows, in elements of `es` bytes: whole 128-byte lines (TMA reads
// a box's rows of 128 bytes at half the rate where each lies in two lines: 16 products
// of 997^2 took 172 us at a pitch of 1000 halves, of 1024^2 135).
inline int64_t line_pitch(int64_t cols, int es) { return (cols * es + 127) / 128 * 128 / es; }

// What a fused product does with its accumulator tile (all in fp32, rounded
// once per stored element).
enum class Epi {
  kLinear,    // z = acc + bias; [Z = z]; D = act(z) + R
  kGated,     // two accumulators g, u: [G = g, U = u]; H = act(g) u
  kGatedBwd,  // acc = dh: dG = dh u act'(g), dU = dh act(g), H = act(g) u
};

// How a second operand pair (A2, B2) of the same shapes and leading
// dimensions joins the first.
enum class Dual {
  kNone,   // out = A B
  kSum,    // out = A B + A2 B2, one accumulation
  kPair,   // out0 = A B, out1 = A2 B2
  kGated,  // g = A B, u = A B2 (Epi::kGated)
};

// One fused product of 16-bit operands.  a_t: A is stored K x M, else M x K;
// b_t: B is stored N x K, else K x N; all row-major.  Outputs and the
// epilogue's inputs are M x N, row-major, of the operands' type.
struct FusedGemm {
  Epi epi = Epi::kLinear;
  Dual dual = Dual::kNone;
  int dtype = 0;  // dgemm_dtype_t: BF16 or F16
  int act = 0;    // dgemm_activation_t
  int M = 0, N = 0, K = 0;
  bool a_t = false, b_t = false;
  const void *A = nullptr, *A2 = nullptr, *B = nullptr, *B2 = nullptr;
  int64_t lda = 0, lda2 = 0, ldb = 0, ldb2 = 0;
  // kLinear: out0 = D, out1 = Z (or null), in0 = R (or null), bias (or null)
  //          (Dual::kPair: out0, out1 the two products, no bias, Z or R)
  // kGated: out0 = H, out1 = G, out2 = U (both or neither)
  // kGatedBwd: in0 = G, in1 = U; out0 = dG, out1 = dU, out2 = H
  void *out0 = nullptr, *out1 = nullptr, *out2 = nullptr;
  int64_t ldo0 = 0, ldo1 = 0, ldo2 = 0;
  const void *in0 = nullptr, *in1 = nullptr;
  int64_t ldi0 = 0, ldi1 = 0;
  const void *bias = nullptr;
};
cudaError_t launch_fused(const FusedGemm &p, int num_sms, cudaStream_t stream);

// Up to kMaxBatch independent Epi::kLinear products of one type: in one launch
// of the small kernel where that is the quicker way, else one after the other.
cudaError_t launch_fused_batch(const FusedGemm *p, int n, int num_sms, cudaStream_t stream);

constexpr int kMaxRepitch = 12;  // jobs in one launch

// A 16-bit rows x cols matrix copied to a 16-byte aligned pitch (ldd >= cols, a
// multiple of 8), the padding zeroed.
struct RepitchJob {
  const void *src;
  int64_t lds;
  void *dst;
  int64_t ldd;
  int64_t rows, cols;
};
cudaError_t launch_repitch(const RepitchJob *jobs, int njobs, int num_sms, cudaStream_t stream);

// Copies of operands that TMA cannot read (rows that do not start on 16-byte
// boundaries): add() them, run() re-pitches all of them in one launch into
// stream-ordered scratch and points the operands there; release() after the
// last launch that reads them.
class Stager {
 public:
  Stager(int num_sms, cudaStream_t stream) : num_sms_(num_sms), stream_(stream) {}
  void add(const void *&p, int64_t &ld, int64_t rows, int64_t cols);
  cudaError_t run();
  cudaError_t release();

 private:
  static constexpr int kMax = kMaxRepitch;
  struct Item {
    const void **p;
    int64_t *ld;
    int64_t rows, cols;
  };
  Item items_[kMax];
  int n_ = 0, num_sms_;
  cudaStream_t stream_;
  void *scratch_ = nullptr;
};

// One operand layout each (one translation unit each): 0: A M x K, B K x N;
// 1: A M x K, B N x K; 2: A K x M, B K x N.  Operands that TMA can read;
// `watchdog` is the device address of the watchdog word.
cudaError_t launch_fused_pair_unit_0(const FusedGemm &p, int *watchdog, cudaStream_t stream);
cudaError_t launch_fused_pair_unit_1(const FusedGemm &p, int *watchdog, cudaStream_t stream);
cudaError_t launch_fused_pair_unit_2(const FusedGemm &p, int *watchdog, cudaStream_t stream);

// How fused_small.cu cuts a product: token columns of a tile (a multiple of
// 16, of 64 when A is stored K x M; at most 256), 64-element rows of K per
// stage (1 or 2), CTAs that share a tile's K range (1 to 8), CTAs per SM whose
// stages have to fit (1 or 2; 2 only up to 128 tokens).
struct SmallPlan {
  int nt, kd, splits, per_sm;
};
// Stages of a plan's operand ring, and how many of its tiles (clusters of
// `splits` CTAs) the device holds at once.
int small_stages(const SmallPlan &plan);
int64_t small_resident(const SmallPlan &plan, int num_sms);
// Tiles of a kernel that the device holds at once, by CTAs per SM and K split; the current
// device's, made once (null: no device, no memory): fused_small.cu's, int8_small.cu's.
struct Residency {
  int64_t tiles[3][9];
};
const Residency *residency(int num_sms);
const Residency *int8_residency(int num_sms);
// `n` products in one launch (three at most for Epi::kLinear, one otherwise;
// their plans agree in splits and per_sm).  0: bf16 linear, 1: fp16 linear, 2:
// bf16 gated, 3: fp16 gated.
constexpr int kMaxBatch = 3;
#define DG_DECLARE_SMALL_UNIT(u)                                                               \
  cudaError_t launch_fused_small_unit_##u(const FusedGemm *p, const SmallPlan *plan, int n,    \
                                          int *watchdog, cudaStream_t stream);
DG_DECLARE_SMALL_UNIT(0)
DG_DECLARE_SMALL_UNIT(1)
DG_DECLARE_SMALL_UNIT(2)
DG_DECLARE_SMALL_UNIT(3)
#undef DG_DECLARE_SMALL_UNIT

// dZ = dD act'(Z) (act != none; else dZ is not written) and, where dbias is
// not null, dbias[j] = sum_i dZ[i][j] in fp32, rounded once.  `partial` is
// fp32 scratch of act_grad_scratch() bytes.
size_t act_grad_scratch(int M, int N, bool with_bias, int num_sms);
cudaError_t launch_act_grad(int dtype, int act, int M, int N, const void *dD, int64_t lddd,
                            const void *Z, int64_t ldz, void *dZ, int64_t lddz, void *dbias,
                            float *partial, int num_sms, cudaStream_t stream);

// out0[col], out1[col] = sums over parts of partial[part][0][col] and
// partial[part][1][col]; a null output is skipped.
cudaError_t launch_column_sums(int dtype, const float *partial, int parts, int cols, void *out0,
                               void *out1, cudaStream_t stream);

// Layer norm over rows of `cols` elements.
cudaError_t launch_layer_norm(int dtype, int rows, int cols, float eps, const void *X, int64_t ldx,
                              const void *weight, const void *bias, void *Y, int64_t ldy,
                              float *mean, float *rstd, cudaStream_t stream);
// `partial`: fp32 scratch of layer_norm_scratch() bytes (0 when neither
// dweight nor dbias is asked for).
size_t layer_norm_scratch(int rows, int cols, bool with_grads, int num_sms);
cudaError_t launch_layer_norm_backward(int dtype, int rows, int cols, const void *dY, int64_t lddy,
                                       const void *X, int64_t ldx, const void *weight,
                                       const float *mean, const float *rstd, const void *dR,
                                       int64_t lddr, void *dX, int64_t lddx, void *dweight,
                                       void *dbias, float *partial, int num_sms,
                                       cudaStream_t stream);

// ------------------------------------------------- 8-bit integer products
// Copies of weights whose rows TMA cannot read to rows of `ldd` bytes (a multiple of 16), made
// by the launch that puts the tokens into 8 bits.
struct ByteCopies {
  struct Job {
    const uint8_t *src;
    uint8_t *dst;
    int64_t lds, ldd;
    int rows, cols;
  } job[3];
  int n = 0;
};
// Rows of X as integers (quant.cu): Q in 8 bits, or T in fp16 with rows of whole
// 16-byte vectors (ldt a multiple of 8), and a scale for each row.
cudaError_t launch_quantize_rows(int dtype, int rows, int cols, const void *X, int64_t ldx,
                                 int8_t *Q, int64_t ldq, float *scale, int num_sms,
                                 cudaStream_t stream);
cudaError_t launch_quantize_tokens(int dtype, int rows, int cols, const void *X, int64_t ldx,
                                   void *T, int64_t ldt, float *scale, const ByteCopies &copies,
                                   int num_sms, cudaStream_t stream);
// T = X, integers already.
cudaError_t launch_expand_tokens(int rows, int cols, const int8_t *X, int64_t ldx, void *T,
                                 int64_t ldt, const ByteCopies &copies, int num_sms,
                                 cudaStream_t stream);
// Columns of X (rows x cols) as rows of Q (cols x rows); `tops`: scratch of cols words.
cudaError_t launch_quantize_columns(int dtype, int rows, int cols, const void *X, int64_t ldx,
                                    int8_t *Q, int64_t ldq, float *scale, uint32_t *tops,
                                    int num_sms, cudaStream_t stream);

// z[i][j] = t_scale[i] w_scale[j] sum_k T[i][k] W[j][k], T the integers in fp16 (M x
// K, a multiple of 8 as leading dimension, written by the kernel just before on
// the stream, one of the two above), W in 8 bits (N x K, rows on 16-byte
// boundaries; early: they may be read before that kernel is done, as everything before it is
// once it signals, which quant.cu's kernels do only after their own wait, and it writes no weights
// itself).  out = act(z + bias) + in0, of `dtype`; gated: out = act(z) z2 in
// fp32 (ldo a multiple of 8), z2 from W2 and w2_scale.
struct Int8Gemm {
  bool gated = false, early = false;
  int dtype = 0, act = 0;
  int M = 0, N = 0, K = 0;
  const void *T = nullptr, *W = nullptr, *W2 = nullptr;
  int64_t ldt = 0, ldw = 0, ldw2 = 0;
  const float *t_scale = nullptr, *w_scale = nullptr, *w2_scale = nullptr;
  const void *bias = nullptr, *in0 = nullptr;
  int64_t ldi0 = 0;
  void *out = nullptr;
  int64_t ldo = 0;
};
cudaError_t launch_int8(const Int8Gemm &p, int num_sms, cudaStream_t stream);
// Whether a product (or two, one after the other) goes to int8_row.cu instead: where it
// can and is the quicker way, weights that TMA cannot read being copied for the others.
// DGEMM_INT8_ROW=0 / =1 forces it.
bool int8_use_row(const Int8Gemm *p, int n, int num_sms);

// The same for one to four tokens X of x_type (or integers, with p.t_scale their
// scales), quantised in the kernel: p.T and p.ldt are not looked at, p.t_scale is
// null for X to be quantised; W on any alignment.  early: the kernel ahead on the
// stream is another of these, so the weights may be read before it is done.
bool int8_row_takes(int M, int K);
double int8_row_time(const Int8Gemm &p);
cudaError_t launch_int8_row(const Int8Gemm &p, const void *X, int64_t ldx, int x_type, bool early, int num_sms,
                            cudaStream_t stream);

// How int8_small.cu cuts a product: tokens of a tile (a multiple of 16 up to
// 128), CTAs that share a tile's K range (1 to 8), CTAs per SM whose stages have to fit.
struct Int8Plan {
  int nt, splits, per_sm;
};
int64_t int8_small_resident(int splits, int per_sm, int num_sms);
cudaError_t launch_int8_small(const Int8Gemm &p, const Int8Plan &plan, int *watchdog,
                              cudaStream_t stream);
// int8_pair.cu, tiles of `nt` tokens (a multiple of 32 up to 192); K > 0.
cudaError_t launch_int8_pair(const Int8Gemm &p, int nt, int *watchdog, cudaStream_t stream);

// ------------------------------------------------- orthogonalised updates
// The products of a Newton-Schulz iteration, fp16 operands:
//   out = alpha f^power A B + beta in0 + gamma I,  f = *factor (1 where null)
// layout 0: A M x K, B K x N; 1: A M x K, B N x K; 2: A K x M, B K x N; rows on
// 16-byte boundaries.  symmetric: the result is (M = N), half of its tiles are
// computed and written to both places; layouts 1 and 2, fp16 results.  With A2, a
// second product A2 B goes to out2 in the same launch, without in0 and gamma
// (symmetric ones only).  A_lo, B_lo (laid out like A, B; not with A2): what A and B leave
// of operands of more than 11 bits; the product is A B + A B_lo + A_lo B then, in one
// accumulator, without the terms that are null.  out and in0 are of `dtype`; out_cols: columns that may be
// written, N or more (a workspace's padding).
struct NewtonGemm {
  int layout = 1;
  bool symmetric = false;
  int dtype = 0;  // dgemm_dtype_t
  int M = 0, N = 0, K = 0;
  const void *A = nullptr, *A2 = nullptr, *B = nullptr, *A_lo = nullptr, *B_lo = nullptr;
  int64_t lda = 0, ldb = 0;
  float alpha = 1.f, beta = 0.f, gamma = 0.f;
  const float *factor = nullptr;
  int power = 0;
  const void *in0 = nullptr;
  int64_t ldi0 = 0;
  void *out = nullptr, *out2 = nullptr;
  int64_t ldo = 0;
  int64_t out_cols = 0;
};
cudaError_t launch_newton_pair(const NewtonGemm &p, int *watchdog, cudaStream_t stream);
// The same on 128 x tn tiles (128, or 64 without a split), the K range of each shared by
// `splits` (1, 2, 4 or 8) CTAs.
cudaError_t launch_newton_small(const NewtonGemm &p, int tn, int splits, int num_sms, int *watchdog,
                                cudaStream_t stream);

// The whole iteration (newton.cu); `work` of newton_workspace() bytes, 16-byte aligned.
struct Orthogonalize {
  int x_dtype = 0, dtype = 0, rows = 0, cols = 0, steps = 0;
  const float *coefficients = nullptr;  // (a, b, c) per step, host memory
  float eps = 0.f, scale = 1.f, residual_scale = 1.f;
  const void *X = nullptr, *R = nullptr;
  void *D = nullptr;
  int64_t ldx = 0, ldr = 0, ldd = 0;
};
size_t newton_workspace(int rows, int cols);
cudaError_t launch_orthogonalize(const Orthogonalize &p, void *work, int num_sms, cudaStream_t stream);

}  // namespace dg
