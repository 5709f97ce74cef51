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

}  // namespace dg
