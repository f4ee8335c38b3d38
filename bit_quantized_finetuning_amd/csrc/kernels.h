// Internal host-side launchers of the gfx950 kernels. Called only by api.cpp after
// argument validation; every launcher enqueues on `st` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "common.h"
#include "qlora.h"

namespace qlora {

// Per-device one-time set-up of a launcher (function attributes): the first
// call on a device runs `fn` under a once flag, every call returns its status.
// Safe to use from any number of host threads.
constexpr int kMaxDevices = 64;
struct DeviceOnce {
  std::once_flag flag[kMaxDevices];
  hipError_t status[kMaxDevices] = {};
  template <class F>
  hipError_t run(int dev, F &&fn) {
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    std::call_once(flag[dev], [&] { status[dev] = fn(); });
    return status[dev];
  }
};
// api.cpp: the current device (-1 if it cannot be read) and its compute-unit
// count (read once per device; 256 if the query fails).
int current_device();
int device_cu_count(int dev);

// api.cpp: the forward's argument checks, the workspace bytes one forward call
// touches, and its kernels on a checked workspace (used by the entry points of
// api.cpp and scratch.hip). r must already be 0 when A = B = NULL for the last two.
int validate_forward(const qlora_nf4_weight *W, const uint16_t *x, int64_t T, const uint16_t *A, const uint16_t *B,
                     int32_t r, uint16_t *h, float *u_out);
size_t forward_workspace_need(int64_t d_out, int64_t d_in, int64_t T, int r);
int enqueue_forward(const qlora_nf4_weight *W, const uint16_t *x, int64_t T, const uint16_t *A, const uint16_t *B,
                    int32_t r, float alpha, uint16_t *h, float *u_out, void *ws, hipStream_t stream);

// quantize.hip
// Up to kQuantizeJobs weights per launch, passed by value as a kernel
// argument (no device buffer): job i covers global groups
// [gstart[i], gstart[i+1]); qscale[i] == NULL selects absmax-only storage.
constexpr int kQuantizeJobs = 32;
struct QuantizeJobs {
  const void *W[kQuantizeJobs];
  uint8_t *codes[kQuantizeJobs];
  uint8_t *qscale[kQuantizeJobs];
  float *smax[kQuantizeJobs];
  int64_t nblocks[kQuantizeJobs];
  int64_t gstart[kQuantizeJobs + 1];
  int n;
};
hipError_t launch_quantize(const QuantizeJobs &jobs, bool bf16_in, uint32_t *flags, const Nf4Consts &c,
                           hipStream_t st);
hipError_t launch_dequantize(const uint8_t *codes, const uint8_t *qscale, const float *smax,
                             int64_t d_out, int64_t d_in, bool bf16_out, void *out, const Nf4Consts &c,
                             hipStream_t st);

// adamw.hip: one AdamW step over n float32 elements (see the kernel file).
// grad, master, m, v are device-accessible addresses (pinned host memory
// mapped for the device, or device memory); param (nullable, device) receives
// bf16(master). host_state: some operand is in host memory, so the step is
// bound by the host link rather than HBM.
struct AdamWArgs {
  float lr, b1, b2, one_minus_b1, one_minus_b2, eps, decay, c1, c2;
};
hipError_t launch_adamw(const float *grad, float *master, float *m, float *v, uint16_t *param, int64_t n,
                        const AdamWArgs &a, bool host_state, hipStream_t st);

// merge.hip: out[d_out, d_in] = bf16(W_hat + scale B A), A [r, d_in], B [d_out, r] bf16 (r may be 0).
hipError_t launch_merge(const uint8_t *codes, const uint8_t *qscale, const float *smax, int64_t d_out, int64_t d_in,
                        const uint16_t *A, const uint16_t *B, int r, float scale, uint16_t *out, hipStream_t st);

// lora_small.hip: out[T, r] = P[T, K] . Q^T with Q given as [r, K] (K contiguous).
// Writes out_f32 (nullable) and out_bf16 = bf16(scale * out) with row pitch r_pad
// (zero-filled up to r_pad, a multiple of 16). Uses `partial` (ksplit*16*r_pad f32
// per 16-token tile) and `counters` (one tile_counter per 16-token tile) when ksplit > 1.
hipError_t launch_lora_small(const uint16_t *P, const uint16_t *Q, int64_t T, int64_t K, int r,
                             float scale, float *out_f32, uint16_t *out_bf16, int r_pad, float *partial,
                             uint32_t *counters, int ksplit, hipStream_t st);
// B [rows, cols] bf16 -> Bt [cols, rows] bf16
hipError_t launch_transpose_bf16(const uint16_t *src, int64_t rows, int64_t cols, uint16_t *dst,
                                 hipStream_t st);

// gemv.hip: T <= 16, one launch:
// h[T, d_out] = x W_hat^T + scale (x A^T) B^T. u_out (nullable) receives x A^T
// [T, r]. uex is the [4, 16, r_pad] exchange buffer of tagged float32 partials
// of x A^T (one per quarter of K); sync points at four reserved words (word 3
// counts the workgroups whose wait for a partial ran out of time and which then
// formed it themselves; the result does not depend on it).
hipError_t launch_gemv_fwd(const uint8_t *codes, const uint8_t *qscale, const float *smax, int64_t d_out,
                           int64_t d_in, const uint16_t *x, int64_t T, const uint16_t *A, const uint16_t *B, int r,
                           int r_pad, float scale, uint16_t *h, float *u_out, uint64_t *uex, uint32_t *sync,
                           hipStream_t st);
// Whether the T <= 16 kernel takes these sizes (its buffer ranges cover whole tensors).
bool gemv_supported(int64_t d_out, int64_t d_in, int64_t T);
// Several independent T <= 16 forwards (launch_gemv_fwd's arguments, each with
// its own exchange buffer uex) in as few launches as their kernel variants
// allow; the status words `sync` are shared. The kernel argument of one launch:
// job j runs on workgroups wg0[j] .. wg0[j+1]-1.
struct GemvJob {
  const uint8_t *codes, *qscale;
  const float *smax;
  int64_t d_out, d_in;
  const uint16_t *x;
  int64_t T;
  const uint16_t *A, *B;
  int r, r_pad;
  float scale;
  uint16_t *h;
  float *u_out;
  uint64_t *uex;
};
constexpr int kGemvJobs = 8;
struct GemvJobs {
  const uint8_t *codes[kGemvJobs];
  const uint8_t *qscale[kGemvJobs];
  const float *smax[kGemvJobs];
  const uint16_t *x[kGemvJobs];
  const uint16_t *A[kGemvJobs];
  const uint16_t *B[kGemvJobs];
  uint16_t *h[kGemvJobs];
  float *u_out[kGemvJobs];
  uint64_t *uex[kGemvJobs];
  float scale[kGemvJobs];
  int d_out[kGemvJobs], d_in[kGemvJobs], T[kGemvJobs], r[kGemvJobs], r_pad[kGemvJobs], sshift[kGemvJobs];
  int wg0[kGemvJobs + 1];
  int n;
};
hipError_t launch_gemv_fwd_many(const GemvJob *jobs, int n, uint32_t *sync, hipStream_t st);

// gemm.hip: T > 16 (and any T the weight-streaming kernel does not take).
// Work split of one contraction over 256 x 256 output tiles (gm x gn of them,
// nk K steps of 64 each): tiles 0 .. full-1 run whole, one workgroup each; each
// of the remaining `rem` tiles is cut into `split` K ranges run by separate
// workgroups, which store their float32 partial tiles (gemm_partial_floats in
// total, in the workspace's shared scratch region) and sum the tile's rows in
// range order, one share each (split_arrive in common.h). Chosen so
// that the chip's last round of tiles is not left mostly idle; depends on the
// current device's compute-unit count.
struct GemmPlan {
  int gm, gn, nk, full, rem, split;
};
GemmPlan gemm_plan(int64_t M, int64_t N, int64_t nk);
size_t gemm_partial_floats(const GemmPlan &p);
hipError_t launch_gemm_fwd(const uint8_t *codes, const uint8_t *qscale, const float *smax, int64_t d_out,
                           int64_t d_in, const uint16_t *x, int64_t T, const uint16_t *su, int r_pad,
                           const uint16_t *B, int r, uint16_t *h, float *partial, uint32_t *counters,
                           hipStream_t st);
// dX[T, d_in] = dY W_hat + sv A (sv = bf16(s*v) [T, r_pad], A [r, d_in]).
hipError_t launch_gemm_dx(const uint8_t *codes, const uint8_t *qscale, const float *smax, int64_t d_out,
                          int64_t d_in, const uint16_t *dY, int64_t T, const uint16_t *sv, int r_pad,
                          const uint16_t *A, int r, uint16_t *dX, float *partial, uint32_t *counters,
                          hipStream_t st);

// lora_wide.hip: the adapter products for T >= kWideMinTokens.
constexpr int64_t kWideMinTokens = 65;
// out[T, r] = P[T, K] . Q[r, K]^T (u = x A^T, v = dY B with Q = B^T); writes
// out_f32 [T, r] (nullable) and out_bf16 = bf16(scale * out) [T, r_pad]
// (nullable, zero columns r .. r_pad-1). Uses `partial`
// (lora_tall_partial_floats) and `counters` (one tile_counter per 64-token tile).
hipError_t launch_lora_tall(const uint16_t *P, const uint16_t *Q, int64_t T, int64_t K, int r, int r_pad, float scale,
                            float *out_f32, uint16_t *out_bf16, float *partial, uint32_t *counters, hipStream_t st);
size_t lora_tall_partial_floats(int64_t T, int64_t K, int r_pad);
// X bf16 [T, D], Y float32 [T, R]. y_is_rows: C[R, D] = scale * Y^T X (dA);
// otherwise C[D, R] = scale * X^T Y (dB). Uses `partial`
// (lora_wgrad_partial_floats) and `counters` (one tile_counter per output tile); counts in
// *fallbacks the waits that ran out of time (the result does not depend on them).
hipError_t launch_lora_wgrad(const uint16_t *X, const float *Y, int64_t T, int64_t D, int64_t R, bool y_is_rows,
                             float scale, float *C, float *partial, uint32_t *counters, uint32_t *fallbacks,
                             hipStream_t st);
size_t lora_wgrad_partial_floats(int64_t D, int64_t R, int64_t T);

// lora_grad.hip: C[M, N] = scale * sum_t P[t, m] Q[t, n] over t < T.
// P and Q are each bf16 or f32 (an f32 operand is split into two bf16 terms).
hipError_t launch_lora_grad(const void *P, bool P_f32, int64_t M, const void *Q, bool Q_f32, int64_t N,
                            int64_t T, float scale, float *C, float *partial, uint32_t *counters,
                            int ksplit, hipStream_t st);
int lora_grad_ksplit(int64_t M, int64_t N, int64_t T);
size_t lora_grad_partial_floats(int64_t M, int64_t N, int64_t T);
int lora_grad_tiles(int64_t M, int64_t N);

// adapter_grad.hip: the adapter gradients of the 8-bit base's backward, X bf16 [T, D], Y float32 [T, R] (R % 8 == 0,
// D % 16 == 0). a: out[R, D] = scale Y^T X (dA); b: out[D, R] = scale X^T Y (dB); a job with out == NULL is none. Uses
// `partial` (adapter_grad_partial_floats) and `counters` (one tile_counter per output tile); counts in *fallbacks the
// waits that ran out of time (the result does not depend on them).
struct AdapterGradJob {
  const uint16_t *X;
  const float *Y;
  float *out;
  int64_t D;
};
hipError_t launch_adapter_grad(const AdapterGradJob &a, const AdapterGradJob &b, int64_t T, int R, float scale,
                               float *partial, uint32_t *counters, uint32_t *fallbacks, hipStream_t st);
size_t adapter_grad_partial_floats(int64_t Da, int64_t Db, int R, int64_t T);

// fp8_rows.hip: one pass over bf16 rows P [T, K] (K % 16 == 0): their 8-bit codes and scales (codes == NULL: not), and
// out[T, r] = P Q^T with Q = A [r, K] or, q_is_b, B [K, r] (r % 8 == 0, r > 0): out_f32 [T, r] (nullable), out_terms [2]
// [T, rp] = scale out as two bf16 terms (nullable, zero columns r .. rp - 1); and lt [d_lt, r] = A^T for A [r, d_lt] (lt == NULL: not).
// Uses `partial` (fp8_rows_partial_floats) and `counters` (one tile_counter per 64 tokens or fewer).
struct RowsJob {
  const uint16_t *P;
  int64_t T, K;
  uint8_t *codes;
  float *scales;
  const uint16_t *Q;
  int r;
  float scale;
  float *out_f32;
  uint16_t *out_terms;
  const uint16_t *A;
  uint16_t *lt;
  int64_t d_lt;
  float *partial;
  uint32_t *counters;
};
hipError_t launch_fp8_rows(const RowsJob &a, int fmt, bool q_is_b, int rp, hipStream_t st);
size_t fp8_rows_partial_floats(int64_t T, int64_t K, int rp);

// fp8_quant.hip: rows [T, d] (d % 8 == 0) to 8 bits in groups of 128 with power-of-two scales [T, ceil(d / 128)];
// a weight [N, K] (K % 8 == 0) to e4m3 in blocks of 128 x 128 with scales [ceil(N / 128), ceil(K / 128)].
hipError_t launch_fp8_quantize_rows(const void *x, bool bf16_in, int64_t T, int64_t d, bool e5m2, uint8_t *codes,
                                    float *scales, hipStream_t st);
hipError_t launch_fp8_quantize_weight(const void *W, bool bf16_in, int64_t N, int64_t K, uint8_t *codes, float *scales,
                                      hipStream_t st);

// fp8_gemm.hip: out[T, N] = the block-scaled product of xq [T, K] with the e4m3 weight [d_out, d_in] (trans false:
// N = d_out, K = d_in; true: the weight read by columns, N = d_in, K = d_out) + su L^T (su [2][T, rp]: the
// sum of two bf16 terms; L bf16 [N, r]; r may be 0). Uses `partial` (fp8_partial_floats) and `counters` (one tile_counter per output tile).
hipError_t launch_fp8_product(const uint8_t *W, const float *ws, int64_t d_out, int64_t d_in, bool trans,
                              const uint8_t *xq, const float *xs, bool e5m2, int64_t T, const uint16_t *su, int rp,
                              const uint16_t *L, int r, uint16_t *out, float *partial, uint32_t *counters,
                              hipStream_t st);
size_t fp8_partial_floats(int64_t T, int64_t N, int64_t K, bool trans);
// T <= kFp8StreamTokens, forward: out = the product + scale (x A^T) B^T in one launch (r = 0: without an adapter).
// u_out (nullable) receives x A^T; ex: fp8_stream_exchange_bytes of scratch; counters: the workspace's counter region
// (one tile_counter per 16 ranks; its last word counts the tiles that a reader formed itself).
constexpr int64_t kFp8StreamTokens = 16;
hipError_t launch_fp8_stream(const uint8_t *W, const float *ws, int64_t N, int64_t K, const uint8_t *xq, const float *xs,
                             bool e5m2, int64_t T, const uint16_t *x, const uint16_t *A, const uint16_t *B, int r, int rp,
                             float scale, float *u_out, void *ex, uint32_t *counters, uint16_t *out,
                             hipStream_t st);
size_t fp8_stream_exchange_bytes(int rp);

// rmsnorm.hip: row strides in elements; s, y, yq, dx and the partial sums are dense. partial: rmsnorm_partial_floats
// floats when dw is wanted, else null.
struct NormFwd {
  const void *x, *res, *w;
  int64_t ldx, ldr;
  void *s, *y;
  uint8_t *yq;
  float *ys, *rstd;
  int64_t T;
  int d;
  float eps;
  bool w_bf16, e5m2;
};
struct NormBwd {
  const void *dy, *s, *ds, *w;
  int64_t ldy, lds, ldd;
  const float *rstd;
  void *dx;
  float *partial;
  int64_t T;
  int d;
  bool w_bf16;
};
hipError_t launch_rmsnorm_fwd(const NormFwd &a, bool bf16, hipStream_t st);
hipError_t launch_rmsnorm_bwd(const NormBwd &a, bool bf16, float *dw, hipStream_t st);
size_t rmsnorm_partial_floats(int64_t T, int64_t d);
hipError_t launch_fill_f32(float *p, int64_t n, float v, hipStream_t st);

// adamw_many.hip: up to kManyJobs tensors per launch, passed by value as a kernel argument. Tensor j's blocks of 256
// are blk0[j] .. blk0[j + 1] - 1 of the launch; base is the first one's place in the state arrays.
constexpr int kManyJobs = 128;
constexpr int kManyPartials = 1024;  // workgroups of one launch of the norm's pass
struct ManyJobs {
  const void *grad[kManyJobs];
  void *param[kManyJobs];
  int64_t n[kManyJobs];
  uint32_t blk0[kManyJobs + 1];
  int count;
};
// The norm's pass needs less of a tensor, so more of them fit: its gradient and the elements of its last block (448
// tensors, 20 million elements, in two launches instead of four: the step takes 152 us instead of 160).
constexpr int kSqJobs = 256;
struct SqJobs {
  const void *grad[kSqJobs];
  uint32_t blk0[kSqJobs + 1];
  uint16_t tail[kSqJobs];
  int count;
};
static_assert(sizeof(SqJobs) + 16 <= 4096, "kernel arguments");
struct ManyState {
  void *m, *v;
  float *m_scale, *v_scale, *master;
  int64_t base;
};
// The factor on the gradients: 1, or *coef, or formed by every workgroup from the n sums of squares in `partial`
// (which also writes *norm).
struct ManyClip {
  const float *coef;
  const double *partial;
  float *norm;
  int n;
  float max_norm;
};
static_assert(sizeof(ManyJobs) + sizeof(ManyState) + sizeof(AdamWArgs) + sizeof(ManyClip) + 16 <= 4096,
              "kernel arguments");
hipError_t launch_grad_sq(const SqJobs &jobs, bool bf16, double *partial, int *wgs, hipStream_t st);
hipError_t launch_grad_norm(const double *partial, int n, float max_norm, float *norm, float *coef, hipStream_t st);
hipError_t launch_adamw_many(const ManyJobs &jobs, const ManyState &s, bool grad_bf16, bool bits8, bool master,
                             const AdamWArgs &a, const ManyClip &clip, uint32_t key, hipStream_t st);

}  // namespace qlora
