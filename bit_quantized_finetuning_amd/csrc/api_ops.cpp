// C entry points around the frozen base: the 8-bit base's quantizers, forward
// and backward, the root-mean-square norm, and the AdamW step over many
// tensors. Like api.cpp: every argument is checked on the host before anything
// is enqueued, and the library allocates no memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host.h"
#include "kernels.h"
#include "qlora.h"

using namespace qlora;

namespace {

bool is_float(int dtype) { return dtype == QLORA_F32 || dtype == QLORA_BF16; }
bool is_fp8(int dtype) { return dtype == QLORA_E4M3 || dtype == QLORA_E5M2; }

int validate_fp8_weight(const qlora_fp8_weight *W) {
  if (!W || !W->codes || !W->scales) return QLORA_ERR_NULL;
  if (W->d_out < 16 || W->d_in < 16 || W->d_out % 16 || W->d_in % 16 || W->d_out > kMaxDim || W->d_in > kMaxDim)
    return QLORA_ERR_SHAPE;
  if (!aligned16(W->codes) || !aligned16(W->scales)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

int64_t groups(int64_t d) { return ceil_div(d, QLORA_FP8_GROUP); }

// Workspace regions of a call over the 8-bit base. The counter region comes
// first, as in every workspace; q8 and qs hold the rows quantized within the
// call, lt the adapter matrix that is contracted over its other dimension.
struct Fp8Layout {
  size_t ex, su, u, v, lt, q8, qs, partial, total;
};
Fp8Layout fp8_layout(int64_t d_out, int64_t d_in, int64_t T, int r) {
  Fp8Layout L{};
  const int rp = rank_pad(r);
  const int64_t d = std::max(d_out, d_in);
  size_t off = align256((size_t)kMaxCounters * sizeof(uint32_t));
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L.ex = take(T <= kFp8StreamTokens ? fp8_stream_exchange_bytes(rp) : 0);
  L.su = take((size_t)T * rp * 2 * 2);  // two bf16 terms
  L.u = take((size_t)T * r * 4);
  L.v = take((size_t)T * r * 4);
  L.lt = take((size_t)r * d_in * 2);
  L.q8 = take((size_t)T * d);
  L.qs = take((size_t)T * groups(d) * 4);
  size_t pf = 0;
  if (r > 0) {
    pf = std::max(pf, fp8_rows_partial_floats(T, d_in, rp));
    pf = std::max(pf, fp8_rows_partial_floats(T, d_out, rp));
    pf = std::max(pf, adapter_grad_partial_floats(d_in, d_out, r, T));
  }
  pf = std::max(pf, fp8_partial_floats(T, d_out, d_in, false));
  pf = std::max(pf, fp8_partial_floats(T, d_in, d_out, true));
  L.partial = take(pf * 4);
  L.total = off;
  return L;
}

int check_workspace(const void *ws, size_t ws_bytes, size_t need) {
  if (ws_bytes < need) return QLORA_ERR_WORKSPACE;
  if (!ws) return QLORA_ERR_NULL;
  return aligned16(ws) ? QLORA_OK : QLORA_ERR_ALIGN;
}

}  // namespace

extern "C" {

int qlora_stream_capture_id(uint64_t *id, hipStream_t stream) {
  if (!id) return QLORA_ERR_NULL;
  *id = 0;
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  unsigned long long n = 0;
  const hipError_t e = hipStreamGetCaptureInfo(stream, &status, &n);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    // the null stream while another stream is captured: itself it is not
    return e == hipErrorStreamCaptureImplicit ? QLORA_OK : QLORA_ERR_HIP;
  }
  if (status == hipStreamCaptureStatusActive) *id = (uint64_t)n + 1;
  return QLORA_OK;
}

size_t qlora_fp8_storage_bytes(int64_t d_out, int64_t d_in) {
  if (d_out < 1 || d_in < 1) return 0;
  return (size_t)(d_out * d_in + 4 * groups(d_out) * groups(d_in));
}

int qlora_fp8_quantize(const void *W, int w_dtype, const qlora_fp8_weight *out, hipStream_t stream) {
  if (!W) return QLORA_ERR_NULL;
  const int s = validate_fp8_weight(out);
  if (s) return s;
  if (!is_float(w_dtype)) return QLORA_ERR_DTYPE;
  if (!aligned16(W)) return QLORA_ERR_ALIGN;
  return hip_status(
      launch_fp8_quantize_weight(W, w_dtype == QLORA_BF16, out->d_out, out->d_in, out->codes, out->scales, stream));
}

int qlora_fp8_quantize_rows(const void *x, int x_dtype, int64_t T, int64_t d, int fmt, uint8_t *codes, float *scales,
                            hipStream_t stream) {
  if (!x || !codes || !scales) return QLORA_ERR_NULL;
  if (!is_float(x_dtype) || !is_fp8(fmt)) return QLORA_ERR_DTYPE;
  if (T < 1 || T > kMaxTokens || d < 16 || d % 16 || d > kMaxDim) return QLORA_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return QLORA_ERR_ALIGN;
  return hip_status(
      launch_fp8_quantize_rows(x, x_dtype == QLORA_BF16, T, d, fmt == QLORA_E5M2, codes, scales, stream));
}

size_t qlora_fp8_workspace_bytes(int64_t d_out, int64_t d_in, int64_t T, int32_t r) {
  if (d_out < 1 || d_in < 1 || T < 1 || r < 0 || r > QLORA_MAX_RANK) return 0;
  return fp8_layout(d_out, d_in, T, r).total;
}

int qlora_fp8_forward(const qlora_fp8_weight *W, const uint8_t *xq, const float *xs, int fmt, const uint16_t *x,
                      int64_t T, const uint16_t *A, const uint16_t *B, int32_t r, float alpha, uint16_t *h,
                      float *u_out, void *ws, size_t ws_bytes, hipStream_t stream) {
  int s = validate_fp8_weight(W);
  if (s) return s;
  if (!h) return QLORA_ERR_NULL;
  if (!is_fp8(fmt)) return QLORA_ERR_DTYPE;
  if (T < 1 || T > kMaxTokens || r < 0 || r > QLORA_MAX_RANK || r % 8) return QLORA_ERR_SHAPE;
  if (!A && !B) r = 0;
  if ((r > 0 && (!A || !B)) || (!xq) != (!xs)) return QLORA_ERR_NULL;
  if (!x && (!xq || r > 0)) return QLORA_ERR_NULL;
  if (!aligned16(h) || !aligned16(x) || !aligned16(xq) || !aligned16(xs) || !aligned16(u_out) ||
      (r > 0 && (!aligned16(A) || !aligned16(B))))
    return QLORA_ERR_ALIGN;
  const Fp8Layout L = fp8_layout(W->d_out, W->d_in, T, r);
  if ((s = check_workspace(ws, ws_bytes, L.total))) return s;
  const bool stream_kernel = T <= kFp8StreamTokens;  // which forms x A^T itself
  const float sc = r > 0 ? alpha / (float)r : 0.f;
  uint8_t *q = xq ? nullptr : at<uint8_t>(ws, L.q8);
  float *qs = at<float>(ws, L.qs), *partial = at<float>(ws, L.partial);
  uint16_t *su = at<uint16_t>(ws, L.su);
  uint32_t *counters = at<uint32_t>(ws, 0);
  hipError_t e = hipSuccess;
  if (r > 0 && !stream_kernel)
    e = launch_fp8_rows({x, T, W->d_in, q, qs, A, r, sc, u_out, su, nullptr, nullptr, 0, partial, counters}, fmt, false,
                        rank_pad(r), stream);
  else if (q)
    e = launch_fp8_quantize_rows(x, true, T, W->d_in, fmt == QLORA_E5M2, q, qs, stream);
  if (e != hipSuccess) return QLORA_ERR_HIP;
  if (q) {
    xq = q;
    xs = qs;
  }
  if (stream_kernel)
    return hip_status(launch_fp8_stream(W->codes, W->scales, W->d_out, W->d_in, xq, xs, fmt == QLORA_E5M2, T, x, A, B, r,
                                        rank_pad(r), sc, u_out, at<uint8_t>(ws, L.ex), counters, h, stream));
  return hip_status(launch_fp8_product(W->codes, W->scales, W->d_out, W->d_in, false, xq, xs, fmt == QLORA_E5M2, T, su,
                                       rank_pad(r), B, r, h, partial, counters, stream));
}

int qlora_fp8_backward(const qlora_fp8_weight *W, const uint16_t *x, const uint16_t *dY, int fmt, int64_t T,
                       const uint16_t *A, const uint16_t *B, int32_t r, float alpha, const float *u_saved, uint16_t *dX,
                       float *dA, float *dB, void *ws, size_t ws_bytes, hipStream_t stream) {
  int s = validate_fp8_weight(W);
  if (s) return s;
  if (!dY) return QLORA_ERR_NULL;
  if (!is_fp8(fmt)) return QLORA_ERR_DTYPE;
  if (T < 1 || T > kMaxTokens || r < 0 || r > QLORA_MAX_RANK || r % 8) return QLORA_ERR_SHAPE;
  if (!A && !B) r = 0;
  if (r > 0 && (!A || !B)) return QLORA_ERR_NULL;
  if (r == 0 && (dA || dB)) return QLORA_ERR_SHAPE;
  if ((dA && !x) || (dB && !u_saved && !x)) return QLORA_ERR_NULL;
  if (!aligned16(dY) || !aligned16(x) || !aligned16(u_saved) || !aligned16(dX) || !aligned16(dA) || !aligned16(dB) ||
      (r > 0 && (!aligned16(A) || !aligned16(B))))
    return QLORA_ERR_ALIGN;
  const int64_t d_out = W->d_out, d_in = W->d_in;
  const Fp8Layout L = fp8_layout(d_out, d_in, T, r);
  if ((s = check_workspace(ws, ws_bytes, L.total))) return s;
  if (!dX && !dA && !dB) return QLORA_OK;

  const float sc = r > 0 ? alpha / (float)r : 0.f;
  uint16_t *sv = at<uint16_t>(ws, L.su);
  float *v = at<float>(ws, L.v), *partial = at<float>(ws, L.partial);
  uint32_t *counters = at<uint32_t>(ws, 0), *fallbacks = counters + kMaxCounters - 1;
  uint8_t *q = dX ? at<uint8_t>(ws, L.q8) : nullptr;
  float *qs = at<float>(ws, L.qs);
  uint16_t *lt = r > 0 && dX ? at<uint16_t>(ws, L.lt) : nullptr;
  hipError_t e = hipSuccess;
  if (r > 0 && (dX || dA))
    e = launch_fp8_rows({dY, T, d_out, q, qs, B, r, sc, v, sv, A, lt, d_in, partial, counters}, fmt, true, rank_pad(r),
                        stream);
  else if (dX)
    e = launch_fp8_quantize_rows(dY, true, T, d_out, fmt == QLORA_E5M2, q, qs, stream);
  if (e == hipSuccess && dX)
    e = launch_fp8_product(W->codes, W->scales, d_out, d_in, true, q, qs, fmt == QLORA_E5M2, T, sv, rank_pad(r), lt, r,
                           dX, partial, counters, stream);
  const float *u = u_saved;
  if (e == hipSuccess && dB && !u) {
    u = at<float>(ws, L.u);
    e = launch_fp8_rows({x, T, d_in, nullptr, nullptr, A, r, 1.f, at<float>(ws, L.u), nullptr, nullptr, nullptr, 0, partial,
                         counters}, fmt, false, rank_pad(r), stream);
  }
  if (e == hipSuccess)
    e = launch_adapter_grad({x, v, dA, d_in}, {dY, u, dB, d_out}, T, r, sc, partial, counters, fallbacks, stream);
  if (e != hipSuccess) return QLORA_ERR_HIP;
  return QLORA_OK;
}

// ---------------------------------------------------------------------------
// the norm
// ---------------------------------------------------------------------------
static int norm_shape(int64_t T, int64_t d, int dtype, int w_dtype, float eps) {
  if (!is_float(dtype) || !is_float(w_dtype)) return QLORA_ERR_DTYPE;
  if (T < 0 || T > kMaxTokens || d < 1 || d > QLORA_NORM_MAX_DIM) return QLORA_ERR_SHAPE;
  return eps >= 0.f && eps < INFINITY ? QLORA_OK : QLORA_ERR_VALUE;
}
static bool off_element(const void *p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == QLORA_BF16 ? 1u : 3u)) != 0;
}

int qlora_rmsnorm_forward(const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, int64_t T, int64_t d,
                          const void *weight, int w_dtype, float eps, void *s, void *y, uint8_t *yq, float *ys, int fmt,
                          float *rstd, hipStream_t stream) {
  const int c = norm_shape(T, d, dtype, w_dtype, eps);
  if (c) return c;
  if (yq && !is_fp8(fmt)) return QLORA_ERR_DTYPE;
  if (T == 0) return QLORA_OK;
  if (!x || (!yq) != (!ys) || (!residual) != (!s) || (!y && !yq)) return QLORA_ERR_NULL;
  if (ldx < d || (residual && ldr < d)) return QLORA_ERR_SHAPE;
  if (off_element(x, dtype) || off_element(residual, dtype) || off_element(weight, w_dtype) || !aligned16(s) ||
      !aligned16(y) || !aligned16(yq) || !aligned16(ys) || !aligned16(rstd))
    return QLORA_ERR_ALIGN;
  const NormFwd a{x, residual, weight, ldx, ldr, s, y, yq, ys, rstd, T, (int)d, eps, w_dtype == QLORA_BF16,
                  fmt == QLORA_E5M2};
  return hip_status(launch_rmsnorm_fwd(a, dtype == QLORA_BF16, stream));
}

size_t qlora_rmsnorm_workspace_bytes(int64_t T, int64_t d) {
  if (T < 1 || d < 1 || d > QLORA_NORM_MAX_DIM) return 0;
  return rmsnorm_partial_floats(T, d) * 4;
}

int qlora_rmsnorm_backward(const void *dy, int64_t ldy, const void *s, int64_t lds, const void *ds, int64_t ldd,
                           int dtype, int64_t T, int64_t d, const void *weight, int w_dtype, const float *rstd, void *dx,
                           float *dw, void *ws, size_t ws_bytes, hipStream_t stream) {
  int c = norm_shape(T, d, dtype, w_dtype, 0.f);
  if (c) return c;
  if (T > 0 && (!dy || !s || !rstd || !dx)) return QLORA_ERR_NULL;
  if (T > 0 && (ldy < d || lds < d || (ds && ldd < d))) return QLORA_ERR_SHAPE;
  if (off_element(dy, dtype) || off_element(s, dtype) || off_element(ds, dtype) || off_element(weight, w_dtype) ||
      off_element(rstd, QLORA_F32) || !aligned16(dx) || !aligned16(dw))
    return QLORA_ERR_ALIGN;
  if (T == 0) return dw ? hip_status(launch_fill_f32(dw, d, 0.f, stream)) : QLORA_OK;
  if (dw && (c = check_workspace(ws, ws_bytes, qlora_rmsnorm_workspace_bytes(T, d)))) return c;
  const NormBwd a{dy, s, ds, weight, ldy, lds, ldd, rstd, dx, dw ? static_cast<float *>(ws) : nullptr, T, (int)d,
                  w_dtype == QLORA_BF16};
  return hip_status(launch_rmsnorm_bwd(a, dtype == QLORA_BF16, dw, stream));
}

// ---------------------------------------------------------------------------
// AdamW over many tensors
// ---------------------------------------------------------------------------
// The factor, then kManyPartials sums of squares per launch of the norm's pass.
size_t qlora_adamw_many_workspace_bytes(int32_t count) {
  if (count < 0) return 0;
  return align256(sizeof(float)) + (size_t)(count / kSqJobs + 1) * kManyPartials * sizeof(double);
}

int qlora_adamw_many(const qlora_adamw_many_hparams *hp, int64_t step, const qlora_adamw_job *jobs, int32_t count,
                     int grad_dtype, int param_dtype, const qlora_adamw_state *state, float max_norm, float *norm,
                     uint32_t seed, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (!hp || !state || (count > 0 && !jobs)) return QLORA_ERR_NULL;
  if (count < 0) return QLORA_ERR_SHAPE;
  if (!is_float(grad_dtype) || !is_float(param_dtype)) return QLORA_ERR_DTYPE;
  if (state->dtype != QLORA_F32 && state->dtype != QLORA_E4M3) return QLORA_ERR_DTYPE;
  const bool bits8 = state->dtype == QLORA_E4M3, master = param_dtype == QLORA_BF16;
  if (step < 1 || !(hp->lr >= 0.0) || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) ||
      !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) || !((float)hp->eps > 0.f) || !(hp->weight_decay >= 0.0) ||
      !(max_norm >= 0.f))
    return QLORA_ERR_VALUE;
  int64_t blocks = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (jobs[i].n < 0 || jobs[i].n >= (int64_t)1 << 38) return QLORA_ERR_SHAPE;
    if (jobs[i].n > 0 && !jobs[i].param) return QLORA_ERR_NULL;
    if (!aligned16(jobs[i].grad) || !aligned16(jobs[i].param)) return QLORA_ERR_ALIGN;
    blocks += ceil_div(jobs[i].n, QLORA_ADAMW_BLOCK);
    if (blocks >= (int64_t)1 << 31) return QLORA_ERR_SHAPE;
  }
  if (blocks > 0 && (!state->m || !state->v || (bits8 && (!state->m_scale || !state->v_scale)) ||
                     (master && !state->master)))
    return QLORA_ERR_NULL;
  if (!aligned16(state->m) || !aligned16(state->v) || !aligned16(state->master) || !aligned16(state->m_scale) ||
      !aligned16(state->v_scale))
    return QLORA_ERR_ALIGN;
  const bool clip = max_norm > 0.f;
  if (clip && !norm) return QLORA_ERR_NULL;
  if (clip) {
    const int s = check_workspace(ws, ws_bytes, qlora_adamw_many_workspace_bytes(count));
    if (s) return s;
  }
  AdamWArgs a;
  a.lr = (float)hp->lr;
  a.b1 = (float)hp->beta1;
  a.b2 = (float)hp->beta2;
  a.one_minus_b1 = (float)(1.0 - hp->beta1);
  a.one_minus_b2 = (float)(1.0 - hp->beta2);
  a.eps = (float)hp->eps;
  a.decay = (float)(1.0 - hp->lr * hp->weight_decay);
  a.c1 = (float)(1.0 / (1.0 - std::pow(hp->beta1, (double)step)));
  a.c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(hp->beta2, (double)step)));
  uint32_t key = seed * 0x9E3779B1u + (uint32_t)step * 0x85157AF5u;
  key ^= key >> 16;
  float *coef = clip ? static_cast<float *>(ws) : nullptr;
  double *partial = clip ? at<double>(ws, align256(sizeof(float))) : nullptr;

  // The tensors of one launch, from `i` on: a run of tensors that have a gradient. Returns the first one after them;
  // `base` is the place of their first block in the state arrays, `next` that of the block after them.
  ManyJobs t;
  int64_t base = 0, next = 0;
  auto fill = [&](int32_t i) {
    t.count = 0;
    t.blk0[0] = 0;
    base = next;
    for (; i < count && t.count < kManyJobs; ++i) {
      const int64_t blocks = ceil_div(jobs[i].n, QLORA_ADAMW_BLOCK);
      if (blocks > 0 && !jobs[i].grad) {
        if (t.count > 0) break;  // it ends the run
        next += blocks;
        base = next;
        continue;
      }
      next += blocks;
      t.grad[t.count] = jobs[i].grad;
      t.param[t.count] = jobs[i].param;
      t.n[t.count] = jobs[i].n;
      t.blk0[t.count + 1] = t.blk0[t.count] + (uint32_t)blocks;
      ++t.count;
    }
    return i;
  };
  ManyClip factor{};
  if (clip) {
    int n = 0, launches = 0;
    for (int32_t i = 0; i < count;) {
      SqJobs q;
      q.count = 0;
      q.blk0[0] = 0;
      for (; i < count && q.count < kSqJobs; ++i) {
        if (!jobs[i].grad || jobs[i].n == 0) continue;
        const int64_t blocks = ceil_div(jobs[i].n, QLORA_ADAMW_BLOCK);
        q.grad[q.count] = jobs[i].grad;
        q.tail[q.count] = (uint16_t)(jobs[i].n - (blocks - 1) * QLORA_ADAMW_BLOCK);
        q.blk0[q.count + 1] = q.blk0[q.count] + (uint32_t)blocks;
        ++q.count;
      }
      if (q.count == 0) continue;
      ++launches;
      int wgs = 0;
      if (launch_grad_sq(q, grad_dtype == QLORA_BF16, partial + n, &wgs, stream) != hipSuccess) return QLORA_ERR_HIP;
      n += wgs;
    }
    // One launch's sums are few enough for every workgroup of the step to add itself, which spares a launch (the
    // adapters of one 7B decoder layer: 13.9 us a step, 15.5 with it); those of several are added once.
    if (launches == 1) {
      factor = ManyClip{nullptr, partial, norm, n, max_norm};
    } else {
      if (launch_grad_norm(partial, n, max_norm, norm, coef, stream) != hipSuccess) return QLORA_ERR_HIP;
      factor.coef = coef;
    }
  }
  ManyState st{state->m, state->v, state->m_scale, state->v_scale, state->master, 0};
  next = 0;
  for (int32_t i = 0; i < count;) {
    i = fill(i);
    if (t.blk0[t.count] == 0) continue;
    st.base = base;
    if (launch_adamw_many(t, st, grad_dtype == QLORA_BF16, bits8, master, a, factor, key, stream) != hipSuccess)
      return QLORA_ERR_HIP;
  }
  return QLORA_OK;
}

}  // extern "C"
