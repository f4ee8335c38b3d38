// C entry points of a decoder layer's steps between its projections: rotary
// positions and attention. Like api.cpp: every argument is checked on the host
// before anything is enqueued, and the library allocates no memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention.h"
#include "host.h"
#include "kernels.h"
#include "qlora.h"

using namespace qlora;

namespace {

// The problem's sizes and the rows that both directions read; `rep` query heads share a key head.
int attention_args(const qlora_attention *p, AttnArgs &a) {
  if (!p) return QLORA_ERR_NULL;
  if (p->B < 1 || p->T < 1 || p->S < 1 || p->T > kMaxTokens || p->S > kMaxTokens || p->heads < 1 ||
      p->heads > QLORA_MAX_HEADS || p->kv_heads < 1 || p->heads % p->kv_heads || (p->D != 64 && p->D != 128))
    return QLORA_ERR_SHAPE;
  // indices of rows and of workgroups are 32-bit
  if (p->B > (1 << 24) || p->B * p->T * p->heads >= ((int64_t)1 << 31) || p->B * p->S * p->kv_heads >= ((int64_t)1 << 31))
    return QLORA_ERR_SHAPE;
  // a launch takes fewer than 2^32 threads: workgroups of 256 for 128 rows, or keys, of a key head
  const int64_t rows = std::max(p->T * (p->heads / p->kv_heads), p->S);
  if (p->B * p->kv_heads * ((rows + 127) / 128) >= ((int64_t)1 << 24)) return QLORA_ERR_SHAPE;
  // (the backward adds lse / scale to the scores: of less than 5e-38 that can pass float32's end)
  if (p->window < 1 || p->sinks < 0 || !(p->scale >= 1e-30f && p->scale <= 1e30f)) return QLORA_ERR_VALUE;
  if ((p->lengths && (reinterpret_cast<uintptr_t>(p->lengths) & 3)) ||
      (p->offsets && (reinterpret_cast<uintptr_t>(p->offsets) & 3)))
    return QLORA_ERR_ALIGN;
  a.lengths = p->lengths;
  a.offsets = p->offsets;
  a.B = (int)p->B;
  a.T = (int)p->T;
  a.S = (int)p->S;
  a.H = p->heads;
  a.G = p->kv_heads;
  a.rep = p->heads / p->kv_heads;
  a.window = p->window < (1 << 30) ? (int)p->window : 1 << 30;
  a.sinks = p->sinks < p->S ? (int)p->sinks : (int)p->S;
  a.scale = p->scale;
  a.c = p->scale * 1.4426950408889634f;
  return QLORA_OK;
}

// Rows of D values: 16-byte aligned, the rows of a head at least D values apart. The kernels add a lane's row of a tile of
// 32 to the tile's address as a 32-bit byte offset: rows 2^24 values apart and more do not go. (Heads and sequences enter
// the 64-bit address.)
int attention_rows(const qlora_attention_rows &r, int64_t rows, int64_t D, AttnRows &out) {
  if (!r.p) return QLORA_ERR_NULL;
  constexpr int64_t kMost = (int64_t)1 << 40;
  const int64_t token = rows > 1 ? r.token : D;  // (the stride of a single row may be anything)
  if (r.batch < 0 || r.batch > kMost || r.head < 0 || r.head > kMost || token < D || token >= QLORA_ATTENTION_MAX_STRIDE)
    return QLORA_ERR_SHAPE;
  if (!aligned16(r.p) || r.batch % 8 || token % 8 || r.head % 8) return QLORA_ERR_ALIGN;
  out = AttnRows{r.p, r.batch, token, r.head};
  return QLORA_OK;
}

int64_t clamped(int64_t v, int64_t most) { return v < most ? v : most; }

}  // namespace

extern "C" {

size_t qlora_attention_workspace_bytes(int64_t B, int64_t T, int64_t S, int32_t heads, int32_t kv_heads, int32_t D,
                                       int64_t window, int64_t sinks) {
  if (B < 1 || T < 1 || S < 1 || T > kMaxTokens || S > kMaxTokens || heads < 1 || kv_heads < 1 || heads % kv_heads ||
      window < 1 || sinks < 0)
    return 0;
  const size_t partial = attn_plan(B, T, S, heads, kv_heads, D, (int)clamped(window, 1 << 30), (int)clamped(sinks, S)).partial_floats;
  return partial ? kExchangeEnd + 4 * partial : kMaxCounters * 4;
}

size_t qlora_attention_backward_workspace_bytes(int64_t B, int64_t T, int64_t S, int32_t heads, int32_t kv_heads,
                                                int32_t D, int64_t window, int64_t sinks) {
  if (B < 1 || T < 1 || S < 1 || T > kMaxTokens || S > kMaxTokens || heads < 1 || kv_heads < 1 || heads % kv_heads ||
      window < 1 || sinks < 0)
    return 0;
  return 4 * attn_bwd_workspace_floats(B, T, S, heads, kv_heads, D, (int)clamped(window, 1 << 30),
                                       (int)clamped(sinks, S), nullptr);
}

int qlora_attention_forward(const qlora_attention *p, const qlora_attention_rows *q, const qlora_attention_rows *k,
                            const qlora_attention_rows *v, uint16_t *o, float *lse, void *ws, size_t ws_bytes,
                            hipStream_t stream) {
  AttnArgs a{};
  int s = attention_args(p, a);
  if (s) return s;
  if (!q || !k || !v || !o) return QLORA_ERR_NULL;
  if ((s = attention_rows(*q, p->T, p->D, a.q)) || (s = attention_rows(*k, p->S, p->D, a.k)) ||
      (s = attention_rows(*v, p->S, p->D, a.v)))
    return s;
  if (!aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3)) return QLORA_ERR_ALIGN;
  if (ws_bytes < qlora_attention_workspace_bytes(p->B, p->T, p->S, p->heads, p->kv_heads, p->D, p->window, p->sinks))
    return QLORA_ERR_WORKSPACE;
  if (!ws) return QLORA_ERR_NULL;
  if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  return hip_status(launch_attn_fwd(a, p->D, o, lse, at<float>(ws, kExchangeEnd), at<uint32_t>(ws, 0), stream));
}

int qlora_attention_backward(const qlora_attention *p, const qlora_attention_rows *dO, const qlora_attention_rows *q,
                             const qlora_attention_rows *k, const qlora_attention_rows *v,
                             const qlora_attention_rows *o, const float *lse, uint16_t *dq, uint16_t *dk, uint16_t *dv,
                             void *ws, size_t ws_bytes, hipStream_t stream) {
  AttnArgs a{};
  int s = attention_args(p, a);
  if (s) return s;
  if (!dO || !q || !k || !v || !o || !lse || !dq || !dk || !dv) return QLORA_ERR_NULL;
  AttnRows ro, rd;
  if ((s = attention_rows(*q, p->T, p->D, a.q)) || (s = attention_rows(*k, p->S, p->D, a.k)) ||
      (s = attention_rows(*v, p->S, p->D, a.v)) || (s = attention_rows(*o, p->T, p->D, ro)) ||
      (s = attention_rows(*dO, p->T, p->D, rd)))
    return s;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3)) return QLORA_ERR_ALIGN;
  if (ws_bytes <
      qlora_attention_backward_workspace_bytes(p->B, p->T, p->S, p->heads, p->kv_heads, p->D, p->window, p->sinks))
    return QLORA_ERR_WORKSPACE;
  if (!ws) return QLORA_ERR_NULL;
  if (!aligned16(ws)) return QLORA_ERR_ALIGN;
  return hip_status(launch_attn_bwd(a, p->D, ro, rd, lse, dq, dk, dv, at<float>(ws, 0), stream));
}

int qlora_rotary(const qlora_rotary_rows *rows, int32_t count, int dtype, int64_t T, int32_t D, int32_t dim,
                 const void *positions, int pos_bits, const double *freqs, float amplitude, int interleaved,
                 int inverse, hipStream_t stream) {
  if (!rows) return QLORA_ERR_NULL;
  if (dtype != QLORA_F32 && dtype != QLORA_BF16) return QLORA_ERR_DTYPE;
  if (count < 1 || count > 2 || T < 0 || T > kMaxTokens || D < 2 || D > QLORA_ROTARY_MAX_DIM || dim < 2 || dim > D ||
      dim % 2)
    return QLORA_ERR_SHAPE;
  if (pos_bits != 0 && pos_bits != 32 && pos_bits != 64) return QLORA_ERR_DTYPE;
  if (!std::isfinite(amplitude)) return QLORA_ERR_VALUE;
  const uintptr_t e = dtype == QLORA_BF16 ? 2 : 4;
  for (int i = 0; i < count; ++i) {
    const qlora_rotary_rows &r = rows[i];
    if (r.heads < 1 || r.heads > QLORA_MAX_HEADS || r.x_token < 0 || r.x_head < 0 || r.y_token < 0 || r.y_head < 0)
      return QLORA_ERR_SHAPE;
    if (T == 0) continue;
    if (!r.x || !r.y) return QLORA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(r.x) % e || reinterpret_cast<uintptr_t>(r.y) % e) return QLORA_ERR_ALIGN;
  }
  if (T == 0) return QLORA_OK;
  if (!freqs || (!positions) != (pos_bits == 0)) return QLORA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(freqs) % 8 || (pos_bits && reinterpret_cast<uintptr_t>(positions) % (pos_bits / 8)))
    return QLORA_ERR_ALIGN;
  return hip_status(launch_rotary(rows, count, dtype == QLORA_BF16, T, D, dim, positions, pos_bits, freqs, amplitude,
                                  interleaved != 0, inverse != 0, stream));
}

}  // extern "C"
