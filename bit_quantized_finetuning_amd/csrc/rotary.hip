// Rotary positions of queries and keys.
//
// Of a head's D values the first `dim` are pairs (a, b): values i and i + dim/2,
// or 2i and 2i + 1 (interleaved). Pair i of a token at position p is turned by
// the angle p f_i and stretched by m:
//     a' = m (a cos - b sin),  b' = m (b cos + a sin)
// and the rest is copied. The turn by the negative angle is the backward (the
// transpose of m R is m R^T).
//
// Bound by memory: every value is read and written once. The sines and cosines
// of a workgroup's tokens are formed once, into LDS, and used by all heads that
// it turns. An angle is formed in 64 bits, in turns, and only its fraction of a
// turn goes on in 32: a position of 10^6 keeps the 24 bits that a small one has.
//
// 16384 tokens of 40 + 8 heads of 128: bf16 88 us a call, float32 176 (169 interleaved), 4.6 to 4.8 TB/s. Heads whose
// halves are no multiple of 16 bytes go value by value: 4096 tokens of 32 + 8 heads of 96, 70 of them turned, bf16 35 us
// (1.8 TB/s: 2 bytes a lane and instruction), float32 47.
#include "kernels.h"

namespace qlora {

constexpr int kRotThreads = 256;  // at most
constexpr int kRotPairs = 2048;   // sines and cosines that a workgroup keeps (16 KB)

struct RotaryArgs {
  const uint8_t *x[2];  // queries and keys; heads past `heads0` belong to the second
  uint8_t *y[2];
  int64_t xt[2], xh[2], yt[2], yh[2];  // token and head strides in elements
  int heads0, heads, T, D, dim;
  const void *positions;
  const double *freqs;
  float amplitude, sign;
  int items, turned;     // of a head: chunks or pairs of them (values), those of them that are turned
  int head_wg, tok_wg;   // heads and tokens of a workgroup
};

template <typename T>
struct Values;
template <>
struct Values<float> {
  static constexpr int kV = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Values<uint16_t> {
  static constexpr int kV = 8;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu); }
};

// Queries and keys are read once: loads past the caches' replacement leave room for what is written (16384 tokens of
// 40 + 8 heads: 85 us without, 67 with).
__device__ __forceinline__ u32x4 ld16_once(const void *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}

// A pair's turn; written out, so that every layout has the same roundings.
__device__ __forceinline__ float turn_a(float u, float v, float c, float s) { return fmaf(-v, s, u * c); }
__device__ __forceinline__ float turn_b(float u, float v, float c, float s) { return fmaf(u, s, v * c); }

// kVec: 16-byte chunks (every stride, offset and half a multiple of them), else value by value. A thread keeps its place
// in the heads (one division) and goes through the workgroup's tokens.
template <typename E, bool kInter, bool kVec>
__global__ __launch_bounds__(kRotThreads) void k_rotary(RotaryArgs a, int pos_bits) {
  __shared__ __attribute__((aligned(16))) float cs[kRotPairs], sn[kRotPairs];
  typedef Values<E> Q;
  constexpr int kV = kVec ? Q::kV : 1;
  const int tid = threadIdx.x, threads = blockDim.x, pairs = a.dim >> 1;
  const int t0 = blockIdx.x * a.tok_wg, nt = a.T - t0 < a.tok_wg ? a.T - t0 : a.tok_wg;
  const int h0 = blockIdx.y * a.head_wg, nh = a.heads - h0 < a.head_wg ? a.heads - h0 : a.head_wg;
  for (int i = tid; i < nt * pairs; i += threads) {
    const int t = i / pairs, p = i - t * pairs;
    const double pos = pos_bits == 64   ? (double)reinterpret_cast<const int64_t *>(a.positions)[t0 + t]
                       : pos_bits == 32 ? (double)reinterpret_cast<const int32_t *>(a.positions)[t0 + t]
                                        : (double)(t0 + t);
    double turns = pos * a.freqs[p] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    cs[i] = a.amplitude * c;
    sn[i] = a.sign * (a.amplitude * s);
  }
  __syncthreads();
  for (int j = tid; j < nh * a.items; j += threads) {
    const int hh = j / a.items, c = j - hh * a.items;
    const int h = h0 + hh, w = h >= a.heads0 ? 1 : 0, hw = h - (w ? a.heads0 : 0);
    const int64_t xt = a.xt[w], yt = a.yt[w];
    const E *x = reinterpret_cast<const E *>(a.x[w]) + t0 * xt + hw * a.xh[w];
    E *y = reinterpret_cast<E *>(a.y[w]) + t0 * yt + hw * a.yh[w];
    // An item is one chunk, or two: the halves of pairs, two neighbouring chunks behind them. Turned and copied ones go
    // through the same loads and stores, so that whole lines are written at once.
    const bool turn = c < a.turned;
    constexpr bool kOne = kInter && kVec;
    const int m = c - a.turned;  // among the copied items
    const int at = kOne ? c * kV : turn ? (kInter ? 2 * c : c * kV) : a.dim + 2 * m * kV;
    const int to2 = turn ? (kInter ? 2 * c + 1 : c * kV + pairs) : at + kV;
    const bool two = !kOne && to2 < a.D;
    if (!turn && x == y) continue;  // (in place: it stays)
    const float *ct = cs + (turn ? (kOne ? c * kV / 2 : c * kV) : 0), *st = sn + (ct - cs);
    x += at;
    y += at;
    const int step2 = to2 - at;
    if constexpr (kVec) {
#pragma unroll 4
      for (int t = 0; t < nt; ++t) {
        u32x4 lo = ld16_once(x + t * xt), hi = lo;
        if (two) hi = ld16_once(x + t * xt + step2);
        if (turn) {
          E *e = reinterpret_cast<E *>(&lo), *g = reinterpret_cast<E *>(&hi);
#pragma unroll
          for (int k = 0; k < (kOne ? kV / 2 : kV); ++k) {
            const float co = ct[t * pairs + k], si = st[t * pairs + k];
            E &ea = kOne ? e[2 * k] : e[k], &eb = kOne ? e[2 * k + 1] : g[k];
            const float u = Q::get(ea), v = Q::get(eb);
            ea = Q::put(turn_a(u, v, co, si));
            eb = Q::put(turn_b(u, v, co, si));
          }
        }
        st16(y + t * yt, lo);
        if (two) st16(y + t * yt + step2, hi);
      }
    } else {
      for (int t = 0; t < nt; ++t, x += xt, y += yt) {
        if (turn) {
          const float co = ct[t * pairs], si = st[t * pairs], u = Q::get(x[0]), v = Q::get(x[step2]);
          y[0] = Q::put(turn_a(u, v, co, si));
          y[step2] = Q::put(turn_b(u, v, co, si));
        } else {
          y[0] = x[0];
          if (two) y[step2] = x[step2];
        }
      }
    }
  }
}

template <typename E, bool kInter>
static void launch_as(bool vec, dim3 g, int threads, hipStream_t st, const RotaryArgs &a, int pos_bits) {
  if (vec)
    k_rotary<E, kInter, true><<<g, threads, 0, st>>>(a, pos_bits);
  else
    k_rotary<E, kInter, false><<<g, threads, 0, st>>>(a, pos_bits);
}

hipError_t launch_rotary(const qlora_rotary_rows *rows, int count, bool bf16, int64_t T, int D, int dim,
                         const void *positions, int pos_bits, const double *freqs, float amplitude, bool interleaved,
                         bool inverse, hipStream_t st) {
  RotaryArgs a{};
  const int e = bf16 ? 2 : 4, V = 16 / e;
  bool vec = D % V == 0 && dim % V == 0 && (interleaved || dim / 2 % V == 0);
  for (int w = 0; w < 2; ++w) {
    const qlora_rotary_rows &r = rows[w < count ? w : 0];
    a.x[w] = static_cast<const uint8_t *>(r.x);
    a.y[w] = static_cast<uint8_t *>(r.y);
    a.xt[w] = r.x_token;
    a.xh[w] = r.x_head;
    a.yt[w] = r.y_token;
    a.yh[w] = r.y_head;
    for (const int64_t s : {(int64_t)((uintptr_t)r.x / e), (int64_t)((uintptr_t)r.y / e), r.x_token, r.x_head,
                            r.y_token, r.y_head})
      vec = vec && s % V == 0;
  }
  a.heads0 = rows[0].heads;
  a.heads = rows[0].heads + (count > 1 ? rows[1].heads : 0);
  a.T = (int)T;
  a.D = D;
  a.dim = dim;
  a.positions = positions;
  a.freqs = freqs;
  a.amplitude = amplitude;
  a.sign = inverse ? -1.f : 1.f;
  a.turned = vec ? (interleaved ? dim / V : dim / 2 / V) : dim / 2;
  const int rest = (D - dim) / (vec ? V : 1);
  a.items = a.turned + (vec && interleaved ? rest : (rest + 1) / 2);
  // Eight tokens a workgroup where there are many; of few tokens one, and only some of its heads as long as the launch has
  // fewer than 512 workgroups and a workgroup more than one chunk or pair a thread (16 tokens of 40 + 8 heads of 128: 32).
  a.tok_wg = 1;
  while (a.tok_wg < 8 && 2 * a.tok_wg * (dim / 2) <= kRotPairs && T / (2 * a.tok_wg) >= 1024) a.tok_wg *= 2;
  a.head_wg = a.heads;
  while (a.head_wg > 1 && a.tok_wg == 1 && T * ((a.heads + a.head_wg - 1) / a.head_wg) < 512 &&
         a.head_wg * a.items > kRotThreads)
    a.head_wg = (a.head_wg + 1) / 2;
  // threads that divide a token's items into even turns
  const int row = a.head_wg * a.items, turns = (row + kRotThreads - 1) / kRotThreads;
  const int threads = ((row + turns - 1) / turns + 63) / 64 * 64;
  const dim3 g((unsigned)((T + a.tok_wg - 1) / a.tok_wg), (unsigned)((a.heads + a.head_wg - 1) / a.head_wg));
  if (bf16)
    interleaved ? launch_as<uint16_t, true>(vec, g, threads, st, a, pos_bits)
                : launch_as<uint16_t, false>(vec, g, threads, st, a, pos_bits);
  else
    interleaved ? launch_as<float, true>(vec, g, threads, st, a, pos_bits)
                : launch_as<float, false>(vec, g, threads, st, a, pos_bits);
  return hipGetLastError();
}

}  // namespace qlora
