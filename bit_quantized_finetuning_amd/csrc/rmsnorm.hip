// Root-mean-square norm with the residual's addition and an 8-bit output, and
// its backward.
//
//   s = x + res (rounded to the rows' type: it is what the residual stream keeps, so it is what is normalized)
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w,  yq, ys = 8-bit values of the float32 y in groups of 128
//   backward, g = dy w, xh = s rstd:  dx = ds + rstd (g - xh mean(g xh)),  dw = sum over rows of dy xh
//
// HBM bounds both: every row is read once and written once, and stays in
// registers between its reduction and its use (8 values per vector, V vectors
// per thread, TPR threads per row, chosen from d so that a row just fits). Sums
// are float32 (the forward adds its threads' sums in float64, since a root that
// is off decides scales); the row sum is a fixed tree, and dw is summed per workgroup in
// registers over its rows, then over workgroups in a fixed order, so results do
// not depend on scheduling. Measured: 4096 x 8192 with residual, bf16 row and
// 8-bit row 65 us (4.6 TB/s, a large copy's rate on this card); backward 2047 x
// 5120 with dw 24 us (3.5 TB/s: 5 of them are dw's second pass).
#include <cmath>

#include "fp8.h"
#include "host.h"
#include "kernels.h"

namespace qlora {

// A row's 8 consecutive values starting at p, of which `left` are inside the
// row (the rest read as zero). UNALIGNED: p is aligned to its element only (an
// odd d or row stride); the hardware takes such wide accesses.
template <bool UNALIGNED>
__device__ __forceinline__ void load_vec(const uint16_t *p, int left, float v[8]) {
  if (!UNALIGNED || left >= 8) {
    u32x4 w;
    if constexpr (UNALIGNED)
      __builtin_memcpy(&w, p, 16);
    else
      w = ld16(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo_to_f32(w[i]);
      v[2 * i + 1] = bf16_hi_to_f32(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
  }
}
template <bool UNALIGNED>
__device__ __forceinline__ void load_vec(const float *p, int left, float v[8]) {
  if (!UNALIGNED || left >= 8) {
    __builtin_memcpy(v, p, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.f;
  }
}
// Store 8 values (rounded to the type), `left` of them inside the row.
template <bool UNALIGNED>
__device__ __forceinline__ void store_vec(uint16_t *p, int left, const float v[8]) {
  const u32x4 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  if constexpr (!UNALIGNED) {
    st16(p, w);
  } else if (left >= 8) {
    __builtin_memcpy(p, &w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}
template <bool UNALIGNED>
__device__ __forceinline__ void store_vec(float *p, int left, const float v[8]) {
  if (!UNALIGNED || left >= 8) {
    __builtin_memcpy(p, v, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = v[i];
  }
}
template <bool UNALIGNED>
__device__ __forceinline__ void store_codes(uint8_t *p, int left, u32x2 q) {
  if (!UNALIGNED || left >= 8) {
    if constexpr (UNALIGNED)
      __builtin_memcpy(p, &q, 8);
    else
      *reinterpret_cast<u32x2 *>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint8_t)(q[i / 4] >> (8 * (i & 3)));
  }
}
// What storing the value in the row's type leaves of it.
template <typename E>
__device__ __forceinline__ float as_stored(float v) {
  if constexpr (sizeof(E) == 2) return bf16_lo_to_f32(pack_bf16x2(v, 0.f));
  return v;
}

// Sum over the TPR threads of a row (one wave, or a whole workgroup).
template <int TPR, typename F>
__device__ __forceinline__ F row_sum(F v, F *red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    __syncthreads();  // the previous row's readers are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) v += red[i];
  }
  return v;
}

template <typename E, int TPR, int V, bool UNALIGNED>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_fwd(NormFwd a) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ double red[16];
  const int lt = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  if (row >= a.T) return;  // whole waves (ROWS > 1 only for one-wave rows)
  const int d = a.d;
  const E *x = static_cast<const E *>(a.x) + row * a.ldx;
  const E *res = a.res ? static_cast<const E *>(a.res) + row * a.ldr : nullptr;
  float v[V][8], sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * TPR + lt) * 8, left = d - col;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    if (left > 0) {
      load_vec<UNALIGNED>(x + col, left, v[i]);
      if (res) {
        float q[8];
        load_vec<UNALIGNED>(res + col, left, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = as_stored<E>(v[i][e] + q[e]);
        store_vec<UNALIGNED>(static_cast<E *>(a.s) + row * d + col, left, v[i]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(v[i][e], v[i][e], sum);
  }
  // the threads' sums are added in float64; the root by one Newton step in it from the float32 one
  const double x2 = row_sum<TPR>((double)sum, red) / (double)d + (double)a.eps;
  const double r0 = (double)(1.f / sqrtf((float)x2));
  const double rd = r0 > 0.0 && r0 < INFINITY ? r0 * (1.5 - 0.5 * x2 * r0 * r0) : r0;
  const float rstd = (float)rd;
  if (a.rstd && lt == 0) a.rstd[row] = rstd;
  const int ng = (d + kFp8Group - 1) / kFp8Group;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * TPR + lt) * 8, left = d - col;
    float y[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (a.w && left > 0) {
      if (a.w_bf16)
        load_vec<UNALIGNED>(static_cast<const uint16_t *>(a.w) + col, left, w);
      else
        load_vec<UNALIGNED>(static_cast<const float *>(a.w) + col, left, w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rstd * w[e];
    if (a.y && left > 0) store_vec<UNALIGNED>(static_cast<E *>(a.y) + row * d + col, left, y);
    if (a.yq) {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
      m = max16(m);
      // Within eight float32 steps of where the scale doubles, the largest value before its roundings decides (v w is
      // exact in float64), so that they do not cost the group a bit.
      const uint32_t mb = __float_as_uint(m);
      if ((mb & 0x7fffffu) - (0x600000u - 8u) < 16u) {
        double md = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) md = fmax(md, fabs((double)v[i][e] * (double)w[e]) * rd);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) md = fmax(md, __shfl_xor(md, o));
        const uint32_t edge = (mb & 0xff800000u) | 0x600000u;
        m = __uint_as_float(edge + (md > (double)__uint_as_float(edge) ? 1u : 0u));
      }
      const RowScale sc = a.e5m2 ? row_scale<true>(m) : row_scale<false>(m);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= sc.inv;
      u32x2 q;
      if (a.e5m2)
        q = u32x2{pack_fp8x4<true>(y[0], y[1], y[2], y[3]), pack_fp8x4<true>(y[4], y[5], y[6], y[7])};
      else
        q = u32x2{pack_fp8x4<false>(y[0], y[1], y[2], y[3]), pack_fp8x4<false>(y[4], y[5], y[6], y[7])};
      if (left > 0) {
        store_codes<UNALIGNED>(a.yq + row * d + col, left, q);
        if ((lt & 15) == 0) a.ys[row * ng + col / kFp8Group] = sc.s;
      }
    }
  }
}

// Rows blockIdx, + gridDim, ...: dw's share of these rows stays in registers
// and is written once, as row `part` of the partial sums.
template <typename E, int TPR, int V, bool UNALIGNED>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_bwd(NormBwd a) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[16];
  const int lt = threadIdx.x % TPR;
  const int64_t part = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR, parts = (int64_t)gridDim.x * ROWS;
  const int d = a.d;
  float dw[V][8], w[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * TPR + lt) * 8, left = d - col;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[i][e] = 0.f;
      w[i][e] = 1.f;
    }
    if (a.w && left > 0) {
      if (a.w_bf16)
        load_vec<UNALIGNED>(static_cast<const uint16_t *>(a.w) + col, left, w[i]);
      else
        load_vec<UNALIGNED>(static_cast<const float *>(a.w) + col, left, w[i]);
    }
  }
  for (int64_t row = part; row < a.T; row += parts) {
    const E *s = static_cast<const E *>(a.s) + row * a.lds;
    const E *dy = static_cast<const E *>(a.dy) + row * a.ldy;
    const E *ds = a.ds ? static_cast<const E *>(a.ds) + row * a.ldd : nullptr;
    const float rstd = a.rstd[row];
    float xh[V][8], g[V][8], dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * TPR + lt) * 8, left = d - col;
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[i][e] = g[i][e] = 0.f;
      if (left > 0) {
        load_vec<UNALIGNED>(s + col, left, xh[i]);
        load_vec<UNALIGNED>(dy + col, left, g[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[i][e] *= rstd;
        dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
        g[i][e] *= w[i][e];
        dot = fmaf(g[i][e], xh[i][e], dot);
      }
    }
    const float c = row_sum<TPR>(dot, red) / (float)d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * TPR + lt) * 8, left = d - col;
      if (left <= 0) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * fmaf(-xh[i][e], c, g[i][e]);
      if (ds) {
        float q[8];
        load_vec<UNALIGNED>(ds + col, left, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += q[e];
      }
      store_vec<UNALIGNED>(static_cast<E *>(a.dx) + row * d + col, left, o);
    }
  }
  if (a.partial && part < a.T) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * TPR + lt) * 8, left = d - col;
      if (left > 0) store_vec<UNALIGNED>(a.partial + part * d + col, left, dw[i]);
    }
  }
}

// dw[c] = sum over parts: 16 columns and 64 interleaved runs of parts per
// workgroup, eight loads of a thread in flight (64 columns and 16 runs, one
// load after another: 10.6 us at 512 x 5120, this 5.4 us).
__global__ __launch_bounds__(1024) void k_rmsnorm_dw(const float *__restrict__ partial, int parts, int d,
                                                     float *__restrict__ dw) {
  __shared__ float red[64][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), run = threadIdx.x >> 4;
  float s = 0.f;
  if (c < d)
    for (int p0 = run; p0 < parts; p0 += 64 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = p0 + 64 * u < parts ? partial[(int64_t)(p0 + 64 * u) * d + c] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  red[run][threadIdx.x & 15] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += red[i][threadIdx.x];
    dw[c] = s;
  }
}

__global__ __launch_bounds__(256) void k_fill_f32(float *__restrict__ p, int64_t n, float v) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = v;
}

hipError_t launch_fill_f32(float *p, int64_t n, float v, hipStream_t st) {
  k_fill_f32<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>(p, n, v);
  return hipGetLastError();
}

namespace {

// Partial rows of dw: enough workgroups to keep HBM busy, few enough that the
// partial sums (written and read once more) stay small beside the rows.
int64_t bwd_blocks(int64_t T, int d) {
  const int rows = d <= 1024 ? 4 : 1;
  const int64_t b = (T + rows - 1) / rows;
  return b < 512 ? b : 512;
}

template <typename E, int TPR, int V>
void fwd(const NormFwd &a, bool unaligned, hipStream_t st) {
  constexpr int BT = TPR < 256 ? 256 : TPR, ROWS = BT / TPR;
  const dim3 grid((unsigned)((a.T + ROWS - 1) / ROWS)), block(BT);
  if (unaligned)
    k_rmsnorm_fwd<E, TPR, V, true><<<grid, block, 0, st>>>(a);
  else
    k_rmsnorm_fwd<E, TPR, V, false><<<grid, block, 0, st>>>(a);
}
template <typename E, int TPR, int V>
void bwd(const NormBwd &a, bool unaligned, hipStream_t st) {
  constexpr int BT = TPR < 256 ? 256 : TPR, ROWS = BT / TPR;
  const int64_t blocks = a.partial ? bwd_blocks(a.T, a.d) : std::min<int64_t>((a.T + ROWS - 1) / ROWS, 1 << 20);
  const dim3 grid((unsigned)blocks), block(BT);
  if (unaligned)
    k_rmsnorm_bwd<E, TPR, V, true><<<grid, block, 0, st>>>(a);
  else
    k_rmsnorm_bwd<E, TPR, V, false><<<grid, block, 0, st>>>(a);
}
#define QLORA_NORM_BY_WIDTH(F, a)                       \
  if (a.d <= 512) F<E, 64, 1>(a, unaligned, st);        \
  else if (a.d <= 1024) F<E, 64, 2>(a, unaligned, st);  \
  else if (a.d <= 2048) F<E, 256, 1>(a, unaligned, st); \
  else if (a.d <= 4096) F<E, 256, 2>(a, unaligned, st); \
  else if (a.d <= 6144) F<E, 256, 3>(a, unaligned, st); \
  else if (a.d <= 8192) F<E, 256, 4>(a, unaligned, st); \
  else if (a.d <= 16384) F<E, 512, 4>(a, unaligned, st); \
  else F<E, 1024, 4>(a, unaligned, st);

template <typename E>
void fwd_by_width(const NormFwd &a, bool unaligned, hipStream_t st) { QLORA_NORM_BY_WIDTH(fwd, a) }
template <typename E>
void bwd_by_width(const NormBwd &a, bool unaligned, hipStream_t st) { QLORA_NORM_BY_WIDTH(bwd, a) }

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace

size_t rmsnorm_partial_floats(int64_t T, int64_t d) { return (size_t)(bwd_blocks(T, (int)d) * (d <= 1024 ? 4 : 1) * d); }

// A launch holds fewer than 2^32 threads: more rows than kRows go by parts.
hipError_t launch_rmsnorm_fwd(const NormFwd &all, bool bf16, hipStream_t st) {
  constexpr int64_t kRows = 1 << 20;
  const int64_t e = bf16 ? 2 : 4, ng = (all.d + kFp8Group - 1) / kFp8Group;
  const bool unaligned = all.d % 8 || all.ldx % 8 || (all.res && all.ldr % 8) || off16(all.x) || off16(all.res) ||
                         off16(all.w);  // (the parts' offsets are multiples of 2^20)
  for (int64_t r = 0; r < all.T; r += kRows) {
    NormFwd a = all;
    a.T = std::min(kRows, all.T - r);
    auto in = [&](const void *p, int64_t ld) -> const void * { return p ? static_cast<const char *>(p) + r * ld * e : p; };
    auto out = [&](void *p) -> void * { return p ? static_cast<char *>(p) + r * all.d * e : p; };
    a.x = in(all.x, all.ldx);
    a.res = in(all.res, all.ldr);
    a.s = out(all.s);
    a.y = out(all.y);
    if (all.yq) {
      a.yq = all.yq + r * all.d;
      a.ys = all.ys + r * ng;
    }
    if (all.rstd) a.rstd = all.rstd + r;
    if (bf16)
      fwd_by_width<uint16_t>(a, unaligned, st);
    else
      fwd_by_width<float>(a, unaligned, st);
    const hipError_t s = hipGetLastError();
    if (s != hipSuccess) return s;
  }
  return hipSuccess;
}

hipError_t launch_rmsnorm_bwd(const NormBwd &a, bool bf16, float *dw, hipStream_t st) {
  const bool unaligned = a.d % 8 || a.lds % 8 || a.ldy % 8 || (a.ds && a.ldd % 8) || off16(a.s) || off16(a.dy) ||
                         off16(a.ds) || off16(a.w);
  if (bf16)
    bwd_by_width<uint16_t>(a, unaligned, st);
  else
    bwd_by_width<float>(a, unaligned, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dw) return e;
  const int64_t rows = a.d <= 1024 ? 4 : 1;
  const int64_t parts = std::min<int64_t>(bwd_blocks(a.T, a.d) * rows, a.T);
  k_rmsnorm_dw<<<dim3((unsigned)((a.d + 15) / 16)), dim3(1024), 0, st>>>(a.partial, (int)parts, a.d, dw);
  return hipGetLastError();
}

}  // namespace qlora
