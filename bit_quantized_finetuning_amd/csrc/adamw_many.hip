// AdamW over a list of tensors in few launches, the moments in 32 bits or in 8,
// with the gradients clipped to a global norm on the device.
//
// Per element, in float32 (decoupled weight decay, as the one-tensor step):
//   g <- c g,  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) + eps)
// c = min(1, max_norm / (|g| + 1e-6)) over all tensors' gradients, |g|^2 summed
// in float64. A norm that is not finite leaves everything as it was.
//
// 8-bit moments: m and sqrt(v) in e4m3, one float32 scale (amax / 448) per block
// of 256 elements. The root halves the exponents that a block has to span (a
// ratio of 2^17.8 between its largest and smallest sqrt(v) is 2^35 in v).
// Rounding is stochastic: v's change in one step, about 1 - b2 of itself, is far
// below half a step of any 8-bit format, so rounding to nearest would never
// move it. sqrt(v) > 0 never rounds to zero (the update divides by it).
//
// HBM bounds it: 18 bytes per element with 8-bit moments and a float32 gradient
// (30 with 32-bit ones), and 4 more for the norm's pass. One wave takes a block
// of 256 (4 elements per lane) at a time and a contiguous run of blocks in all;
// the tensors' addresses travel as a kernel argument, so nothing is copied to
// the device and a captured launch holds them. Measured: 560 tensors, 250
// million elements, 8-bit moments, clipped: 1198 us (4.6 TB/s; a large copy
// reaches 4.7); 14 tensors of one 7B layer, 1.2 million elements: 13.5 us (one
// launch for the norm, one for the step).
#include "fp8.h"
#include "host.h"
#include "kernels.h"

namespace qlora {

constexpr int kManyBlock = 256;

// The job that block b of the launch belongs to (jobs without elements have no
// blocks): every lane compares its share of the jobs' ends, so it takes one
// load's time (a binary search takes seven, one after another).
template <typename J>
__device__ __forceinline__ int find_job(const J &jobs, uint32_t b) {
  constexpr int kMost = sizeof(jobs.blk0) / sizeof(uint32_t) - 1;
  const int lane = threadIdx.x & 63;
  int j = 0;
#pragma unroll
  for (int u = 0; u < kMost; u += 64) {
    const uint32_t end = lane + u < jobs.count ? jobs.blk0[lane + u + 1] : ~0u;
    j += __popcll(__ballot(b >= end));
  }
  return j;
}

// Four gradients at p, `left` of them inside the tensor.
__device__ __forceinline__ void load_grad4(const float *p, int64_t left, float g[4]) {
  if (left >= 4) {
    const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = e < left ? p[e] : 0.f;
  }
}
__device__ __forceinline__ void load_grad4(const uint16_t *p, int64_t left, float g[4]) {
  if (left >= 4) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    g[0] = bf16_lo_to_f32(v[0]);
    g[1] = bf16_hi_to_f32(v[0]);
    g[2] = bf16_lo_to_f32(v[1]);
    g[3] = bf16_hi_to_f32(v[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = e < left ? __uint_as_float((uint32_t)p[e] << 16) : 0.f;
  }
}

// ---------------------------------------------------------------------------
// the norm
// ---------------------------------------------------------------------------
// Whole blocks of one tensor go four at a time, their loads in flight together (50 million float32 elements: 42 us, one
// block after another 50).
constexpr int kSqAhead = 4;

template <typename G>
__global__ __launch_bounds__(256) void k_grad_sq(SqJobs jobs, double *__restrict__ partial) {
  __shared__ double red[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t total = jobs.blk0[jobs.count], nw = gridDim.x * 4;
  const uint32_t per = (total + nw - 1) / nw;
  uint32_t b = (blockIdx.x * 4 + wave) * per;
  const uint32_t end = b + per < total ? b + per : total;
  double sum = 0.0;
  if (b < end) {
    int j = find_job(jobs, b);
    while (b < end) {
      while (b >= jobs.blk0[j + 1]) ++j;
      const uint32_t last = jobs.blk0[j + 1] - 1;
      const int tail = jobs.tail[j];
      const G *p = static_cast<const G *>(jobs.grad[j]) + (int64_t)(b - jobs.blk0[j]) * kManyBlock + lane * 4;
      if (end - b >= kSqAhead && last + (tail == kManyBlock) - b >= kSqAhead) {
        float g[kSqAhead][4];
#pragma unroll
        for (int u = 0; u < kSqAhead; ++u) load_grad4(p + u * kManyBlock, 4, g[u]);
#pragma unroll
        for (int u = 0; u < kSqAhead; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = fma((double)g[u][e], (double)g[u][e], sum);
        b += kSqAhead;
      } else {
        float g[4];
        load_grad4(p, b < last ? 4 : tail - lane * 4, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = fma((double)g[e], (double)g[e], sum);
        ++b;
      }
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) red[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) partial[blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// The norm from the workgroups' sums of squares, in every thread of a workgroup of 256.
__device__ __forceinline__ float norm_of(const double *__restrict__ partial, int n, double *red) {
  double sum = 0.0;
  for (int i0 = threadIdx.x; i0 < n; i0 += 1024) {
    double v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i0 + 256 * u < n ? partial[i0 + 256 * u] : 0.0;
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += v[u];
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  return (float)sqrt(red[0] + red[1] + red[2] + red[3]);
}
// The factor on the gradients; NaN: leave everything as it was.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  return norm < INFINITY ? fminf(1.f, max_norm * (1.f / (norm + 1e-6f))) : NAN;
}

__global__ __launch_bounds__(256) void k_grad_norm(const double *__restrict__ partial, int n, float max_norm,
                                                   float *__restrict__ norm_out, float *__restrict__ coef) {
  __shared__ double red[4];
  const float norm = norm_of(partial, n, red);
  if (threadIdx.x == 0) {
    *norm_out = norm;
    *coef = clip_factor(norm, max_norm);
  }
}

// ---------------------------------------------------------------------------
// the step
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max64(float v) {
  v = max16(v);
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// 32 bits for the element at place i of the moments: multiplicative hashing
// (Knuth, The Art of Computer Programming, volume 3, section 6.4) by three odd
// numbers (the fractions of the golden ratio, sqrt 2 and sqrt 5), with the high half folded
// into the low between them. The low 16 bits round m, the high 16 sqrt(v).
__device__ __forceinline__ uint32_t random_bits(uint32_t i, uint32_t key) {
  uint32_t x = i * 0x9E3779B1u + key;
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  x = (x ^ (x >> 13)) * 0x3C6EF373u;
  return x ^ (x >> 16);
}

// Non-negative x <= 448 to e4m3's grid: up with the probability of its place
// between its neighbours (16 bits of it). Below 2^-6 the grid is that of
// [2^-6, 2^-5), so x is moved there and back. 448 itself, one float32 rounding
// above it (x is a product with 448 / amax) and NaN go on to the conversion.
__device__ __forceinline__ float round_e4m3(float x, uint32_t r16) {
  const bool small = x < 0x1p-6f;
  const float y = small ? x + 0x1p-6f : x;
  const float z = __uint_as_float((__float_as_uint(y) + (r16 << 4)) & 0xfff00000u);
  return x < kE4m3Max ? (small ? z - 0x1p-6f : z) : x;
}

__device__ __forceinline__ void moments(float &m, float &v, float g, const AdamWArgs &a) {
#pragma clang fp contract(off)
  m = a.b1 * m + a.one_minus_b1 * g;
  v = a.b2 * v + a.one_minus_b2 * (g * g);
}

template <typename G, bool BITS8, bool MASTER, bool WHOLE>
__device__ __forceinline__ void step_block(const G *grad, void *param, int64_t left, int64_t at, int64_t block,
                                           const ManyState &st, const AdamWArgs &a, float coef, uint32_t key) {
  // at: this lane's first element in the state arrays; left: elements of the tensor from here on
  const int lane = threadIdx.x & 63;
  float g[4], p[4], m[4], v[4];
  load_grad4(grad, WHOLE ? 4 : left, g);
  float *pm = MASTER ? st.master + at : static_cast<float *>(param);
  if (WHOLE) {
    const f32x4 t = *reinterpret_cast<const f32x4 *>(pm);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = e < left ? pm[e] : 0.f;
  }
  if constexpr (BITS8) {
    const float sm = st.m_scale[block], sv = st.v_scale[block];
    uint32_t cm = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(st.m) + at);
    uint32_t cv = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(st.v) + at);
    if (!WHOLE) {
      const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - 8 * left);
      cm &= keep;
      cv &= keep;
    }
    const f32x2 m0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cm, false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cm, true);
    const f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cv, false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)cv, true);
    const float r[4] = {v0[0] * sv, v0[1] * sv, v1[0] * sv, v1[1] * sv};
    m[0] = m0[0] * sm;
    m[1] = m0[1] * sm;
    m[2] = m1[0] * sm;
    m[3] = m1[1] * sm;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = r[e] * r[e];
  } else {
    const float *mp = static_cast<const float *>(st.m) + at, *vp = static_cast<const float *>(st.v) + at;
    if (WHOLE) {
      const f32x4 t = *reinterpret_cast<const f32x4 *>(mp), u = *reinterpret_cast<const f32x4 *>(vp);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[e] = t[e];
        v[e] = u[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[e] = e < left ? mp[e] : 0.f;
        v[e] = e < left ? vp[e] : 0.f;
      }
    }
  }
  float root[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    moments(m[e], v[e], g[e] * coef, a);
    root[e] = sqrtf(v[e]);
    p[e] = p[e] * a.decay - a.lr * ((m[e] * a.c1) / (root[e] * a.c2 + a.eps));
  }
  if (WHOLE) {
    *reinterpret_cast<f32x4 *>(pm) = f32x4{p[0], p[1], p[2], p[3]};
    if (MASTER) *reinterpret_cast<u32x2 *>(param) = u32x2{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) {
        pm[e] = p[e];
        if (MASTER) static_cast<uint16_t *>(param)[e] = (uint16_t)pack_bf16x2(p[e], 0.f);
      }
  }
  if constexpr (BITS8) {
    float am = 0.f, av = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      am = fmaxf(am, fabsf(m[e]));
      av = fmaxf(av, root[e]);
    }
    am = fmaxf(max64(am), kFp8Tiny);
    av = fmaxf(max64(av), kFp8Tiny);
    const float im = kE4m3Max * (1.f / am), iv = kE4m3Max * (1.f / av);
    float qm[4], qv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t r = random_bits((uint32_t)at + e, key);
      qm[e] = copysignf(round_e4m3(fabsf(m[e]) * im, r & 0xffffu), m[e]);
      qv[e] = round_e4m3(root[e] * iv, r >> 16);
      if (root[e] > 0.f && qv[e] == 0.f) qv[e] = 0x1p-9f;
    }
    const uint32_t cm = pack_fp8x4<false>(qm[0], qm[1], qm[2], qm[3]), cv = pack_fp8x4<false>(qv[0], qv[1], qv[2], qv[3]);
    uint8_t *mp = static_cast<uint8_t *>(st.m) + at, *vp = static_cast<uint8_t *>(st.v) + at;
    if (WHOLE) {
      *reinterpret_cast<uint32_t *>(mp) = cm;
      *reinterpret_cast<uint32_t *>(vp) = cv;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) {
          mp[e] = (uint8_t)(cm >> (8 * e));
          vp[e] = (uint8_t)(cv >> (8 * e));
        }
    }
    if (lane == 0) {
      st.m_scale[block] = am * (1.f / kE4m3Max);
      st.v_scale[block] = av * (1.f / kE4m3Max);
    }
  } else {
    float *mp = static_cast<float *>(st.m) + at, *vp = static_cast<float *>(st.v) + at;
    if (WHOLE) {
      *reinterpret_cast<f32x4 *>(mp) = f32x4{m[0], m[1], m[2], m[3]};
      *reinterpret_cast<f32x4 *>(vp) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) {
          mp[e] = m[e];
          vp[e] = v[e];
        }
    }
  }
}

// a.c1 and a.c2 hold 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t) here (ten instructions less for each division, of 470 a block:
// 250 million elements 1214 -> 1198 us).
template <typename G, bool BITS8, bool MASTER>
__global__ __launch_bounds__(256) void k_adamw_many(ManyJobs jobs, ManyState st, AdamWArgs a, ManyClip clip,
                                                    uint32_t key) {
  using P = typename std::conditional<MASTER, uint16_t, float>::type;
  __shared__ double red[4];
  float coef = 1.f;
  if (clip.partial) {
    const float norm = norm_of(clip.partial, clip.n, red);
    if (blockIdx.x == 0 && threadIdx.x == 0) *clip.norm = norm;
    coef = clip_factor(norm, clip.max_norm);
  } else if (clip.coef) {
    coef = *clip.coef;
  }
  if (coef != coef) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t total = jobs.blk0[jobs.count], nw = gridDim.x * 4;
  const uint32_t per = (total + nw - 1) / nw;
  uint32_t b = (blockIdx.x * 4 + wave) * per;
  const uint32_t end = b + per < total ? b + per : total;
  if (b >= end) return;
  int j = find_job(jobs, b);
  for (; b < end; ++b) {
    while (b >= jobs.blk0[j + 1]) ++j;
    const int64_t first = (int64_t)(b - jobs.blk0[j]) * kManyBlock, n = jobs.n[j], e0 = first + lane * 4;
    const int64_t block = st.base + b, at = block * kManyBlock + lane * 4;
    const G *grad = static_cast<const G *>(jobs.grad[j]) + e0;
    P *param = static_cast<P *>(jobs.param[j]) + e0;
    if (first + kManyBlock <= n)
      step_block<G, BITS8, MASTER, true>(grad, param, 4, at, block, st, a, coef, key);
    else
      step_block<G, BITS8, MASTER, false>(grad, param, n - e0, at, block, st, a, coef, key);
  }
}

// Workgroups of a launch over `blocks` blocks of 256: four waves each, at most
// eight workgroups per compute unit (all resident at once).
static unsigned many_grid(uint32_t blocks) {
  const int64_t cap = (int64_t)device_cu_count(current_device()) * 8;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(cap, (blocks + 3) / 4));
}

hipError_t launch_grad_sq(const SqJobs &jobs, bool bf16, double *partial, int *wgs, hipStream_t st) {
  const unsigned grid = std::min<unsigned>(many_grid(jobs.blk0[jobs.count]), kManyPartials);
  *wgs = (int)grid;
  if (bf16)
    k_grad_sq<uint16_t><<<dim3(grid), dim3(256), 0, st>>>(jobs, partial);
  else
    k_grad_sq<float><<<dim3(grid), dim3(256), 0, st>>>(jobs, partial);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double *partial, int n, float max_norm, float *norm, float *coef, hipStream_t st) {
  k_grad_norm<<<dim3(1), dim3(256), 0, st>>>(partial, n, max_norm, norm, coef);
  return hipGetLastError();
}

hipError_t launch_adamw_many(const ManyJobs &jobs, const ManyState &s, bool grad_bf16, bool bits8, bool master,
                             const AdamWArgs &a, const ManyClip &clip, uint32_t key, hipStream_t st) {
  const dim3 grid(many_grid(jobs.blk0[jobs.count])), block(256);
#define QLORA_MANY(G, B8, M) k_adamw_many<G, B8, M><<<grid, block, 0, st>>>(jobs, s, a, clip, key)
  if (grad_bf16) {
    if (bits8)
      master ? QLORA_MANY(uint16_t, true, true) : QLORA_MANY(uint16_t, true, false);
    else
      master ? QLORA_MANY(uint16_t, false, true) : QLORA_MANY(uint16_t, false, false);
  } else {
    if (bits8)
      master ? QLORA_MANY(float, true, true) : QLORA_MANY(float, true, false);
    else
      master ? QLORA_MANY(float, false, true) : QLORA_MANY(float, false, false);
  }
#undef QLORA_MANY
  return hipGetLastError();
}

}  // namespace qlora
