// Quantizers of the 8-bit base: rows (activations, upstream gradients) in
// groups of 128 with a power-of-two scale, weights in blocks of 128 x 128 with
// scale amax / 448.
//
// Rows whose call also multiplies them with an adapter are quantized in the same
// pass as that product (fp8_rows.hip), by the same rule.
//
// Both quantizers read every value once and write one byte for it, so HBM bounds
// them: 3 bytes per value from bf16 (rows of 4096 x 8192: 21 us, 4.8 TB/s; a
// weight of 8192 x 8192 from float32: 72 us, 4.7 TB/s). The group maximum of a
// row is taken over 16 lanes of 8 values each (four DPP steps, no LDS).
#include "fp8.h"
#include "kernels.h"

namespace qlora {

// 8 consecutive values as float32
__device__ __forceinline__ void load8(const uint16_t *p, float v[8]) {
  const u32x4 w = ld16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo_to_f32(w[i]);
    v[2 * i + 1] = bf16_hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ void load8(const float *p, float v[8]) {
  const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ float amax8(const float v[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// One workgroup per unit of 2048 consecutive columns of one row (16 groups);
// d % 8 == 0, so a lane's 8 values are all inside the row or all outside.
template <typename E, bool E5M2>
__global__ __launch_bounds__(256) void k_fp8_quantize_rows(const E *__restrict__ x, int64_t units, int upr, int d,
                                                           uint8_t *__restrict__ codes, float *__restrict__ scales) {
  const int tid = threadIdx.x, ng = (d + kFp8Group - 1) / kFp8Group;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t row = u / upr;
    const int col = (int)(u - row * upr) * 2048 + tid * 8;
    const bool in = col < d;
    float v[8] = {};
    if (in) load8(x + row * d + col, v);
    const RowScale sc = row_scale<E5M2>(max16(amax8(v)));
    if (in) {
      u32x2 q;
      q[0] = pack_fp8x4<E5M2>(v[0] * sc.inv, v[1] * sc.inv, v[2] * sc.inv, v[3] * sc.inv);
      q[1] = pack_fp8x4<E5M2>(v[4] * sc.inv, v[5] * sc.inv, v[6] * sc.inv, v[7] * sc.inv);
      *reinterpret_cast<u32x2 *>(codes + row * d + col) = q;
      if ((tid & 15) == 0) scales[row * ng + col / kFp8Group] = sc.s;
    }
  }
}

hipError_t launch_fp8_quantize_rows(const void *x, bool bf16_in, int64_t T, int64_t d, bool e5m2, uint8_t *codes,
                                    float *scales, hipStream_t st) {
  const int upr = (int)((d + 2047) / 2048);
  const int64_t units = T * upr;
  const dim3 grid((unsigned)(units < 65536 ? units : 65536)), block(256);
  if (bf16_in) {
    auto *p = static_cast<const uint16_t *>(x);
    if (e5m2)
      k_fp8_quantize_rows<uint16_t, true><<<grid, block, 0, st>>>(p, units, upr, (int)d, codes, scales);
    else
      k_fp8_quantize_rows<uint16_t, false><<<grid, block, 0, st>>>(p, units, upr, (int)d, codes, scales);
  } else {
    auto *p = static_cast<const float *>(x);
    if (e5m2)
      k_fp8_quantize_rows<float, true><<<grid, block, 0, st>>>(p, units, upr, (int)d, codes, scales);
    else
      k_fp8_quantize_rows<float, false><<<grid, block, 0, st>>>(p, units, upr, (int)d, codes, scales);
  }
  return hipGetLastError();
}

// One workgroup per 128 x 128 block: 16 lanes cover a row's 128 columns, 16
// rows per pass, the whole block in registers between the maximum and the codes.
template <typename E>
__global__ __launch_bounds__(256) void k_fp8_quantize_weight(const E *__restrict__ W, int64_t N, int64_t K, int64_t nbk,
                                                             uint8_t *__restrict__ codes, float *__restrict__ scales) {
  __shared__ float red[4];
  const int tid = threadIdx.x;
  const int64_t bn = blockIdx.x / nbk, bk = blockIdx.x - bn * nbk;
  const int64_t col = bk * kFp8Group + (tid & 15) * 8, row0 = bn * kFp8Group + (tid >> 4);
  float v[8][8] = {};
  float m = 0.f;
#pragma unroll
  for (int p = 0; p < 8; ++p)
    if (row0 + 16 * p < N && col < K) load8(W + (row0 + 16 * p) * K + col, v[p]);
#pragma unroll
  for (int p = 0; p < 8; ++p) m = fmaxf(m, amax8(v[p]));
  m = max16(m);
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32));
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
  const float amax = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), kFp8Tiny);
  const float inv = kE4m3Max / amax;
  if (tid == 0) scales[blockIdx.x] = amax / kE4m3Max;
#pragma unroll
  for (int p = 0; p < 8; ++p)
    if (row0 + 16 * p < N && col < K) {
      u32x2 q;
      q[0] = pack_fp8x4<false>(v[p][0] * inv, v[p][1] * inv, v[p][2] * inv, v[p][3] * inv);
      q[1] = pack_fp8x4<false>(v[p][4] * inv, v[p][5] * inv, v[p][6] * inv, v[p][7] * inv);
      *reinterpret_cast<u32x2 *>(codes + (row0 + 16 * p) * K + col) = q;
    }
}

hipError_t launch_fp8_quantize_weight(const void *W, bool bf16_in, int64_t N, int64_t K, uint8_t *codes, float *scales,
                                      hipStream_t st) {
  const int64_t nbn = (N + kFp8Group - 1) / kFp8Group, nbk = (K + kFp8Group - 1) / kFp8Group;
  const dim3 grid((unsigned)(nbn * nbk)), block(256);  // at most 2^26 blocks
  if (bf16_in)
    k_fp8_quantize_weight<uint16_t><<<grid, block, 0, st>>>(static_cast<const uint16_t *>(W), N, K, nbk, codes, scales);
  else
    k_fp8_quantize_weight<float><<<grid, block, 0, st>>>(static_cast<const float *>(W), N, K, nbk, codes, scales);
  return hipGetLastError();
}

}  // namespace qlora
