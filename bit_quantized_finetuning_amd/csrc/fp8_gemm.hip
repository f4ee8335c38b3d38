// Products over the 8-bit frozen base.
//
//   Y[t, n] = sum_b xs[t, b] ws[n / 128, b] (sum_{k in block b} xq[t, k] wq[n, k]) + sum_j su[t, j] L[n, j]
//
// (forward: K = d_in, L = B; backward dX: the weight read by columns, K = d_out,
// L = A^T.) The inner sum over a block of 128 is one v_mfma_f32_16x16x128_f8f6f4;
// it is scaled in float32 and added to the running float32 sum, so nothing is
// rounded below 32 bits before the one rounding to bf16. The weight is the first
// operand: a lane then holds one token (one xs) and four consecutive outputs.
#include "fp8.h"
#include "kernels.h"

namespace qlora {

// One wave per 16 x 16 outputs, operands straight from memory.
template <bool TRANS, bool E5M2>
__global__ __launch_bounds__(64) void k_fp8_product_simple(const uint8_t *__restrict__ W, const float *__restrict__ ws,
                                                           int64_t N, int64_t K, int64_t ldw, int64_t lds_,
                                                           const uint8_t *__restrict__ xq, const float *__restrict__ xs,
                                                           int64_t T, const uint16_t *__restrict__ su, int rp,
                                                           const uint16_t *__restrict__ L, int r,
                                                           uint16_t *__restrict__ out) {
  const int lane = threadIdx.x, li = lane & 15, g = lane >> 4;
  const int64_t nt = N / 16, n0 = (blockIdx.x % nt) * 16, t0 = (int64_t)(blockIdx.x / nt) * 16;
  const int64_t nb = (K + 127) / 128;
  const int64_t t = t0 + li < T ? t0 + li : T - 1;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t b = 0; b < nb; ++b) {
    u32x4 wv[2] = {}, xv[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = b * 128 + 64 * h + 16 * g;
      if (k < K) {
        xv[h] = ld16(xq + t * K + k);
        if constexpr (TRANS) {
#pragma unroll
          for (int i = 0; i < 16; ++i) wv[h][i / 4] |= (uint32_t)W[(k + i) * ldw + n0 + li] << (8 * (i & 3));
        } else {
          wv[h] = ld16(W + (n0 + li) * ldw + k);
        }
      }
    }
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    const f32x4 p = mfma_fp8<E5M2>(join8(wv[0], wv[1]), join8(xv[0], xv[1]), z);
    const float s = xs[t * nb + b] * (TRANS ? ws[b * lds_ + n0 / 128] : ws[(n0 / 128) * lds_ + b]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
  }
  for (int j = 0; j < r; j += 32) {
    u32x4 a = {}, c = {};
    const int k = j + 8 * g;
    if (k < r) {
      a = ld16(L + (n0 + li) * r + k);
      c = ld16(su + t * rp + k);
    }
    acc = mfma16(a, c, acc);
  }
  if (t0 + li < T)
    *reinterpret_cast<u32x2 *>(out + t * N + n0 + 4 * g) = u32x2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
}

hipError_t launch_fp8_product(const uint8_t *W, const float *ws, int64_t d_out, int64_t d_in, bool trans,
                              const uint8_t *xq, const float *xs, bool e5m2, int64_t T, const uint16_t *su, int rp,
                              const uint16_t *L, int r, uint16_t *out, hipStream_t st) {
  const int64_t N = trans ? d_in : d_out, K = trans ? d_out : d_in;
  const int64_t sld = (d_in + 127) / 128;
  const int64_t blocks = (N / 16) * ((T + 15) / 16);
  if (blocks >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(64);
  auto *k = trans ? (e5m2 ? k_fp8_product_simple<true, true> : k_fp8_product_simple<true, false>)
                  : (e5m2 ? k_fp8_product_simple<false, true> : k_fp8_product_simple<false, false>);
  k<<<grid, block, 0, st>>>(W, ws, N, K, d_in, sld, xq, xs, T, su, rp, L, r, out);
  return hipGetLastError();
}

}  // namespace qlora
