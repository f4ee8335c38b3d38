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
#include "tiles.h"

namespace qlora {

// ---------------------------------------------------------------------------
// The tiled kernel: 256 outputs x 256 tokens per workgroup of eight waves, each
// 128 outputs x 64 tokens; K advances by one scale block of 128. Both operands'
// tiles go from memory straight into LDS (two tiles of each, step k + 1 on its
// way during step k), as do the step's 256 token scales.
// ---------------------------------------------------------------------------
constexpr int kTileN = 256, kTileT = 256, kStep = 128;
constexpr int kWaveN = 128, kWaveT = 64;
constexpr int kDown = 4;
constexpr int kOperand = kTileN * kStep;              // bytes of one operand's tile
constexpr int kStage = 2 * kOperand;                  // weight tile, token tile
constexpr int kScales = kTileT * 16;                  // four steps' token scales
constexpr size_t kFp8Lds = (size_t)2 * kStage + 2 * kScales;

// One dword per lane from memory into LDS (lane L lands at M0 + 4 L).
__device__ __forceinline__ void dma4_asm(const i32x4 &rs, uint32_t m0v, uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, %3 offen lds"
      :
      : "s"(m0v), "v"(voff), "s"(rs), "s"(soff)
      : "memory");
}

typedef __attribute__((address_space(3))) i32x2v lds_i32x2;

template <bool TRANS, bool E5M2>
__global__ __launch_bounds__(512, 2) void k_fp8_gemm(const uint8_t *__restrict__ W, const float *__restrict__ ws,
                                                     int N, int K, int ldw, int sld, const uint8_t *__restrict__ xq,
                                                     const float *__restrict__ xs, int64_t T,
                                                     const uint16_t *__restrict__ su, int rp,
                                                     const uint16_t *__restrict__ L, int r, int gn, int gt,
                                                     uint16_t *__restrict__ out) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, g = lane >> 4;
  const int wn = wave & 1, wt = wave >> 1;
  // The workgroups of one XCD (blockIdx % 8) take a contiguous share of the tiles in an order that walks down kDown
  // token tiles before the next column, so that the 32 tiles it holds at once read 4 token tiles and 8 weight tiles.
  const int tiles = gn * gt, share = tiles / 8, extra = tiles % 8, xcd = blockIdx.x % 8;
  const int seq = xcd * share + (xcd < extra ? xcd : extra) + blockIdx.x / 8;
  const int band = seq / (kDown * gn), in_band = seq - band * kDown * gn;
  const int down = gt - band * kDown < kDown ? gt - band * kDown : kDown;
  const int tn = in_band / down, tt = band * kDown + in_band % down;
  const int64_t n0 = (int64_t)tn * kTileN, t0 = (int64_t)tt * kTileT;
  const int nb = (K + kStep - 1) / kStep;
  const int rows_t = T - t0 < kTileT ? (int)(T - t0) : kTileT;
  const int rows_n = N - n0 < kTileN ? (int)(N - n0) : kTileN;

  // copies: wave w, instruction q fills LDS bytes (4 w + q) KB of each operand's tile
  const i32x4 xr = rsrc_words(xq + t0 * K, (int64_t)rows_t * K);
  const i32x4 sr = rsrc_words(xs + t0 * nb, (int64_t)rows_t * nb * 4);
  const i32x4 wr0 = rsrc_words(W + n0 * (TRANS ? 1 : (int64_t)ldw), TRANS ? 0 : (int64_t)rows_n * ldw);
  uint32_t xv[4], wv[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = 8 * (4 * wave + q) + (lane >> 3);
    const int c = 16 * ((lane & 7) ^ ((row >> 1) & 7));
    xv[q] = (uint32_t)(row * K + c);
    if constexpr (TRANS) {
      const int k = 4 * (4 * wave + q) + (lane >> 4);
      wv[q] = (uint32_t)(k * ldw + 16 * ((lane & 15) ^ ((k & 7) | (((k >> 4) & 1) << 3))));
    } else {
      wv[q] = (uint32_t)(row * ldw + c);
    }
  }
  const uint32_t lds0 = lds_addr(smem) + 4096u * (uint32_t)wave;
  // Column of the lane's chunk in pieces q = 0, 2 (and, 64 further on or back, q = 1, 3). A chunk is whole or past K
  // (K % 16 == 0); past K it reads zeros, and so does every chunk of a step past the last.
  const int c0 = 16 * ((lane & 7) ^ ((lane >> 4) & 7)), c1 = c0 ^ 64;
  auto copy_x = [&](int b, int q) {
    const int k0 = b * kStep;
    const bool in = k0 + ((q & 1) ? c1 : c0) < K;
    dma16_asm(xr, lds0 + (uint32_t)((b & 1) * kStage + kOperand + 1024 * q), in ? xv[q] + (uint32_t)k0 : kOOB, 0u);
  };
  auto copy_w = [&](int b, int q) {
    const int k0 = b * kStep;
    const uint32_t to = lds0 + (uint32_t)((b & 1) * kStage + 1024 * q);
    if constexpr (TRANS) {
      const int left = K - k0 < kStep ? K - k0 : kStep;
      dma16_asm(rsrc_words(W + (int64_t)k0 * ldw + n0, left > 0 ? (int64_t)left * ldw - n0 : 0), to, wv[q], 0u);
    } else {
      const bool in = k0 + ((q & 1) ? c1 : c0) < K;
      dma16_asm(wr0, to, in ? wv[q] + (uint32_t)k0 : kOOB, 0u);
    }
  };
  // Token scales of four steps at once, 16 bytes per token; the last group starts early enough to end with the row.
  // Rows of fewer than four scales: one step after another, tokens side by side.
  const bool wide = nb >= 4;
  const int s_tok = wide ? 16 : 4, s_step = wide ? 4 : kTileT * 4;
  auto scale_start = [&](int group) { return wide && 4 * group + 4 > nb ? nb - 4 : 4 * group; };
  auto copy_s = [&](int group) {
    if (wave >= 4) return;
    const uint32_t to = lds_addr(smem) + (uint32_t)(2 * kStage + (group & 1) * kScales);
    const uint32_t at = (uint32_t)((wave * 64 + lane) * nb + scale_start(group)) * 4u;
    if (wide) {
      dma16_asm(sr, to + 1024u * (uint32_t)wave, at, 0u);
    } else {
      for (int k = 0; k < nb; ++k) dma4_asm(sr, to + (uint32_t)(k * s_step) + 256u * (uint32_t)wave, at + 4u * (uint32_t)k, 0u);
    }
  };

  f32x4 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const uint32_t frag = (uint32_t)(li * 128 + ((g ^ ((li >> 1) & 7)) << 4));
  // columns by transposing reads: lane l of 16 points at 8 bytes of row l / 2, and gets the 8 rows of column l
  const uint32_t tr_row = (uint32_t)((16 * g + (li >> 1)) * 256 + (li & 1) * 8), tr_f = (uint32_t)((li >> 1) | ((g & 1) << 3));
  // a wave past the last column reads the last block's scale: its results are not stored
  const int64_t nblk = n0 / 128 + wn, nlast = (N - 1) / 128;
  const float *wsp = ws + (nblk < nlast ? nblk : nlast) * (TRANS ? 1 : sld);
  const int64_t wstep = TRANS ? sld : 1;

  auto load_x = [&](const uint8_t *st, int j) {
    const uint8_t *t = st + kOperand + wt * (kWaveT * kStep) + j * 2048;
    return join8(ld16(t + frag), ld16(t + (frag ^ 64u)));
  };
  auto load_w = [&](const uint8_t *st, int i) {
    if constexpr (TRANS) {
      const uint8_t *t = st + tr_row + (((uint32_t)(wn * 8 + i) ^ tr_f) << 4);
      i32x8 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x2v v =
            __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(t + (q & 1) * 2048 + (q >> 1) * 16384));
        w[2 * q] = v[0];
        w[2 * q + 1] = v[1];
      }
      return w;
    } else {
      const uint8_t *t = st + wn * (kWaveN * kStep) + i * 2048;
      return join8(ld16(t + frag), ld16(t + (frag ^ 64u)));
    }
  };
  auto load_s = [&](int b, int j) {
    const uint8_t *t = smem + 2 * kStage + ((b >> 2) & 1) * kScales + (b - scale_start(b >> 2)) * s_step;
    return *reinterpret_cast<const float *>(t + (wt * kWaveT + j * 16 + li) * s_tok);
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  i32x8 xf[4], w0;
  float sc[4];
  auto add = [&](const f32x4 &p, int i, int j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], sc[j], acc[i][j][e]);
    pin(acc[i][j]);  // (or the sums sink past the branches of the copy, and every product waits in registers)
  };

#pragma unroll
  for (int q = 0; q < 4; ++q) {
    copy_x(0, q);
    copy_w(0, q);
  }
  copy_s(0);
  wait_barrier<0>();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    copy_x(1, q);
  }
  float wsc = wsp[0];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    xf[j] = load_x(smem, j);
    sc[j] = load_s(0, j) * wsc;
  }
  w0 = load_w(smem, 0);

  for (int b = 0; b < nb; ++b) {
    const uint8_t *st = smem + (size_t)(b & 1) * kStage, *next = smem + (size_t)((b & 1) ^ 1) * kStage;
    i32x8 wf[3];
    wf[0] = w0;
    f32x4 p[2][4];
    // outputs 16 i .. +15 of the wave, i = 0 .. 5: four products, the sums of the i before, the weights of the i after
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      wf[(i + 1) % 3] = load_w(st, i + 1);
      if (i == 5) wf[1] = load_w(st, 7);
      if (i == 3) wsc = wsp[(b + 1 < nb ? b + 1 : b) * wstep];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i & 1][j] = mfma_fp8<E5M2>(wf[i % 3], xf[j], zero);
        QLORA_SCHED_FENCE();
        if (i < 2 && (j & 1)) copy_w(b + 1, 2 * i + (j >> 1));
        if (i > 0) add(p[(i & 1) ^ 1][j], i - 1, j);
        QLORA_SCHED_FENCE();
      }
    }
    // every fragment of this step is in registers: the next step's tiles are awaited and the one after is sent for
    // while i = 6, 7 are still to be multiplied
    wait_barrier<0>();
    if ((b & 3) == 0 && b + 4 < nb) copy_s((b >> 2) + 1);
    QLORA_SCHED_FENCE();
    f32x4 q6, q7;
    float sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4 a6 = mfma_fp8<E5M2>(wf[0], xf[j], zero), a7 = mfma_fp8<E5M2>(wf[1], xf[j], zero);
      QLORA_SCHED_FENCE();
      copy_x(b + 2, j);
      add(p[1][j], 5, j);
      if (j > 0) {
        add(q6, 6, j - 1);
        add(q7, 7, j - 1);
      }
      q6 = a6;
      q7 = a7;
      xf[j] = load_x(next, j);
      sn[j] = load_s(b + 1 < nb ? b + 1 : b, j);
      if (j == 1) w0 = load_w(next, 0);
      QLORA_SCHED_FENCE();
    }
    add(q6, 6, 3);
    add(q7, 7, 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) sc[j] = sn[j] * wsc;
  }

  wait_vmem();  // no copy into LDS outlives the workgroup

  // the adapter term: rank columns in steps of 32, operands from memory
  const int64_t nw = n0 + wn * kWaveN, tw = t0 + wt * kWaveT;
  for (int k = 8 * g; k < r + 8 * g; k += 32) {
    u32x4 sf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sf[j] = u32x4{0, 0, 0, 0};
      if (k < r && tw + j * 16 + li < T) sf[j] = ld16(su + (tw + j * 16 + li) * rp + k);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u32x4 lf = {0, 0, 0, 0};
      if (k < r && nw + i * 16 + li < N) lf = ld16(L + (nw + i * 16 + li) * r + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mfma16(lf, sf[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t t = tw + j * 16 + li;
    if (t < T) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t n = nw + i * 16 + 4 * g;
        if (n < N)
          *reinterpret_cast<u32x2 *>(out + t * N + n) =
              u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
      }
    }
  }
}

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
  if (T > 16) {
    auto *k = trans ? (e5m2 ? k_fp8_gemm<true, true> : k_fp8_gemm<true, false>)
                    : (e5m2 ? k_fp8_gemm<false, true> : k_fp8_gemm<false, false>);
    static DeviceOnce once;
    const hipError_t e = once.run(current_device(), [] {
      for (auto *f : {k_fp8_gemm<true, true>, k_fp8_gemm<true, false>, k_fp8_gemm<false, true>, k_fp8_gemm<false, false>}) {
        const hipError_t s = hipFuncSetAttribute(reinterpret_cast<const void *>(f),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)kFp8Lds);
        if (s != hipSuccess) return s;
      }
      return hipSuccess;
    });
    if (e != hipSuccess) return e;
    const int64_t gn = (N + kTileN - 1) / kTileN, gt = (T + kTileT - 1) / kTileT;
    if (gn * gt >= (int64_t)1 << 31) return hipErrorInvalidValue;
    k<<<dim3((unsigned)(gn * gt)), dim3(512), kFp8Lds, st>>>(W, ws, (int)N, (int)K, (int)d_in, (int)sld, xq, xs, T, su,
                                                             rp, L, r, (int)gn, (int)gt, out);
    return hipGetLastError();
  }
  const int64_t blocks = (N / 16) * ((T + 15) / 16);
  if (blocks >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(64);
  auto *k = trans ? (e5m2 ? k_fp8_product_simple<true, true> : k_fp8_product_simple<true, false>)
                  : (e5m2 ? k_fp8_product_simple<false, true> : k_fp8_product_simple<false, false>);
  k<<<grid, block, 0, st>>>(W, ws, N, K, d_in, sld, xq, xs, T, su, rp, L, r, out);
  return hipGetLastError();
}

}  // namespace qlora
