// Products over the 8-bit frozen base.
//
//   Y[t, n] = sum_b xs[t, b] ws[n / 128, b] (sum_{k in block b} xq[t, k] wq[n, k]) + sum_j su[t, j] L[n, j]
//
// (forward: K = d_in, L = B; backward dX: the weight read by columns, K = d_out,
// L = A^T.) The inner sum over a block of 128 is one v_mfma_f32_16x16x128_f8f6f4.
// The unit brings eight products to the exponent of the largest of them and drops
// what lies below 2^-13 of that; apart from it sums are float32: a block's is
// scaled and added to the running one, and that is rounded once, to bf16. su, a
// float32, enters the bf16 matrix instruction as two terms, 16 bits of it (as one
// bf16 its error, 2^-8, is that of the rounding of the result again: 2.3e-3 of an
// adapter's output alone instead of 1.65e-3). The weight is the first operand: a
// lane then holds one token (one xs) and four consecutive outputs.
#include <atomic>
#include <cmath>

#include "exchange.h"
#include "fp8.h"
#include "host.h"
#include "kernels.h"
#include "tiles.h"

namespace qlora {

// ---------------------------------------------------------------------------
// The large-tile kernel: 32 MI outputs x 64 MJ tokens per workgroup of eight
// waves, each 16 MI outputs x 16 MJ tokens; K advances by one scale block of 128.
// Both operands' tiles go from memory straight into LDS (S tiles of each, steps
// k + 1 .. k + S - 1 on their way during step k), as do the token scales.
// 256 outputs x 256 tokens for whole batches, and 256 x 192, 192 x 192 (by rows)
// or 256 x 128 where that leaves fewer compute units idle. 256 x 256 has room for
// two stages; the smaller tiles' steps wait longer for their copies, so those that
// have room for three stages have them (515 tokens, 13824 x 5120: 192 x 192 54 ->
// 48 us, 256 x 128 92 -> 84). Measured in a trace of 43 calls: 4096 tokens, 22016 x
// 8192: 756 us (least 734: 2010 TFLOP/s) by rows, 743 (715: 2070) by columns. The
// matrix unit is busy half of the cycles there, LDS a fifth, and the clock falls to
// 1.8 - 1.9 GHz from the 2.35 of the 515 tokens' product.
// ---------------------------------------------------------------------------
constexpr int kStep = 128;
constexpr int kScales = 256 * 16;                     // four steps' token scales

template <bool TRANS, int MI, int MJ, int S>
struct Fp8Lds {
  static constexpr int w = TRANS ? 256 * kStep : 32 * MI * kStep;  // (by columns rows are always 256 bytes apart)
  static constexpr int stage = w + 64 * MJ * kStep;
  static constexpr int bytes = S * stage + 2 * kScales;
};

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

// Which tile (and K range) a workgroup takes. The workgroups of one XCD
// (blockIdx % 8) take a contiguous share of the work in an order that walks
// down kDown token tiles before the next K range or weight tile: what it holds
// at once then shares its weight tiles kDown times and its token tiles among
// the weight tiles (32 large tiles read 4 token tiles and 8 weight tiles), so
// its L2 pulls each of them in once.
constexpr int kDown = 4;
struct WorkPlace {
  int tn, tt, part;
};
__device__ __forceinline__ WorkPlace tile_place(int seq, int gn, int gt, int parts) {
  const int band = seq / (kDown * gn * parts), in_band = seq - band * kDown * gn * parts;
  const int down = gt - band * kDown < kDown ? gt - band * kDown : kDown;
  const int col = in_band / down;
  return WorkPlace{col / parts, band * kDown + in_band % down, col % parts};
}
// blockIdx of `work` workgroups -> its place
__device__ __forceinline__ WorkPlace work_place(int work, int gn, int gt, int parts) {
  const int share = work / 8, extra = work % 8, xcd = blockIdx.x % 8;
  return tile_place(xcd * share + (xcd < extra ? xcd : extra) + blockIdx.x / 8, gn, gt, parts);
}

template <bool TRANS, bool E5M2, int MI, int MJ, int S>
__global__ __launch_bounds__(512, 2) void k_fp8_gemm(const uint8_t *__restrict__ W, const float *__restrict__ ws,
                                                     int N, int K, int ldw, int sld, const uint8_t *__restrict__ xq,
                                                     const float *__restrict__ xs, int64_t T,
                                                     const uint16_t *__restrict__ su, int rp,
                                                     const uint16_t *__restrict__ L, int r, int gn, int gt, int full,
                                                     int parts, float *__restrict__ partial,
                                                     uint32_t *__restrict__ counters, uint16_t *__restrict__ out) {
  constexpr int kTileN = 32 * MI, kWaveN = 16 * MI, kTileT = 64 * MJ, kWaveT = 16 * MJ;
  using Lds = Fp8Lds<TRANS, MI, MJ, S>;
  constexpr int QW = TRANS ? 4 : MI / 2, kStage = Lds::stage;  // KB of the weight tile per wave
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, g = lane >> 4;
  const int wn = wave & 1, wt = wave >> 1;
  // tiles 0 .. full - 1 (in work_place's order) run whole, the others in `parts` K ranges of whole scale groups
  const bool cut = (int)blockIdx.x >= full;
  const int rest = gn * gt - full, e = (int)blockIdx.x - full;
  const int tail = cut ? e % rest : 0, part = cut ? e / rest : 0;
  const WorkPlace at = cut ? tile_place(full + tail, gn, gt, 1) : work_place(full, gn, gt, 1);
  const int tn = at.tn, tt = at.tt;
  const int64_t n0 = (int64_t)tn * kTileN, t0 = (int64_t)tt * kTileT;
  const int nb = (K + kStep - 1) / kStep, nb4 = (nb + 3) / 4;
  const int b0 = cut ? 4 * (nb4 * part / parts) : 0;
  const int b1 = cut && part + 1 < parts ? 4 * (nb4 * (part + 1) / parts) : nb;
  const int klim = b1 * kStep < K ? b1 * kStep : K;
  const int rows_t = T - t0 < kTileT ? (int)(T - t0) : kTileT;
  const int rows_n = N - n0 < kTileN ? (int)(N - n0) : kTileN;

  // copies: wave w's piece q fills KB QW w + q of the weight tile, KB MJ w + q of the token tile
  const i32x4 xr = rsrc_words(xq + t0 * K, (int64_t)rows_t * K);
  const i32x4 sr = rsrc_words(xs + t0 * nb, (int64_t)rows_t * nb * 4);
  const i32x4 wr0 = rsrc_words(W + n0 * (TRANS ? 1 : (int64_t)ldw), TRANS ? 0 : (int64_t)rows_n * ldw);
  uint32_t xv[MJ], wv[QW];
#pragma unroll
  for (int q = 0; q < MJ; ++q) {
    const int row = 8 * (MJ * wave + q) + (lane >> 3);
    xv[q] = (uint32_t)(row * K + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
  }
#pragma unroll
  for (int q = 0; q < QW; ++q) {
    const int row = 8 * (QW * wave + q) + (lane >> 3);
    if constexpr (TRANS) {
      const int k = 4 * (4 * wave + q) + (lane >> 4), c = 16 * ((lane & 15) ^ ((k & 7) | (((k >> 4) & 1) << 3)));
      wv[q] = c < kTileN ? (uint32_t)(k * ldw + c) : kOOB;
    } else {
      wv[q] = (uint32_t)(row * ldw + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
    }
  }
  const uint32_t lds_w = lds_addr(smem) + 1024u * QW * (uint32_t)wave;
  const uint32_t lds_x = lds_addr(smem) + Lds::w + 1024u * MJ * (uint32_t)wave;
  // Column of the lane's chunk in even KB of a tile and, 64 further on or back, in odd ones. A chunk is whole or past
  // the range's end (K % 16 == 0); there it reads zeros, and so does every chunk of a step past the last.
  const int c0 = 16 * ((lane & 7) ^ ((lane >> 4) & 7)), c1 = c0 ^ 64;
  auto copy_x = [&](int b, int q) {
    const int k0 = b * kStep;
    const bool in = k0 + (((MJ * wave + q) & 1) ? c1 : c0) < klim;
    dma16_asm(xr, lds_x + (uint32_t)((b % S) * kStage + 1024 * q), in ? xv[q] + (uint32_t)k0 : kOOB, 0u);
  };
  auto copy_w = [&](int b, int q) {
    const int k0 = b * kStep;
    const uint32_t to = lds_w + (uint32_t)((b % S) * kStage + 1024 * q);
    if constexpr (TRANS) {
      const int left = klim - k0 < kStep ? klim - k0 : kStep;
      dma16_asm(rsrc_words(W + (int64_t)k0 * ldw + n0, left > 0 ? (int64_t)left * ldw - n0 : 0), to, wv[q], 0u);
    } else {
      const bool in = k0 + (((QW * wave + q) & 1) ? c1 : c0) < klim;
      dma16_asm(wr0, to, in ? wv[q] + (uint32_t)k0 : kOOB, 0u);
    }
  };
  // Token scales of four steps at once, 16 bytes per token; the last group starts early enough to end with the row.
  // Rows of fewer than four scales: one step after another, tokens side by side.
  const bool wide = nb >= 4;
  const int s_tok = wide ? 16 : 4, s_step = wide ? 4 : kTileT * 4;
  auto scale_start = [&](int group) { return wide && 4 * group + 4 > nb ? nb - 4 : 4 * group; };
  auto copy_s = [&](int group) {
    if (wave >= MJ) return;
    const uint32_t to = lds_addr(smem) + (uint32_t)(S * kStage + (group & 1) * kScales);
    const uint32_t at = (uint32_t)((wave * 64 + lane) * nb + scale_start(group)) * 4u;
    if (wide) {
      dma16_asm(sr, to + 1024u * (uint32_t)wave, at, 0u);
    } else {
      for (int k = 0; k < nb; ++k) dma4_asm(sr, to + (uint32_t)(k * s_step) + 256u * (uint32_t)wave, at + 4u * (uint32_t)k, 0u);
    }
  };

  f32x4 acc[MI][MJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const uint32_t frag = (uint32_t)(li * 128 + ((g ^ ((li >> 1) & 7)) << 4));
  // columns by transposing reads: lane l of 16 points at 8 bytes of row l / 2, and gets the 8 rows of column l
  const uint32_t tr_row = (uint32_t)((16 * g + (li >> 1)) * 256 + (li & 1) * 8), tr_f = (uint32_t)((li >> 1) | ((g & 1) << 3));
  // A wave past the last column reads the last block's scale: its results are not stored. 96 outputs of a wave may lie in
  // two blocks: those from i = turn on have the second scale.
  const int64_t nblk = (n0 + wn * kWaveN) / 128, nlast = (N - 1) / 128;
  const float *wsp = ws + (nblk < nlast ? nblk : nlast) * (TRANS ? 1 : sld);
  const float *wsp2 = ws + (nblk + 1 < nlast ? nblk + 1 : nlast) * (TRANS ? 1 : sld);
  const int turn = MI == 8 ? 8 : (int)(128 * (nblk + 1) - (n0 + wn * kWaveN)) / 16;
  const int64_t wstep = TRANS ? sld : 1;

  auto load_x = [&](const uint8_t *st, int j) {
    const uint8_t *t = st + Lds::w + wt * (kWaveT * kStep) + j * 2048;
    return join8(ld16(t + frag), ld16(t + (frag ^ 64u)));
  };
  auto load_w = [&](const uint8_t *st, int i) {
    if constexpr (TRANS) {
      const uint8_t *t = st + tr_row + (((uint32_t)(wn * MI + i) ^ tr_f) << 4);
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
    const uint8_t *t = smem + S * kStage + ((b >> 2) & 1) * kScales + (b - scale_start(b >> 2)) * s_step;
    return *reinterpret_cast<const float *>(t + (wt * kWaveT + j * 16 + li) * s_tok);
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  i32x8 xf[MJ], w0;
  float sc[MJ], sc2[MJ];
  auto add = [&](const f32x4 &p, int i, int j) {
    const float s = MI == 8 || i < turn ? sc[j] : sc2[j];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s, acc[i][j][e]);
    pin(acc[i][j]);  // (or the sums sink past the branches of the copy, and every product waits in registers)
  };

#pragma unroll
  for (int q = 0; q < QW; ++q) copy_w(b0, q);
#pragma unroll
  for (int q = 0; q < MJ; ++q) copy_x(b0, q);
  copy_s(b0 >> 2);
  if constexpr (S == 3) {
#pragma unroll
    for (int q = 0; q < QW; ++q) copy_w(b0 + 1, q);
#pragma unroll
    for (int q = 0; q < MJ; ++q) copy_x(b0 + 1, q);
  }
  wait_barrier<(S - 2) * (QW + MJ)>();
#pragma unroll
  for (int q = 0; q < MJ; ++q) copy_x(b0 + S - 1, q);
  float wsc = wsp[b0 * wstep], wsc2 = MI == 8 ? 0.f : wsp2[b0 * wstep];
  const uint8_t *first = smem + (size_t)(b0 % S) * kStage;
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    xf[j] = load_x(first, j);
    const float sx = load_s(b0, j);
    sc[j] = sx * wsc;
    sc2[j] = sx * wsc2;
  }
  w0 = load_w(first, 0);

  for (int b = b0; b < b1; ++b) {
    const uint8_t *st = smem + (size_t)(b % S) * kStage, *next = smem + (size_t)((b + 1) % S) * kStage;
    i32x8 wf[3];
    wf[0] = w0;
    f32x4 p[2][MJ];
    // outputs 16 i .. +15 of the wave, all but the last two i: the products, the sums of the i before, the weights of the
    // i after
    constexpr int IL = MI - 3;
#pragma unroll
    for (int i = 0; i <= IL; ++i) {
      wf[(i + 1) % 3] = load_w(st, i + 1);
      if (i == IL) wf[(IL + 2) % 3] = load_w(st, IL + 2);
      if (i == IL - 2) {
        wsc = wsp[(b + 1 < b1 ? b + 1 : b) * wstep];
        if constexpr (MI < 8) wsc2 = wsp2[(b + 1 < b1 ? b + 1 : b) * wstep];
      }
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        p[i & 1][j] = mfma_fp8<E5M2>(wf[i % 3], xf[j], zero);
        QLORA_SCHED_FENCE();
        // (sent early in the step, two to a group where there are four: the last must land before its end)
        const int q = MJ == 4 ? 2 * i + (j >> 1) : i;
        if (q < QW && (MJ == 4 ? (j & 1) : j == 1)) copy_w(b + S - 1, q);
        if (i > 0) add(p[(i & 1) ^ 1][j], i - 1, j);
        QLORA_SCHED_FENCE();
      }
    }
    // every fragment of this step is in registers: the next step's tiles are awaited and the one after is sent for
    // while the last two i are still to be multiplied (three stages: the newest QW + MJ copies are of the step after)
    wait_barrier<(S - 2) * (QW + MJ)>();
    if ((b & 3) == 0 && b + 4 < b1) copy_s((b >> 2) + 1);
    QLORA_SCHED_FENCE();
    f32x4 q6, q7;
    float sn[MJ];
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const f32x4 a6 = mfma_fp8<E5M2>(wf[(IL + 1) % 3], xf[j], zero), a7 = mfma_fp8<E5M2>(wf[(IL + 2) % 3], xf[j], zero);
      QLORA_SCHED_FENCE();
      copy_x(b + S, j);
      add(p[IL & 1][j], IL, j);
      if (j > 0) {
        add(q6, IL + 1, j - 1);
        add(q7, IL + 2, j - 1);
      }
      q6 = a6;
      q7 = a7;
      xf[j] = load_x(next, j);
      sn[j] = load_s(b + 1 < b1 ? b + 1 : b, j);
      if (j == 1) w0 = load_w(next, 0);
      QLORA_SCHED_FENCE();
    }
    add(q6, IL + 1, MJ - 1);
    add(q7, IL + 2, MJ - 1);
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      sc[j] = sn[j] * wsc;
      sc2[j] = sn[j] * wsc2;
    }
  }

  wait_vmem();  // no copy into LDS outlives the workgroup

  if (cut) {
    // [part][group of four floats][thread]: one 16-byte store each, whole lines per wave
    constexpr int kGroups = MI * MJ, kPart = kGroups * 512 * 16;
    float *mine = partial + ((int64_t)tail * parts + part) * (kPart / 4);
    const rsrc_t pr = make_rsrc(mine, kPart);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), pr,
                                               (uint32_t)((i * MJ + j) * 512 + tid) * 16u, 0, 16);
    wait_vmem();
    __syncthreads();
    uint32_t *arrived = reinterpret_cast<uint32_t *>(smem);
    if (tid == 0) {
      uint32_t *line = tile_counter(counters, tail);
      *arrived = add_dev_u32(line, 1u);
      if (*arrived == (uint32_t)(parts - 1)) st_dev_u32(line, 0u);
    }
    __syncthreads();
    if (*arrived != (uint32_t)(parts - 1)) return;
    // the last to arrive adds the ranges in order, its own from its registers
    const rsrc_t all = make_rsrc(partial + (int64_t)tail * parts * (kPart / 4), (int64_t)parts * kPart);
#pragma unroll
    for (int i = 0; i < MI; i += 2) {
      f32x4 sum[2 * MJ];
#pragma unroll
      for (int q = 0; q < 2 * MJ; ++q) sum[q] = zero;
      for (int p = 0; p < parts; ++p) {
        u32x4 v[2 * MJ];
        if (p != part) {
#pragma unroll
          for (int q = 0; q < 2 * MJ; ++q)
            v[q] = bld16_dev(all, (uint32_t)((p * kGroups + i * MJ + q) * 512 + tid) * 16u);
          QLORA_SCHED_FENCE();
#pragma unroll
          for (int q = 0; q < 2 * MJ; ++q) sum[q] += __builtin_bit_cast(f32x4, v[q]);
        } else {
#pragma unroll
          for (int q = 0; q < 2 * MJ; ++q) sum[q] += acc[i + q / MJ][q % MJ];
        }
      }
#pragma unroll
      for (int q = 0; q < 2 * MJ; ++q) acc[i + q / MJ][q % MJ] = sum[q];
    }
  }

  // the adapter term: rank columns in steps of 32, operands from memory
  const int64_t nw = n0 + wn * kWaveN, tw = t0 + wt * kWaveT;
  for (int k = 8 * g; k < r + 8 * g; k += 32) {
    u32x4 sf[MJ], sl[MJ];
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      sf[j] = sl[j] = u32x4{0, 0, 0, 0};
      if (k < r && tw + j * 16 + li < T) {
        sf[j] = ld16(su + (tw + j * 16 + li) * rp + k);
        sl[j] = ld16(su + (T + tw + j * 16 + li) * rp + k);
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      u32x4 lf = {0, 0, 0, 0};
      if (k < r && nw + i * 16 + li < N) lf = ld16(L + (nw + i * 16 + li) * r + k);
#pragma unroll
      for (int j = 0; j < MJ; ++j) acc[i][j] = mfma16(lf, sf[j], mfma16(lf, sl[j], acc[i][j]));
    }
  }
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int64_t t = tw + j * 16 + li;
    if (t < T) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int64_t n = nw + i * 16 + 4 * g;
        if (n < N)
          *reinterpret_cast<u32x2 *>(out + t * N + n) =
              u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The small-tile kernel, where the large tiles are too few to fill the chip:
// 128 outputs x 64 tokens per workgroup of four waves (32 outputs x 64 tokens
// each), three steps' tiles in LDS so that two are on their way during one, and
// a K range per workgroup: `parts` workgroups share a tile, each stores its
// float32 partial, and the last to arrive sums them in range order (so the
// result does not depend on who is last) and writes the tile. Measured: 333
// tokens, 5120 x 5120 by columns: 26 us; its copies alone take 19 of them, its
// products alone as long, launch and sum 7 (in a trace with the backward's other
// launches around it: 28).
// ---------------------------------------------------------------------------
constexpr int kSmN = 128, kSmT = 64, kSmStages = 3;
constexpr int kSmStage = (kSmN + kSmT) * kStep + kSmT * 4;  // weight tile, token tile, token scales
constexpr size_t kSmLds = (size_t)kSmStages * kSmStage;

template <bool TRANS, bool E5M2>
__global__ __launch_bounds__(256, 2) void k_fp8_gemm_small(const uint8_t *__restrict__ W, const float *__restrict__ ws,
                                                           int N, int K, int ldw, int sld,
                                                           const uint8_t *__restrict__ xq, const float *__restrict__ xs,
                                                           int64_t T, const uint16_t *__restrict__ su, int rp,
                                                           const uint16_t *__restrict__ L, int r, int gn, int gt, int parts,
                                                           float *__restrict__ partial, uint32_t *__restrict__ counters,
                                                           uint16_t *__restrict__ out) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, g = lane >> 4;
  const WorkPlace at = work_place(gn * gt * parts, gn, gt, parts);
  const int part = at.part, tile = at.tt * gn + at.tn;
  const int64_t n0 = (int64_t)at.tn * kSmN, t0 = (int64_t)at.tt * kSmT;
  const int nb = (K + kStep - 1) / kStep;
  const int b0 = (int)((int64_t)nb * part / parts), b1 = (int)((int64_t)nb * (part + 1) / parts);
  const int rows_t = T - t0 < kSmT ? (int)(T - t0) : kSmT;
  const int rows_n = N - n0 < kSmN ? (int)(N - n0) : kSmN;

  const i32x4 xr = rsrc_words(xq + t0 * K, (int64_t)rows_t * K);
  const i32x4 sr = rsrc_words(xs + t0 * nb, (int64_t)rows_t * nb * 4);
  const i32x4 wr0 = rsrc_words(W + n0 * (TRANS ? 1 : (int64_t)ldw), TRANS ? 0 : (int64_t)rows_n * ldw);
  // wave w's pieces: KB 4 w .. +3 of the weight tile, KB 2 w, 2 w + 1 of the token tile
  uint32_t xv[2], wv[4];
  const int c0 = 16 * ((lane & 7) ^ ((lane >> 4) & 7)), c1 = c0 ^ 64;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = 8 * (4 * wave + q) + (lane >> 3);
    if constexpr (TRANS)
      wv[q] = (uint32_t)(row * ldw + 16 * ((lane & 7) ^ (((row >> 1) & 3) | (((row >> 4) & 1) << 2))));
    else
      wv[q] = (uint32_t)(row * ldw + ((q & 1) ? c1 : c0));
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) xv[q] = (uint32_t)((8 * (2 * wave + q) + (lane >> 3)) * K + ((q & 1) ? c1 : c0));
  // Copies of step b (six, and one more by wave 0); past b1 they read zeros, so the counts of the waits stay the same.
  auto copy = [&](int b) {
    const uint32_t base = lds_addr(smem) + (uint32_t)(b % kSmStages) * kSmStage;
    const int k0 = b < b1 ? b * kStep : K;
    i32x4 wr = wr0;
    if constexpr (TRANS) {
      const int left = K - k0 < kStep ? K - k0 : kStep;
      wr = rsrc_words(W + (int64_t)k0 * ldw + n0, left > 0 ? (int64_t)left * ldw - n0 : 0);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = k0 + ((q & 1) ? c1 : c0) < K;
      dma16_asm(wr, base + 1024u * (uint32_t)(4 * wave + q), TRANS ? wv[q] : in ? wv[q] + (uint32_t)k0 : kOOB, 0u);
      if (q < 2)
        dma16_asm(xr, base + kSmN * kStep + 1024u * (uint32_t)(2 * wave + q), in ? xv[q] + (uint32_t)k0 : kOOB, 0u);
    }
    if (wave == 0)
      dma4_asm(sr, base + (kSmN + kSmT) * kStep, b < b1 ? (uint32_t)(lane * nb + b) * 4u : kOOB, 0u);
  };

  f32x4 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t frag = (uint32_t)(li * 128 + ((g ^ ((li >> 1) & 7)) << 4));
  // transposing reads: rows of 128 bytes, chunk c of row k at c ^ ((k / 2 & 3) | (k / 16 & 1) << 2)
  const uint32_t tr_row = (uint32_t)((16 * g + (li >> 1)) * 128 + (li & 1) * 8);
  const uint32_t tr_f = (uint32_t)(((li >> 2) & 3) | ((g & 1) << 2));
  const float *wsp = ws + (n0 / 128) * (TRANS ? 1 : sld);
  const int64_t wstep = TRANS ? sld : 1;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  copy(b0);
  copy(b0 + 1);
  float wsc = wsp[b0 * wstep];
  for (int b = b0; b < b1; ++b) {
    // step b's copies have landed (step b + 1's may be on their way) and every wave has read step b - 1
    if (wave == 0)
      wait_barrier<7>();
    else
      wait_barrier<6>();
    copy(b + 2);
    const uint8_t *st = smem + (size_t)(b % kSmStages) * kSmStage;
    i32x8 wf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (TRANS) {
        const uint8_t *t = st + tr_row + (((uint32_t)(2 * wave + i) ^ tr_f) << 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const i32x2v v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(t + (q & 1) * 1024 + (q >> 1) * 8192));
          wf[i][2 * q] = v[0];
          wf[i][2 * q + 1] = v[1];
        }
      } else {
        const uint8_t *t = st + (2 * wave + i) * 2048;
        wf[i] = join8(ld16(t + frag), ld16(t + (frag ^ 64u)));
      }
    }
    const uint8_t *xt = st + kSmN * kStep;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const i32x8 xf = join8(ld16(xt + j * 2048 + frag), ld16(xt + j * 2048 + (frag ^ 64u)));
      const float sc = reinterpret_cast<const float *>(xt + kSmT * kStep)[j * 16 + li] * wsc;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 p = mfma_fp8<E5M2>(wf[i], xf, zero);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], sc, acc[i][j][e]);
      }
    }
    wsc = wsp[(b + 1 < b1 ? b + 1 : b) * wstep];
  }
  wait_vmem();  // no copy into LDS outlives the workgroup

  const int64_t nw = n0 + 32 * wave;
  if (parts > 1) {
    // lane's 8 groups of four floats, [part][group][thread]: one 16-byte store each, whole lines per wave
    float *mine = partial + ((int64_t)tile * parts + part) * (kSmN * kSmT);
    const rsrc_t pr = make_rsrc(mine, kSmN * kSmT * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), pr,
                                               (uint32_t)((i * 4 + j) * 256 + tid) * 16u, 0, 16);
    wait_vmem();
    __syncthreads();
    if (tid == 0) {
      uint32_t *line = tile_counter(counters, tile);
      arrived = add_dev_u32(line, 1u);
      if (arrived == (uint32_t)(parts - 1)) st_dev_u32(line, 0u);
    }
    __syncthreads();
    if (arrived != (uint32_t)(parts - 1)) return;
    const rsrc_t all = make_rsrc(partial + (int64_t)tile * parts * (kSmN * kSmT), (int64_t)parts * kSmN * kSmT * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = zero;
    for (int p = 0; p < parts; p += 4) {  // four parts' loads in flight; past the last they read zeros
      u32x4 v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < 8; ++q) v[u][q] = bld16_dev(all, (uint32_t)(((p + u) * 8 + q) * 256 + tid) * 16u);
      QLORA_SCHED_FENCE();
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q >> 2][q & 3] += __builtin_bit_cast(f32x4, v[u][q]);
    }
  }
  for (int k = 8 * g; k < r + 8 * g; k += 32) {
    u32x4 lf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lf[i] = u32x4{0, 0, 0, 0};
      if (k < r && nw + i * 16 + li < N) lf[i] = ld16(L + (nw + i * 16 + li) * r + k);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 sf = {0, 0, 0, 0}, sl = {0, 0, 0, 0};
      if (k < r && t0 + j * 16 + li < T) {
        sf = ld16(su + (t0 + j * 16 + li) * rp + k);
        sl = ld16(su + (T + t0 + j * 16 + li) * rp + k);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][j] = mfma16(lf[i], sf, mfma16(lf[i], sl, acc[i][j]));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t t = t0 + j * 16 + li;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = nw + i * 16 + 4 * g;
      if (t < T && n < N)
        *reinterpret_cast<u32x2 *>(out + t * N + n) =
            u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
    }
  }
}

// ---------------------------------------------------------------------------
// The weight-streaming kernel for at most 16 tokens: 16 outputs per workgroup,
// its waves take turns at the K steps (together whole lines of every row), both
// operands go from memory straight into the registers of the matrix
// instruction, kAhead steps of a wave at a time, and the waves' sums meet in LDS.
// The weight's bytes bound it: without an adapter 4096 x 4096 takes 5.9 us, 16
// tokens of 4096 x 11008 13.1 (3.5 TB/s).
//
// The adapter's u = x A^T [T, r] is formed by the first workgroups of the same
// launch (one per 16 ranks and slice of K; the last of the slices to arrive adds
// them in order) while the others stream, and reaches them as 64-bit words: half
// of a float32 and 48 bits that only this launch has (exchange.h). A reader whose
// wait runs out (other launches hold the compute units) forms what it misses
// itself, in the same order of operations, so no wait needs another workgroup to
// run and the result does not depend on who formed what.
//
// Where the slices' partials are at most one per thread of a reader (one token up
// to rank 64 of 4096 x 8192, four up to 16), every reader takes and adds those
// instead, which spares the hop through the last slice (1 token, 4096 x 4096: rank
// 16 8.6 -> 7.1 us, rank 64 9.3 -> 8.3). One compute unit reads about 28 GB/s from
// memory, so a slice is kept to about 1024 of K (16 tokens, 4096 x 11008, r = 64:
// 33.8 us with the whole of K in one workgroup, 19.8 with four slices, 17.0 with
// eleven; 18 since each value travels as a float32 instead of a bf16).
// ---------------------------------------------------------------------------
constexpr int kStreamWaves = 8, kAhead = 4;
constexpr int kUSlices = 16;  // at most
constexpr int kSuPitch = QLORA_MAX_RANK + 8;
constexpr int kDirect = 64 * kStreamWaves;  // partials that a reader takes at most: one per thread

struct StreamAdapter {
  const uint16_t *x, *A, *B;
  int r, rp, slices;
  float scale;
  float *u_out;
  bool direct;     // readers add the slices' partials themselves
  uint64_t mark;   // of this launch's words (exchange.h)
  uint64_t *ex;    // [T][rp][2] halves of u's float32 values as words; direct: [slices][T][rp][2] of the partials
  float *partial;  // [rp / 16][slices][4][64] quarters
  uint32_t *counters;
};

// Slice ks of K of u for ranks 16 rt .. +15, all tokens: lane l of wave 0 gets token l & 15, ranks 16 rt + 4 (l >> 4) + i.
__device__ __forceinline__ f32x4 u_partial(const StreamAdapter &a, int K, int T, int rt, int ks, f32x4 (*red)[64]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, g = lane >> 4;
  const int steps = (K + 31) / 32, sb = steps * ks / a.slices, se = steps * (ks + 1) / a.slices;
  const rsrc_t ar = make_rsrc(a.A, (int64_t)a.r * K * 2), xr = make_rsrc(a.x, (int64_t)T * K * 2);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = sb + wave; s0 < se; s0 += kStreamWaves * kAhead) {
    u32x4 av[kAhead], xv[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u * kStreamWaves, k = s * 32 + 8 * g;
      const bool in = s < se && k < K;
      av[u] = bld16(ar, in && 16 * rt + li < a.r ? (uint32_t)(((16 * rt + li) * K + k) * 2) : kOOB);
      xv[u] = bld16(xr, in && li < T ? (uint32_t)((li * K + k) * 2) : kOOB);
    }
    QLORA_SCHED_FENCE();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) acc = mfma16(av[u], xv[u], acc);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w) acc += red[w][lane];
  }
  __syncthreads();
  return acc;
}

template <bool E5M2>
__global__ __launch_bounds__(64 * kStreamWaves) void k_fp8_stream(const uint8_t *__restrict__ W,
                                                                  const float *__restrict__ ws, int N, int K,
                                                                  const uint8_t *__restrict__ xq,
                                                                  const float *__restrict__ xs, int T,
                                                                  StreamAdapter ad, int producers,
                                                                  uint16_t *__restrict__ out) {
  __shared__ f32x4 red[kStreamWaves][64];
  __shared__ __attribute__((aligned(16))) uint16_t su[2][16 * kSuPitch];  // s u as two bf16 terms
  __shared__ uint32_t missing[QLORA_MAX_RANK / 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, g = lane >> 4;
  if ((int)blockIdx.x < producers) {
    const int rt = blockIdx.x / ad.slices, ks = blockIdx.x - rt * ad.slices;
    f32x4 u = u_partial(ad, K, T, rt, ks, red);
    if (wave != 0) return;
    auto publish = [&](uint64_t *to, const f32x4 &v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st_dev_u64(to + 2 * i, exchange_word(ad.mark, __float_as_uint(v[i])));
        st_dev_u64(to + 2 * i + 1, exchange_word(ad.mark, __float_as_uint(v[i]) >> 16));
      }
    };
    if (ad.direct) {
      if (li < T) publish(ad.ex + 2 * (((int64_t)ks * T + li) * ad.rp + 16 * rt + 4 * g), u);
      return;
    }
    if (ad.slices > 1) {
      float *mine = ad.partial + (int64_t)rt * ad.slices * 256 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) st_dev(mine + ks * 256 + 64 * i, u[i]);
      wait_vmem();
      uint32_t *line = tile_counter(ad.counters, rt);
      uint32_t arrived = 0;
      if (lane == 0) arrived = add_dev_u32(line, 1u);
      if ((int)__builtin_amdgcn_readfirstlane(arrived) != ad.slices - 1) return;
      if (lane == 0) st_dev_u32(line, 0u);
      f32x4 q[kUSlices];
#pragma unroll
      for (int k = 0; k < kUSlices; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) q[k][i] = k < ad.slices ? ld_dev(mine + k * 256 + 64 * i) : 0.f;
      QLORA_SCHED_FENCE();
      u = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kUSlices; ++k) u += q[k];
    }
    if (li < T) {
      const int j = 16 * rt + 4 * g;
      publish(ad.ex + 2 * (li * ad.rp + j), u);
      if (ad.u_out && j < ad.r) *reinterpret_cast<f32x4 *>(ad.u_out + li * ad.r + j) = u;
    }
    return;
  }
  const bool first = (int)blockIdx.x == producers;
  const int64_t n0 = (int64_t)(blockIdx.x - producers) * 16;
  const int nb = (K + kStep - 1) / kStep;
  const rsrc_t wr = make_rsrc(W + n0 * K, (int64_t)16 * K), xr = make_rsrc(xq, (int64_t)T * K);
  const rsrc_t sr = make_rsrc(xs, (int64_t)T * nb * 4), wsr = make_rsrc(ws + n0 / 128 * nb, (int64_t)nb * 4);
  u32x4 bv = {0, 0, 0, 0};
  if (producers && 32 * wave + 8 * g < ad.r) bv = ld16(ad.B + (n0 + li) * ad.r + 32 * wave + 8 * g);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const f32x4 zero = acc;
  // operands of `kAhead` steps; steps past the last, chunks past K and tokens past T read zeros
  u32x4 wv[kAhead][2], xv[kAhead][2];
  float sx[kAhead], sw[kAhead];
  auto load = [&](int b) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = b + u * kStreamWaves, k = s * kStep + 16 * g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + 64 * h < K;
        wv[u][h] = bld16(wr, in ? (uint32_t)(li * K + k + 64 * h) : kOOB);
        xv[u][h] = bld16(xr, in && li < T ? (uint32_t)(li * K + k + 64 * h) : kOOB);
      }
      sx[u] = __uint_as_float(bld32(sr, s < nb && li < T ? (uint32_t)(li * nb + s) * 4u : kOOB));
      sw[u] = __uint_as_float(bld32(wsr, s < nb ? (uint32_t)s * 4u : kOOB));
    }
  };
  for (int b = wave; b < nb; b += kStreamWaves * kAhead) {
    load(b);
    QLORA_SCHED_FENCE();  // every load of the batch is on its way before the first use
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const f32x4 p = mfma_fp8<E5M2>(join8(wv[u][0], wv[u][1]), join8(xv[u][0], xv[u][1]), zero);
      const float s = sx[u] * sw[u];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(p[e], s, acc[e]);
    }
  }
  if (producers) {
    constexpr int kAll = 64 * kStreamWaves, kPoll = 4;  // words of a thread asked for at once
    const int tiles = ad.rp / 16, values = T * ad.rp;
    auto value_of = [](uint64_t lo, uint64_t hi) {
      return __uint_as_float((uint32_t)hi << 16 | ((uint32_t)lo & 0xffffu));
    };
    auto put = [&](int t, int j, float u) {
      uint32_t hi, lo;
      split_bf16x2(u * ad.scale, 0.f, hi, lo);
      su[0][t * kSuPitch + j] = (uint16_t)hi;
      su[1][t * kSuPitch + j] = (uint16_t)lo;
    };
    if (tid < tiles) missing[tid] = 0u;
    __syncthreads();
    const long long t0 = wall_clock64(), limit = wait_limit(ad.counters + kMaxCounters - 1);
    if (ad.direct) {
      float *const part = reinterpret_cast<float *>(red);
      while (tid < values * ad.slices) {
        const uint64_t lo = ld_dev_u64(ad.ex + 2 * tid), hi = ld_dev_u64(ad.ex + 2 * tid + 1);
        if (exchange_holds(lo, ad.mark) && exchange_holds(hi, ad.mark)) {
          part[tid] = value_of(lo, hi);
          break;
        }
        if (wall_clock64() - t0 > limit) {
          missing[tid % ad.rp / 16] = 1u;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
      __syncthreads();
      if (tid < values) {
        const int t = tid / ad.rp, j = tid - t * ad.rp;
        float u = 0.f;
        for (int ks = 0; ks < ad.slices; ++ks) u += part[ks * values + tid];
        put(t, j, u);
        if (ad.u_out && first && j < ad.r) ad.u_out[t * ad.r + j] = u;
      }
    }
    for (int e0 = tid; !ad.direct && e0 < values; e0 += kAll * kPoll) {
      for (;;) {
        uint64_t v[kPoll][2];
        bool all = true;
#pragma unroll
        for (int u = 0; u < kPoll; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) v[u][h] = e0 + u * kAll < values ? ld_dev_u64(ad.ex + 2 * (e0 + u * kAll) + h) : ad.mark;
        auto holds = [&](int u) { return exchange_holds(v[u][0], ad.mark) && exchange_holds(v[u][1], ad.mark); };
#pragma unroll
        for (int u = 0; u < kPoll; ++u) all = all && holds(u);
        const bool late = !all && wall_clock64() - t0 > limit;
        if (all || late) {
#pragma unroll
          for (int u = 0; u < kPoll; ++u) {
            const int e = e0 + u * kAll, t = e / ad.rp, j = e - t * ad.rp;
            if (e >= values) continue;
            if (holds(u))
              put(t, j, value_of(v[u][0], v[u][1]));
            else
              missing[j / 16] = 1u;
          }
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
    }
    __syncthreads();
    for (int rt = 0; rt < tiles; ++rt) {
      if (!missing[rt]) continue;  // (the same for the whole workgroup)
      if (tid == 0) add_dev_u32(ad.counters + kMaxCounters - 1, 1u);
      f32x4 u = zero;
      for (int ks = 0; ks < ad.slices; ++ks) u += u_partial(ad, K, T, rt, ks, red);
      if (wave == 0 && li < T) {
#pragma unroll
        for (int i = 0; i < 4; ++i) put(li, 16 * rt + 4 * g + i, u[i]);
      }
      if (ad.direct && ad.u_out && first && wave == 0 && li < T && 16 * rt + 4 * g < ad.r)
        *reinterpret_cast<f32x4 *>(ad.u_out + li * ad.r + 16 * rt + 4 * g) = u;
      __syncthreads();
    }
    // rank columns in steps of 32, one per wave (r <= 256)
    u32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    const int k = 32 * wave + 8 * g;
    if (k < ad.r && li < T) {
#pragma unroll
      for (int h = 0; h < 2; ++h) c[h] = *reinterpret_cast<const u32x4 *>(su[h] + li * kSuPitch + k);
    }
    acc = mfma16(bv, c[0], mfma16(bv, c[1], acc));
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (tid < 64 && li < T) {
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w) acc += red[w][lane];
    *reinterpret_cast<u32x2 *>(out + (int64_t)li * N + n0 + 4 * g) =
        u32x2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
  }
}

__global__ __launch_bounds__(256) void k_clear_words(uint64_t *__restrict__ p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0u;
}

namespace {

// How a product is cut: the large-tile kernel with 32 mi outputs x 64 mj tokens per tile, its first `full` tiles whole and the others
// in `parts` K ranges; or (mj = 0) the small-tile kernel with `parts` K ranges for every tile.
struct Fp8Plan {
  int mi, mj, parts;
  int64_t gn, gt, full;
  int64_t workgroups() const { return full + (gn * gt - full) * parts; }
};
Fp8Plan fp8_plan(int64_t T, int64_t N, int64_t K, bool trans) {
  const int64_t cus = device_cu_count(current_device()), nb = (K + kStep - 1) / kStep;
  const double cus_d = (double)cus, steps = (double)nb;
  Fp8Plan best{};
  double least = INFINITY;
  auto offer = [&](const Fp8Plan &p, double us) {
    if (us < least) {
      least = us;
      best = p;
    }
  };
  // Times in us from the measured steps. What the rule chose among (us; outputs x tokens 256 x 256, 256 x 192, 256 x 128,
  // 192 x 192, then small tiles in 1, 2, 3, 4 and 8 K ranges), the choice in brackets:
  //   515 tokens  13824 x 5120              66  57  84 [48]  67
  //   333 tokens   5120 x 5120 by columns   61  55  42   -   33 [26] 34 32 40
  //   100 tokens   4096 x 4096              46  37  31  33   19  14  12 [11] 15
  //    40 tokens   4096 x 11008            110  99  71  78   44  26  20  17 [15]
  //   768 tokens  12288 x 8192              93  83 124 [78] 121
  //  1024 tokens  11008 x 4096             [54] 93  69  76   73
  //  4096 tokens   5120 x 5120             135 [116] 128 141 161
  // Over 80 drawn shapes of 17 tokens and more a call takes 3 % longer than with the best choice on average, 56 of
  // them at most 2 %, and the worst 29 % (20 tokens, 3936 x 6656 by columns: nine K ranges, which are more workgroups
  // than compute units, where eight take 15.3 us instead of 19.8).
  // Large tiles: rounds of one workgroup per compute unit; where the last round would leave half of them idle, its tiles
  // are cut into K ranges, whose partial tiles are written once more and read by one workgroup (45 bytes a ns).
  struct Large {
    int mi, mj;
    double step, ends;
  };
  for (const Large &t : {Large{8, 4, 1.42, 7.0}, Large{8, 3, 1.25, 6.0}, Large{8, 2, 0.95, 4.7}, Large{6, 3, 1.07, 5.0}}) {
    if (trans && t.mi == 6) continue;  // (by columns the narrower tile takes as much of LDS)
    const int64_t gl = (N + 32 * t.mi - 1) / (32 * t.mi), gt = (T + 64 * t.mj - 1) / (64 * t.mj);
    const int64_t tiles = gl * gt, rest = tiles % cus;
    const double round = steps * t.step + t.ends, size = t.mi * t.mj / 8.0;
    offer(Fp8Plan{t.mi, t.mj, 1, gl, gt, tiles}, (double)((tiles + cus - 1) / cus) * round);
    const int parts = rest ? (int)std::min<int64_t>(std::min<int64_t>(cus / rest, 8), nb / 8) : 1;
    if (parts > 1 && rest <= kMaxTileCounters)
      offer(Fp8Plan{t.mi, t.mj, parts, gl, gt, tiles - rest},
            (double)(tiles / cus) * round + steps / parts * t.step + t.ends + 2.0 + 1.45 * size * (parts - 1) +
                0.008 * size * (double)(rest * parts));
  }
  // Small tiles: two workgroups share a compute unit; the last part's sum of the others
  const int64_t gn = (N + kSmN - 1) / kSmN, gt = (T + kSmT - 1) / kSmT, tiles = gn * gt;
  for (int parts = 1; parts <= 16; ++parts) {
    if (parts > 1 && (tiles > kMaxTileCounters || tiles * parts > 4 * cus || nb < 2 * parts)) break;
    const double fill = (double)(tiles * parts) / (2.0 * cus_d);
    const double rounds = fill <= 1.0 ? 1.0 : std::ceil(2.0 * fill) / 2.0;
    const double step = fill <= 0.5 ? (trans ? 0.7 : 0.5) : (trans ? 0.70 : 0.66) + 0.12 * std::min(1.0, 2.0 * fill - 1.0);
    offer(Fp8Plan{0, 0, parts, gn, gt, 0}, rounds * (std::ceil(steps / parts) * step + 3.0) +
                                         (parts > 1 ? 2.0 + 0.012 * (double)(tiles * parts) : 0.0));
  }
  return best;
}

template <typename F>
hipError_t with_lds(F *f, DeviceOnce &once, size_t bytes) {
  return once.run(current_device(), [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(f), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
}

template <bool TRANS, bool E5M2>
hipError_t product(const uint8_t *W, const float *ws, int64_t d_out, int64_t d_in, const uint8_t *xq, const float *xs,
                   int64_t T, const uint16_t *su, int rp, const uint16_t *L, int r, uint16_t *out, float *partial,
                   uint32_t *counters, hipStream_t st) {
  const int64_t N = TRANS ? d_in : d_out, K = TRANS ? d_out : d_in, sld = (d_in + 127) / 128;
  const Fp8Plan p = fp8_plan(T, N, K, TRANS);
  if (p.workgroups() >= (int64_t)1 << 31) return hipErrorInvalidValue;
  const dim3 grid((unsigned)p.workgroups());
  if (p.mj) {
    static DeviceOnce once[4];
    auto large = [&](auto *k, DeviceOnce &o, int lds) {
      const hipError_t e = with_lds(k, o, lds);
      if (e != hipSuccess) return e;
      k<<<grid, dim3(512), lds, st>>>(W, ws, (int)N, (int)K, (int)d_in, (int)sld, xq, xs, T, su, rp, L, r, (int)p.gn,
                                      (int)p.gt, (int)p.full, p.parts, partial, counters, out);
      return hipGetLastError();
    };
    if constexpr (!TRANS)
      if (p.mi == 6) return large(k_fp8_gemm<TRANS, E5M2, 6, 3, 3>, once[3], Fp8Lds<TRANS, 6, 3, 3>::bytes);
    if (p.mj == 4) return large(k_fp8_gemm<TRANS, E5M2, 8, 4, 2>, once[0], Fp8Lds<TRANS, 8, 4, 2>::bytes);
    if (p.mj == 3) return large(k_fp8_gemm<TRANS, E5M2, 8, 3, 2>, once[1], Fp8Lds<TRANS, 8, 3, 2>::bytes);
    return large(k_fp8_gemm<TRANS, E5M2, 8, 2, 3>, once[2], Fp8Lds<TRANS, 8, 2, 3>::bytes);
  }
  static DeviceOnce once;
  auto *k = k_fp8_gemm_small<TRANS, E5M2>;
  const hipError_t e = with_lds(k, once, kSmLds);
  if (e != hipSuccess) return e;
  k<<<grid, dim3(256), kSmLds, st>>>(W, ws, (int)N, (int)K, (int)d_in, (int)sld, xq, xs, T, su, rp, L, r, (int)p.gn,
                                     (int)p.gt, p.parts, partial, counters, out);
  return hipGetLastError();
}

}  // namespace

size_t fp8_partial_floats(int64_t T, int64_t N, int64_t K, bool trans) {
  const Fp8Plan p = fp8_plan(T, N, K, trans);
  if (p.parts == 1) return 0;
  return (size_t)((p.gn * p.gt - p.full) * p.parts) * (p.mj ? 32 * p.mi * 64 * p.mj : kSmN * kSmT);
}

// the words of the exchange (at least 2 kDirect), then the slices' partials
namespace {
size_t exchange_words(int rp) { return (size_t)std::max(2 * 16 * rp, 2 * kDirect); }
}  // namespace
size_t fp8_stream_exchange_bytes(int rp) { return exchange_words(rp) * 8 + (size_t)rp / 16 * kUSlices * 256 * 4; }

hipError_t launch_fp8_stream(const uint8_t *W, const float *ws, int64_t N, int64_t K, const uint8_t *xq, const float *xs,
                             bool e5m2, int64_t T, const uint16_t *x, const uint16_t *A, const uint16_t *B, int r, int rp,
                             float scale, float *u_out, void *ex, uint32_t *counters, uint16_t *out,
                             hipStream_t st) {
  static std::atomic<uint64_t> launches{0};
  const int slices = (int)std::min<int64_t>(kUSlices, (K + 1023) / 1024);
  const bool direct = T * rp * slices <= kDirect;
  if (r > 0) {
    // (a query that fails is of a stream that the launches below fail on too)
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(st, &capture) != hipSuccess) (void)hipGetLastError();
    if (capture != hipStreamCaptureStatusNone) {
      const int words = (int)T * rp * 2 * (direct ? slices : 1);
      k_clear_words<<<dim3((unsigned)((words + 255) / 256)), dim3(256), 0, st>>>(static_cast<uint64_t *>(ex), words);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const StreamAdapter ad{x, A, B, r, rp, slices, scale, u_out, direct, exchange_mark(launches.fetch_add(1)),
                         static_cast<uint64_t *>(ex),
                         reinterpret_cast<float *>(static_cast<uint64_t *>(ex) + exchange_words(rp)), counters};
  const int producers = r > 0 ? rp / 16 * slices : 0;
  const dim3 grid((unsigned)(N / 16 + producers)), block(64 * kStreamWaves);
  if (e5m2)
    k_fp8_stream<true><<<grid, block, 0, st>>>(W, ws, (int)N, (int)K, xq, xs, (int)T, ad, producers, out);
  else
    k_fp8_stream<false><<<grid, block, 0, st>>>(W, ws, (int)N, (int)K, xq, xs, (int)T, ad, producers, out);
  return hipGetLastError();
}

hipError_t launch_fp8_product(const uint8_t *W, const float *ws, int64_t d_out, int64_t d_in, bool trans,
                              const uint8_t *xq, const float *xs, bool e5m2, int64_t T, const uint16_t *su, int rp,
                              const uint16_t *L, int r, uint16_t *out, float *partial, uint32_t *counters,
                              hipStream_t st) {
  auto *f = trans ? (e5m2 ? product<true, true> : product<true, false>)
                  : (e5m2 ? product<false, true> : product<false, false>);
  return f(W, ws, d_out, d_in, xq, xs, T, su, rp, L, r, out, partial, counters, st);
}

}  // namespace qlora
