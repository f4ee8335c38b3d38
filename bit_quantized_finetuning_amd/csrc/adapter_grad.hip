// Adapter gradients of the 8-bit base's backward, both in one launch:
//   dA[r, d_in]  = s sum_t v[t, :]^T x[t, :]       v = dY B  [T, r]
//   dB[d_out, r] = s sum_t dY[t, :]^T u[t, :]      u = x A^T [T, r]
// Both are sums over tokens of a rank-sized float32 row times a wide bf16 row
// (X below), each element of which is needed once per 16 ranks' matrix
// instruction: the bytes of X bound the kernel.
//
// The float32 operand enters the bf16 matrix instructions as three terms,
// f = h + m + l: the upper 8 bits of f's significand, the next 8 and the last 8,
// all 24 of them in three products. (Two terms leave 2^-17 of f behind, which is more
// than all the rest of the sum does; the third product costs nothing here, as
// the matrix unit waits for X.)
//
// A workgroup owns 256 columns of X (64 per wave), up to 64 ranks and a range
// of tokens, in steps of 32 tokens. X tiles are copied into LDS two steps ahead
// and Y tiles one step ahead; each lane converts the 16 bytes of Y that it
// copied itself, so one barrier a step is enough. Both operands need 8
// consecutive tokens of a column per lane: ds_read_b64_tr_b16 gathers them. The
// ranks are the first operand, so that an accumulator is 4 ranks of one column:
// 64-byte runs of dA's rows, 16 bytes of dB's.
//
// Token ranges of a tile store float32 tiles and share their sum, in range
// order (split_arrive in common.h): the result does not depend on who sums it.
// Measured: 4096 tokens, 22016 + 8192 columns, rank 64: 60 us, 4.1 TB/s of X;
// 333 tokens, 5120 + 5120 columns, rank 16: 8.1 us, most of it the launch, three
// steps' latency and the sum.
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "tiles.h"

namespace qlora {

constexpr int kAgD = 256, kAgTok = 32;
constexpr int kAgX = kAgTok * 2 * kAgD;  // bytes of an X tile
constexpr int kAgMaxSplit = 16;

template <int NR>  // tiles of 16 ranks per workgroup: 1, 2 or 4
struct AgSize {
  static constexpr int raw = NR == 1 ? 4096 : 2048 * NR;   // float32 Y as copied: 1 KB a copy, every wave the same copies
  static constexpr int plane = 1024 * NR;                  // one bf16 term of a Y tile
  static constexpr int lds = 3 * kAgX + raw + 6 * plane;   // terms of two steps: 80 KB at NR = 4, two workgroups per CU
  static constexpr int copies = raw / 4096;                // Y copies per wave and step
  static constexpr int tile = 16 * NR * kAgD;              // floats of an output tile
};

// X rows take 512 bytes; 16-byte chunk c of row t sits at c ^ axsw(t): a
// transposed read (32 lanes: rows q and 8 + q, q < 4, 32 bytes each) falls on 64 banks.
__device__ __forceinline__ int axsw(int t) { return 2 * (t & 3) + (t & 8); }
// A term of a Y tile is one KB per 16 ranks: 32 rows of 32 bytes, row t at slot
// yslot(t), so that the same read takes 256 consecutive bytes; the slots of rank
// tile n are turned by n (8 / NR) to spread the stores, which take several rank tiles at once.
__device__ __forceinline__ int yslot(int t) { return (t & 19) | ((t >> 3) & 1) << 2 | ((t >> 2) & 1) << 3; }
template <int NR>
__device__ __forceinline__ int yturn(int n) {
  return NR == 1 ? 0 : n * (8 / NR);
}

template <int NR>
__global__ __launch_bounds__(256, 2) void k_adapter_grad(
    AdapterGradJob ja, AdapterGradJob jb, int tiles_a, int64_t T, int R, float scale, float *__restrict__ partial,
    uint32_t *__restrict__ counters, uint32_t *__restrict__ fallbacks, int ksplit) {
  using S = AgSize<NR>;
  constexpr int RT = 16 * NR;
  extern __shared__ __attribute__((aligned(16))) uint8_t gsm[];  // [3][X][raw Y][2][3][plane]
  uint8_t *const raw = gsm + 3 * kAgX, *const planes = raw + S::raw;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = blockIdx.x / ksplit, part = blockIdx.x - tile * ksplit;
  const bool is_b = tile >= tiles_a;
  const AdapterGradJob job = is_b ? jb : ja;
  const int gr = (R + RT - 1) / RT, jt = is_b ? tile - tiles_a : tile;
  const int64_t D = job.D, d0 = (int64_t)(jt / gr) * kAgD;
  const int r0 = (jt % gr) * RT;
  const int nkt = (int)((T + kAgTok - 1) / kAgTok);
  const int k0 = (int)((int64_t)nkt * part / ksplit), k1 = (int)((int64_t)nkt * (part + 1) / ksplit);

  // X copy q of wave w: token rows 8w + 2q, + 1; lane L fills row L/32, chunk position L%32
  uint32_t xsrc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = 8 * wave + 2 * q + (lane >> 5);
    const int64_t d = d0 + 8 * ((lane & 31) ^ axsw(row));
    xsrc[q] = d < D ? (uint32_t)((row * D + d) * 2) : kOOB;  // columns past D read zeros
  }
  // Y copies: wave w's tokens are 8w .. 8w + 7, RT/4 lanes to a token (16 ranks: the upper half of the lanes has none)
  constexpr int LT = RT / 4, TC = 64 / LT;  // lanes per token, tokens per copy
  uint32_t ysrc[S::copies], ydst[S::copies];
#pragma unroll
  for (int q = 0; q < S::copies; ++q) {
    const int row = 8 * wave + TC * q + lane / LT, c = 4 * (lane % LT), n = c >> 4;
    const bool in = TC <= 8 || lane / LT < 8;
    ysrc[q] = in && r0 + c < R ? (uint32_t)((row * R + r0 + c) * 4) : kOOB;  // ranks past R read zeros
    ydst[q] = (uint32_t)(1024 * n + 32 * (yslot(row & 31) ^ yturn<NR>(n)) + 2 * (c & 15));
  }
  auto copy_x = [&](int kt) {
    const int kc = kt < k1 ? kt : k1 - 1;  // steps past the range copy its last step again: the same counts every step
    const int64_t t0 = (int64_t)kc * kAgTok, rows = T - t0 < kAgTok ? T - t0 : kAgTok;
    const i32x4 rs = rsrc_words(job.X + t0 * D, rows * D * 2);
    const uint32_t base = lds_addr(gsm + ((kt - k0) % 3) * kAgX);
#pragma unroll
    for (int q = 0; q < 4; ++q) dma16_asm(rs, base + 1024u * (uint32_t)(4 * wave + q), xsrc[q], 0u);
  };
  auto copy_y = [&](int kt) {
    const int kc = kt < k1 ? kt : k1 - 1;
    const int64_t t0 = (int64_t)kc * kAgTok, rows = T - t0 < kAgTok ? T - t0 : kAgTok;
    const i32x4 rs = rsrc_words(job.Y + t0 * R, rows * R * 4);
    const uint32_t base = lds_addr(raw);
#pragma unroll
    for (int q = 0; q < S::copies; ++q)
      dma16_asm(rs, base + 1024u * (uint32_t)(S::copies * wave + q), ysrc[q], 0u);
  };
  // 16 bytes of Y -> 8 bytes of each term, at the lane's own places
  auto convert = [&](uint8_t *dst) {
#pragma unroll
    for (int q = 0; q < S::copies; ++q) {
      const f32x4 f = *reinterpret_cast<const f32x4 *>(raw + 1024 * (S::copies * wave + q) + 16 * lane);
      if (TC > 8 && lane / LT >= 8) continue;
      float a[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        // the upper halves: cut, not rounded, so that nothing rounds up to an infinity and three terms hold all 24 bits
        const uint32_t p0 = perm(__float_as_uint(a[1]), __float_as_uint(a[0]), 0x07060302u);
        const uint32_t p1 = perm(__float_as_uint(a[3]), __float_as_uint(a[2]), 0x07060302u);
        *reinterpret_cast<u32x2 *>(dst + term * S::plane + ydst[q]) = u32x2{p0, p1};
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (an infinity leaves nothing behind)
          a[i] = term == 0 && fabsf(a[i]) == INFINITY ? 0.f : a[i] - __uint_as_float(__float_as_uint(a[i]) & 0xffff0000u);
      }
    }
  };

  // Transposed reads: lane u of group g addresses token 8g + u/4 (then + 4), columns 4 (u%4) .. + 3 of a tile of 16,
  // and receives tokens 8g .. 8g + 7 of column u.
  const int g = lane >> 4, u = lane & 15;
  uint32_t xoff[4][2], yoff[NR][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * g + 4 * h + (u >> 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = 64 * wave + 16 * j + 4 * (u & 3);
      xoff[j][h] = (uint32_t)(row * 512 + (((c >> 3) ^ axsw(row)) << 4) + (c & 7) * 2);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n)
      yoff[n][h] = (uint32_t)(1024 * n + 32 * (yslot(row) ^ yturn<NR>(n)) + 8 * (u & 3));
  }
  auto tr = [&](const uint8_t *base, const uint32_t off[2]) {
    const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(base + off[0]));
    const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(base + off[1]));
    const u32x2 a2 = __builtin_bit_cast(u32x2, a), b2 = __builtin_bit_cast(u32x2, b);
    return u32x4{a2[0], a2[1], b2[0], b2[1]};
  };

  f32x4 acc[4][NR];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[j][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  copy_x(k0);
  copy_y(k0);
  copy_x(k0 + 1);
  for (int kt = k0; kt < k1; ++kt) {
    // Step kt's copies have landed (the next step's X may fly); the lane's own Y needs no barrier.
    asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    uint8_t *const pl = planes + ((kt - k0) & 1) * 3 * S::plane;  // last read in step kt - 2
    convert(pl);
    // X and the terms of step kt are there for all; every wave is done with step kt - 1 and with its raw Y.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    copy_y(kt + 1);
    copy_x(kt + 2);  // into the slot of step kt - 1
    const uint8_t *xs = gsm + ((kt - k0) % 3) * kAgX;
    u32x4 fx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) fx[j] = tr(xs, xoff[j]);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int term = 2; term >= 0; --term) {
        const u32x4 fy = tr(pl + term * S::plane, yoff[n]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j][n] = mfma16(fy, fx[j], acc[j][n]);
      }
  }
  wait_vmem();  // the last steps' copies (never read)

  // acc[j][n] of lane l: column 64 w + 16 j + l%16, ranks 16 n + 4 (l/16) .. + 3. A range's tile is stored in
  // register order: 16-byte chunk ((w 4 + j) NR + n) 64 + l.
  auto write = [&](int chunk, const f32x4 &v) {
    const int l = chunk & 63, n = (chunk >> 6) % NR, wj = (chunk >> 6) / NR;
    const int64_t d = d0 + 16 * wj + (l & 15);
    const int rank = r0 + 16 * n + 4 * (l >> 4);
    if (d >= D || rank >= R) return;  // R % 8 == 0: four ranks are in or out together
    const f32x4 o = v * scale;
    if (is_b) {
      *reinterpret_cast<f32x4 *>(job.out + d * R + rank) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) job.out[(int64_t)(rank + i) * D + d] = o[i];
    }
  };
  auto chunk_of = [&](int j, int n) { return ((wave * 4 + j) * NR + n) * 64 + lane; };
  if (ksplit == 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < NR; ++n) write(chunk_of(j, n), acc[j][n]);
    return;
  }
  const rsrc_t prs = make_rsrc(partial + (size_t)tile * ksplit * S::tile, (int64_t)ksplit * S::tile * 4);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int n = 0; n < NR; ++n)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[j][n]), prs,
                                             (uint32_t)(part * S::tile * 4 + 16 * chunk_of(j, n)), 0, 16);
  wait_barrier<0>();  // every wave's stores have completed, and every wave is done with LDS
  uint32_t *const claim = reinterpret_cast<uint32_t *>(raw);
  uint32_t *const line = tile_counter(counters, tile);
  if (tid == 0) {
    bool last;
    claim[0] = split_arrive(line, part, ksplit, last, fallbacks);
    claim[1] = last ? 1u : 0u;
  }
  wait_barrier<0>();
  // A power of two of ranges: every range's load of up to four chunks goes out before the first is used.
  auto sum_shares_ks = [&](uint32_t mask, auto ks_c) __attribute__((always_inline)) {
    constexpr int KS = decltype(ks_c)::value, CPB = KS >= 4 ? 16 / KS : 4;
    for (int sh = 0; sh < KS; ++sh) {
      if (!((mask >> sh) & 1u)) continue;
      const int lo = sh * (S::tile / 4) / KS, hi = (sh + 1) * (S::tile / 4) / KS;
      for (int c0 = lo + tid; c0 < hi; c0 += 256 * CPB) {
        u32x4 w[CPB][KS];
#pragma unroll
        for (int b = 0; b < CPB; ++b)
#pragma unroll
          for (int p = 0; p < KS; ++p) {
            const int c = c0 + 256 * b;
            w[b][p] = bld16_dev(prs, c < hi ? (uint32_t)(p * S::tile * 4 + 16 * c) : kOOB);
          }
#pragma unroll
        for (int b = 0; b < CPB; ++b) {
          f32x4 v = __builtin_bit_cast(f32x4, w[b][0]);
#pragma unroll
          for (int p = 1; p < KS; ++p) v += __builtin_bit_cast(f32x4, w[b][p]);
          if (c0 + 256 * b < hi) write(c0 + 256 * b, v);
        }
      }
    }
  };
  auto sum_shares = [&](uint32_t mask) __attribute__((always_inline)) {
    switch (ksplit) {
      case 2: sum_shares_ks(mask, std::integral_constant<int, 2>{}); break;
      case 4: sum_shares_ks(mask, std::integral_constant<int, 4>{}); break;
      case 8: sum_shares_ks(mask, std::integral_constant<int, 8>{}); break;
      default: sum_shares_ks(mask, std::integral_constant<int, 16>{}); break;
    }
  };
  const uint32_t mine = claim[0];
  const bool last = claim[1] != 0u;
  sum_shares(mine);
  if (last) {
    wait_barrier<0>();  // every wave has read the claim words
    if (wave == 0) {
      const uint32_t m = split_sweep(line, part, ksplit, lane);
      if (lane == 0) claim[0] = m;
    }
    wait_barrier<0>();
    sum_shares(claim[0]);
  }
  if (tid == 0) split_depart(line, ksplit);
}

namespace {
// Ranks above 64 are cut into chunks of 64 that read X again: two workgroups per CU hide each other's waits, which a
// chunk of 128 (112 KB of LDS) does not allow (4096 tokens, 22016 + 8192 columns, rank 128: 104 us against 130).
int ag_tiles16(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }
int64_t ag_tiles(int64_t D, int R) {
  const int rt = 16 * ag_tiles16(R);
  return ((D + kAgD - 1) / kAgD) * ((R + rt - 1) / rt);
}
// Ranges of tokens, a power of two, by estimated time in ns: a workgroup's steps (or X's bytes, if memory takes longer),
// and for a split what its tiles' stores and sums add. All workgroups fit on the card at two per CU, since the ranges of
// a tile wait for each other. Ranges 1 / 2 / 4 / 8 measured: 333 tokens, 5120 + 5120 columns, rank 16: 8.6 / 9.2 / 8.1 /
// 12.3 us, rank 128: 15.7 / 15.9 / 19.4 / 29 us; 4096 tokens, 22016 + 8192 columns, rank 64: 128 / 75 / 60 / 79 us.
int ag_ksplit(int64_t tiles, int R, int64_t T) {
  const int64_t room = 2 * (int64_t)device_cu_count(current_device()), nkt = (T + kAgTok - 1) / kAgTok;
  const int nr = ag_tiles16(R);
  if (tiles > kMaxTileCounters) return 1;
  const double step = 450. + 140. * nr, memory = (double)tiles * kAgD * 2 * (double)T / 4400.;
  double best = 0;
  int pick = 1;
  for (int ks = 1; ks <= kAgMaxSplit && ks <= nkt && (ks == 1 || tiles * ks <= room); ks *= 2) {
    const double steps = step * (double)((nkt + ks - 1) / ks);
    double t = steps > memory ? steps : memory;
    if (ks > 1) t += 2500. + 0.4e-3 * (double)(tiles * ks) * 16 * nr * kAgD * 4;
    if (ks == 1 || t < best) {
      best = t;
      pick = ks;
    }
  }
  return pick;
}

template <int NR>
hipError_t launch_ag(const AdapterGradJob &a, const AdapterGradJob &b, int64_t T, int R, float scale, float *partial,
                     uint32_t *counters, uint32_t *fallbacks, hipStream_t st) {
  constexpr int kLds = AgSize<NR>::lds;
  static DeviceOnce once;
  const hipError_t e = once.run(current_device(), [] {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(k_adapter_grad<NR>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  });
  if (e != hipSuccess) return e;
  const int64_t ta = a.out ? ag_tiles(a.D, R) : 0, tb = b.out ? ag_tiles(b.D, R) : 0;
  const int ks = ag_ksplit(ta + tb, R, T);
  k_adapter_grad<NR><<<dim3((unsigned)((ta + tb) * ks)), dim3(256), kLds, st>>>(a, b, (int)ta, T, R, scale, partial,
                                                                               counters, fallbacks, ks);
  return hipGetLastError();
}
}  // namespace

size_t adapter_grad_partial_floats(int64_t Da, int64_t Db, int R, int64_t T) {
  size_t most = 0;  // either gradient alone may be asked for: fewer tiles, more ranges
  const int64_t ta = ag_tiles(Da, R), tb = ag_tiles(Db, R);
  for (const int64_t t : {ta, tb, ta + tb}) {
    const int ks = ag_ksplit(t, R, T);
    if (ks > 1) most = std::max(most, (size_t)t * ks * 16 * ag_tiles16(R) * kAgD);
  }
  return most;
}

hipError_t launch_adapter_grad(const AdapterGradJob &a, const AdapterGradJob &b, int64_t T, int R, float scale,
                               float *partial, uint32_t *counters, uint32_t *fallbacks, hipStream_t st) {
  if (!a.out && !b.out) return hipSuccess;
  switch (ag_tiles16(R)) {
    case 1: return launch_ag<1>(a, b, T, R, scale, partial, counters, fallbacks, st);
    case 2: return launch_ag<2>(a, b, T, R, scale, partial, counters, fallbacks, st);
    default: return launch_ag<4>(a, b, T, R, scale, partial, counters, fallbacks, st);
  }
}

}  // namespace qlora
