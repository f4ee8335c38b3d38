// What a call over the 8-bit base does with its bf16 rows before the product, in
// one pass over them: the rows in 8 bits, and their product with the adapter,
//   out[T, r] = P[T, K] Q^T, Q = A [r, K] (u = x A^T)  or  B [K, r] (v = dY B).
// A backward call's A^T (which the product with the base takes) is written by the
// same launch.
//
// The bytes of P bound it: two read and one written per value. (Quantizer and
// adapter product in launches of their own read P twice, and the adapter matrix
// that is contracted over its other dimension was transposed first. 333 tokens,
// K = 5120, 16 ranks: 7.0 us, in three launches 11.2; 4096 tokens, K = 8192: 23 us
// with 16 ranks, in three 36; 31 with 64, in three 36.)
//
// A workgroup owns 16 tokens per wave and a range of K, in steps of one scale
// group (128). Tiles of P and Q are copied into LDS RS - 1 steps ahead. A lane's
// fragments of a step are 32 consecutive values of one token
// (4 x 8, the K of lane group g being 32 g .. 32 g + 31), so the group's maximum
// takes two exchanges between lanes and the codes leave as whole 16 bytes; the
// same registers are the second operand of the matrix instruction. The K ranges
// of a token tile are summed in range order, by whoever sums them.
#include "fp8.h"
#include "host.h"
#include "kernels.h"
#include "tiles.h"

namespace qlora {

constexpr int kRwMaxSplit = 16;

// Row t (= k of the step) of a [128][16] tile of B sits at slot rw_slot(t): 32 bytes each, so that a transposed read (32
// lanes: rows q and 32 + q, q < 4) takes 256 consecutive bytes. rw_row is its inverse.
__device__ __forceinline__ int rw_slot(int t) { return (t & 3) | ((t >> 5) & 1) << 2 | ((t >> 2) & 7) << 3 | (t & 64); }
__device__ __forceinline__ int rw_row(int s) { return (s & 3) | ((s >> 3) & 7) << 2 | ((s >> 2) & 1) << 5 | (s & 64); }
// Chunk c of a row of 256 bytes sits at c ^ rw_turn(row): a 16-byte read takes 16 lanes at a time, rows 0 .. 3 and 12 ..
// 15 of one lane group with rows 4 .. 11 of the next, and these fall on 16 different chunks (with the row itself instead:
// half of the LDS cycles were conflicts).
__device__ __forceinline__ int rw_turn(int row) { return (row + 4) & 15; }

// Stores issued from asm. The registers of a store of more than 8 bytes may not be written in the next two wait states;
// the compiler keeps that distance for stores it knows, here the s_nop behind the store does, whatever comes next.
__device__ __forceinline__ void store16_asm(const i32x4 &rs, const u32x4 &v, uint32_t off) {
  asm volatile("buffer_store_dwordx4 %0, %1, %2, 0 offen\n\ts_nop 1" : : "v"(v), "v"(off), "s"(rs) : "memory");
}
__device__ __forceinline__ void store4_asm(const i32x4 &rs, uint32_t v, uint32_t off) {
  asm volatile("buffer_store_dword %0, %1, %2, 0 offen" : : "v"(v), "v"(off), "s"(rs) : "memory");
}

// FMT: 0 no codes, 1 e4m3, 2 e5m2. BT: Q is B [K, r].
template <int FMT, bool BT, int NR, int NW, int RS>
__global__ __launch_bounds__(64 * NW) void k_fp8_rows(RowsJob a, int rp, int ksplit, int tiles_a, int extra) {
  constexpr int kRwTok = 16 * NW, kRwP = 4096 * NW;  // tokens, bytes of a step's P tile
  constexpr int RT = 16 * NR, kSlot = kRwP + 4096 * NR, QC = 4 * NR / NW, kCopies = 4 + QC, kStores = FMT ? 3 : 0;
  static_assert(QC * NW == 4 * NR);
  extern __shared__ __attribute__((aligned(16))) uint8_t rsm[];  // [RS][P tile, Q tile]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Pieces i0, + every, .. of A^T: 32 ranks and 128 columns of A each, 32 x 32 at a time through LDS.
  auto transposes = [&](int i0, int every) __attribute__((always_inline)) {
    constexpr int NY = 2 * NW, NI = 32 / NY;  // rows at a time, times
    uint16_t(*t)[33] = reinterpret_cast<uint16_t(*)[33]>(rsm);
    const int tr = (a.r + 31) / 32, tx = tid & 31, ty = tid >> 5;
    for (; i0 < tiles_a; i0 += every) {
      const int64_t r0 = (int64_t)(i0 % tr) * 32, c0 = (int64_t)(i0 / tr) * 128;
      uint16_t v[4][NI];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int64_t row = r0 + ty + NY * i, col = c0 + 32 * j + tx;
          v[j][i] = row < a.r && col < a.d_lt ? a.A[row * a.d_lt + col] : (uint16_t)0;
        }
      __syncthreads();  // every wave is done with LDS
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) t[32 * j + ty + NY * i][tx] = v[j][i];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int64_t col = c0 + 32 * j + ty + NY * i, row = r0 + tx;
          if (col < a.d_lt && row < a.r) a.lt[col * a.r + row] = t[32 * j + tx][ty + NY * i];
        }
    }
  };
  // A^T by workgroups of their own where compute units are left for them, else on the side of the others' stores
  const int main = gridDim.x - extra;
  if ((int)blockIdx.x >= main) return transposes(blockIdx.x - main, extra);
  const int li = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / ksplit, part = blockIdx.x - tile * ksplit;
  const int64_t t0 = (int64_t)tile * kRwTok, K = a.K, T = a.T;
  const int nk = (int)((K + 127) / 128);
  const int k0 = (int)((int64_t)nk * part / ksplit), k1 = (int)((int64_t)nk * (part + 1) / ksplit);
  const int64_t rows = T - t0 < kRwTok ? T - t0 : kRwTok;
  const i32x4 pr = rsrc_words(a.P + t0 * K, rows * K * 2), qr = rsrc_words(a.Q, (int64_t)a.r * K * 2);
  const i32x4 cr = rsrc_words(FMT ? a.codes + t0 * K : nullptr, FMT ? rows * K : 0);
  const i32x4 sr = rsrc_words(FMT ? a.scales + t0 * nk : nullptr, FMT ? rows * nk * 4 : 0);

  // P: wave w's rows are 16 w .. +15 of the tile, 256 bytes each, 16-byte chunk c of row t at c ^ rw_turn(t); copy q takes
  // rows 4 q .. +3 of them. Q by rows: 16 ranks' tiles of the same form; B's: [128][16] tiles by rw_slot. Copies of Q:
  // wave w takes KB w QC .. +QC-1. A chunk at or past K reads zeros, as do rows past T, r and K.
  uint32_t psrc[4], qsrc[QC];
  int pk[4], qk[QC];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = 4 * q + (lane >> 4);
    pk[q] = 8 * ((lane & 15) ^ rw_turn(row));
    psrc[q] = (uint32_t)(((16 * wave + row) * K + pk[q]) * 2);
  }
#pragma unroll
  for (int j = 0; j < QC; ++j) {
    const int kb = wave * QC + j, n = kb >> 2, q = kb & 3;
    if constexpr (BT) {
      const int row = rw_row(32 * q + (lane >> 1)), col = 16 * n + 8 * (lane & 1);
      qk[j] = row;
      qsrc[j] = col < a.r ? (uint32_t)((row * a.r + col) * 2) : kOOB;
    } else {
      const int row = 4 * q + (lane >> 4);
      qk[j] = 8 * ((lane & 15) ^ rw_turn(row));
      qsrc[j] = 16 * n + row < a.r ? (uint32_t)(((int64_t)(16 * n + row) * K + qk[j]) * 2) : kOOB;
    }
  }
  auto copy = [&](int kt) {
    const int kc = kt < k1 ? kt : k1 - 1;  // steps past the range copy its last again: the same counts every step
    const uint32_t base = lds_addr(rsm + ((kt - k0) % RS) * kSlot);
    const int left = (int)(K - (int64_t)kc * 128);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      dma16_asm(pr, base + 1024u * (uint32_t)(4 * wave + q), pk[q] < left ? psrc[q] + (uint32_t)kc * 256u : kOOB, 0u);
#pragma unroll
    for (int j = 0; j < QC; ++j) {
      const uint32_t at = qsrc[j] + (uint32_t)kc * (BT ? 256u * (uint32_t)a.r : 256u);  // (past kOOB, and below 2^32, stays outside)
      dma16_asm(qr, base + kRwP + 1024u * (uint32_t)(wave * QC + j), BT || qk[j] < left ? at : kOOB, 0u);
    }
  };
  // The codes' stores count among the wave's outstanding operations as the copies do: every step has three, issued from
  // asm so that there are neither more nor fewer, which write nothing where there is nothing to write (before the first
  // step, past K, past T).
  auto store = [&](const u32x4 &lo, const u32x4 &hi, float s, uint32_t lo_at, uint32_t hi_at, uint32_t s_at) {
    store16_asm(cr, lo, lo_at);
    store16_asm(cr, hi, hi_at);
    store4_asm(sr, __float_as_uint(s), s_at);
  };

  f32x4 acc[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t pfrag = (uint32_t)((16 * wave + li) * 256);
  uint32_t qfrag[2];
  if constexpr (BT) {
#pragma unroll
    for (int h = 0; h < 2; ++h) qfrag[h] = (uint32_t)(32 * rw_slot(32 * g + 4 * h + (li >> 2)) + 8 * (li & 3));
  } else {
    qfrag[0] = (uint32_t)(li * 256);
  }

#pragma unroll
  for (int s = 0; s < RS - 1; ++s) {
    copy(k0 + s);
    if constexpr (FMT) store(u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}, 0.f, kOOB, kOOB, kOOB);
  }
  for (int kt = k0; kt < k1; ++kt) {
    // step kt's copies have landed (later steps' and the stores since may be on their way); every wave is done with kt - 1
    wait_barrier<(RS - 2) * kCopies + (RS - 1) * kStores>();
    copy(kt + RS - 1);
    const uint8_t *ps = rsm + ((kt - k0) % RS) * kSlot, *qs = ps + kRwP;
    u32x4 p[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) p[kk] = ld16(ps + pfrag + (((4 * g + kk) ^ rw_turn(li)) << 4));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        u32x4 f;
        if constexpr (BT) {
          // rows 32 g + 8 kk + 4 h + ..: 8 kk is 16 slots on (bits 3 and 4 of the row are bits 4 and 5 of the slot)
          const uint8_t *b = qs + 4096 * n + 512 * kk;
          const u32x2 f0 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(b + qfrag[0])));
          const u32x2 f1 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(b + qfrag[1])));
          f = u32x4{f0[0], f0[1], f1[0], f1[1]};
        } else {
          f = ld16(qs + 4096 * n + qfrag[0] + (((4 * g + kk) ^ rw_turn(li)) << 4));
        }
        acc[n] = mfma16(f, p[kk], acc[n]);
      }
    if constexpr (FMT) {
      float m = 0.f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = fmaxf(m, fmaxf(fabsf(bf16_lo_to_f32(p[kk][i])), fabsf(bf16_hi_to_f32(p[kk][i]))));
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const RowScale sc = row_scale<FMT == 2>(m);
      u32x4 c[2];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          c[kk >> 1][2 * (kk & 1) + i] =
              pack_fp8x4<FMT == 2>(bf16_lo_to_f32(p[kk][2 * i]) * sc.inv, bf16_hi_to_f32(p[kk][2 * i]) * sc.inv,
                                   bf16_lo_to_f32(p[kk][2 * i + 1]) * sc.inv, bf16_hi_to_f32(p[kk][2 * i + 1]) * sc.inv);
      const int row = 16 * wave + li, k = kt * 128 + 32 * g;
      const uint32_t at = (uint32_t)(row * K + k);  // (rows past T are past the range's end)
      store(c[0], c[1], sc.s, k < K ? at : kOOB, k + 16 < K ? at + 16u : kOOB, g == 0 ? (uint32_t)(row * nk + kt) * 4u : kOOB);
    }
  }
  wait_vmem();  // no copy into LDS outlives the workgroup

  // acc[n] of lane l: token 16 w + l % 16, ranks 16 n + 4 (l / 16) .. + 3
  auto write = [&](int tok, int j, const f32x4 &v) {
    const int64_t t = t0 + tok;
    if (t >= T) return;
    const bool real = j < a.r;  // r % 8 == 0: four ranks are in or out together
    if (a.out_f32 && real) *reinterpret_cast<f32x4 *>(a.out_f32 + t * a.r + j) = v;
    if (a.out_terms && j < rp) {
      u32x2 hi = {0, 0}, lo = {0, 0};
      if (real) {
        uint32_t h0, l0, h1, l1;
        split_bf16x2(a.scale * v[0], a.scale * v[1], h0, l0);
        split_bf16x2(a.scale * v[2], a.scale * v[3], h1, l1);
        hi = u32x2{h0, h1};
        lo = u32x2{l0, l1};
      }
      *reinterpret_cast<u32x2 *>(a.out_terms + t * rp + j) = hi;
      *reinterpret_cast<u32x2 *>(a.out_terms + (T + t) * rp + j) = lo;
    }
  };
  if (ksplit == 1) {
#pragma unroll
    for (int n = 0; n < NR; ++n) write(16 * wave + li, 16 * n + 4 * g, acc[n]);
    if (!extra) transposes(blockIdx.x, main);
    return;
  }
  // a range's float32 tile in register order: 16-byte chunk (w NR + n) 64 + l
  constexpr int kTile = kRwTok * RT;
  const rsrc_t prs = make_rsrc(a.partial + (size_t)tile * ksplit * kTile, (int64_t)ksplit * kTile * 4);
#pragma unroll
  for (int n = 0; n < NR; ++n)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[n]), prs,
                                           (uint32_t)(part * kTile * 4 + 16 * ((wave * NR + n) * 64 + lane)), 0, 16);
  if (!extra) transposes(blockIdx.x, main);
  wait_barrier<0>();  // every wave's stores have completed, and every wave is done with LDS
  uint32_t *const claim = reinterpret_cast<uint32_t *>(rsm);
  uint32_t *const line = tile_counter(a.counters, tile);
  // (every range's load of a chunk goes out before the first is used; ranges past the last read zeros)
  constexpr int kChunks = kTile / 4;
  auto sum = [&](int lo, int hi) __attribute__((always_inline)) {
    for (int c = lo + tid; c < hi; c += 64 * NW) {
      u32x4 w[kRwMaxSplit];
#pragma unroll
      for (int p = 0; p < kRwMaxSplit; ++p) w[p] = bld16_dev(prs, p < ksplit ? (uint32_t)(p * kTile * 4 + 16 * c) : kOOB);
      f32x4 v = __builtin_bit_cast(f32x4, w[0]);
#pragma unroll
      for (int p = 1; p < kRwMaxSplit; ++p) v += __builtin_bit_cast(f32x4, w[p]);
      write(16 * ((c >> 6) / NR) + (c & 15), 16 * ((c >> 6) % NR) + 4 * ((c >> 4) & 3), v);
    }
  };
  auto sum_shares = [&](uint32_t mask) __attribute__((always_inline)) {
    for (int sh = 0; sh < ksplit; ++sh)
      if ((mask >> sh) & 1u) sum(kChunks * sh / ksplit, kChunks * (sh + 1) / ksplit);
  };
  // Few ranks: the last to arrive adds all the ranges, since waiting for each other takes longer (333 tokens, K = 5120, 32
  // ranks: 6.9 us against 8.4; with 64 ranks the shared sum takes 3 us less).
  if constexpr (NR <= 2) {
    if (tid == 0) {
      const uint32_t prev = add_dev_u32(line, 1u);
      if (prev == (uint32_t)(ksplit - 1)) st_dev_u32(line, 0u);
      claim[0] = prev;
    }
    wait_barrier<0>();
    if (claim[0] == (uint32_t)(ksplit - 1)) sum(0, kChunks);
    return;
  }
  if (tid == 0) {
    bool last;
    claim[0] = split_arrive(line, part, ksplit, last, a.counters + kMaxCounters - 1);
    claim[1] = last ? 1u : 0u;
  }
  wait_barrier<0>();
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
// Tiles of 16 ranks (the adapter's own number, rounded up to a power of two), waves, steps in LDS. Two waves share a
// SIMD, so that one's copies are awaited while the other converts: two workgroups of four waves up to 64 ranks (at most
// 80 KB each; 64 ranks and 333 tokens, K = 5120: 10.4 us, one workgroup of eight waves 12.8; at 4096 tokens the same),
// one of eight up to 128 (4096 tokens, K = 8192, codes not wanted: 24 us, one of four waves 27); above, the ranks'
// tile leaves room for one of four.
int rw_tiles16(int rp) { return rp <= 16 ? 1 : rp <= 32 ? 2 : rp <= 64 ? 4 : rp <= 128 ? 8 : 16; }
int rw_tokens(int rp) { return rp <= 64 || rp > 128 ? 64 : 128; }
int64_t rw_room(int rp) { return (int64_t)device_cu_count(current_device()) * (rp <= 64 ? 2 : 1); }
// K ranges per token tile: as many as fill the card
int rw_ksplit(int64_t T, int64_t K, int rp) {
  const int64_t tiles = (T + rw_tokens(rp) - 1) / rw_tokens(rp), nk = (K + 127) / 128;
  if (tiles > kMaxTileCounters) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(rw_room(rp) / tiles, nk), kRwMaxSplit));
}

template <int FMT, bool BT, int NR, int NW, int RS>
hipError_t rows_launch(const RowsJob &a, int rp, hipStream_t st) {
  constexpr int kLds = RS * 4096 * (NW + NR);
  static DeviceOnce once;
  const hipError_t e = once.run(current_device(), [] {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(k_fp8_rows<FMT, BT, NR, NW, RS>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  });
  if (e != hipSuccess) return e;
  const int ks = rw_ksplit(a.T, a.K, rp);
  const int ta = a.lt ? (a.r + 31) / 32 * (int)((a.d_lt + 127) / 128) : 0;
  const int64_t main = (a.T + 16 * NW - 1) / (16 * NW) * ks;
  const int extra = main + ta <= rw_room(rp) ? ta : 0;
  k_fp8_rows<FMT, BT, NR, NW, RS><<<dim3((unsigned)(main + extra)), dim3(64 * NW), kLds, st>>>(a, rp, ks, ta, extra);
  return hipGetLastError();
}
template <int FMT, bool BT>
hipError_t rows_by_rank(const RowsJob &a, int rp, hipStream_t st) {
  switch (rw_tiles16(rp)) {
    case 1: return rows_launch<FMT, BT, 1, 4, 4>(a, rp, st);
    case 2: return rows_launch<FMT, BT, 2, 4, 3>(a, rp, st);
    case 4: return rows_launch<FMT, BT, 4, 4, 2>(a, rp, st);
    case 8: return rows_launch<FMT, BT, 8, 8, 2>(a, rp, st);
    default: return rows_launch<FMT, BT, 16, 4, 2>(a, rp, st);
  }
}
}  // namespace

size_t fp8_rows_partial_floats(int64_t T, int64_t K, int rp) {
  const int ks = rw_ksplit(T, K, rp);
  return ks > 1 ? (size_t)((T + rw_tokens(rp) - 1) / rw_tokens(rp)) * ks * rw_tokens(rp) * 16 * rw_tiles16(rp) : 0;
}

hipError_t launch_fp8_rows(const RowsJob &a, int fmt, bool q_is_b, int rp, hipStream_t st) {
  if (!a.codes) return q_is_b ? rows_by_rank<0, true>(a, rp, st) : rows_by_rank<0, false>(a, rp, st);
  if (fmt == QLORA_E5M2) return q_is_b ? rows_by_rank<2, true>(a, rp, st) : rows_by_rank<2, false>(a, rp, st);
  return q_is_b ? rows_by_rank<1, true>(a, rp, st) : rows_by_rank<1, false>(a, rp, st);
}

}  // namespace qlora
