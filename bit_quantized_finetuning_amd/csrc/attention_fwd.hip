// Attention with a sliding window and sinks, forward (see attention.h).
//
// k_attn_fwd: a workgroup of four waves takes 128 packed rows of one key head,
// 32 per wave; key and value tiles of 32 go from memory straight into LDS, four
// of each in a ring. One pass over the keys with the running maximum and sum of
// the softmax in float32. The softmax of tile i is vector work in the shadow of
// the matrix work of its neighbours: a step runs V P of tile i - 1 and K Q^T of
// tile i + 1, and the pieces of tile i's softmax stand between their products.
// Two workgroups share a compute unit, so that one's first loads and last
// stores (113 of 309 us at 4 x 4096 tokens with one of 256 rows) are hidden.
// The bookkeeping of a step is kept to a few scalar instructions, and no wave
// skips a tile that only others of its workgroup see. 4 x 4096 ragged tokens, 40
// over 8 heads, window 1024: 280 us, the matrix unit busy 40 % of the cycles;
// some 205 instructions per tile and wave, two waves a SIMD. Of a wave's time
// (counters) 47 % are an instruction's of its own, 30 % it waits for its turn or a
// busy unit, 23 % for data. A wave alone on its SIMD (777 tokens behind 1000) takes
// some 1450 cycles a tile, 512 of them matrix work: 51, 17 and 32 %.
//
// k_attn_split: few rows (single tokens): a workgroup takes 32 rows and every
// kSplit-th run of key tiles; each wave streams tiles of its own, with no
// barrier. The parts' maxima, sums and outputs are joined by the workgroup that
// arrives last, in the order of the parts.
#include "attention.h"
#include "kernels.h"

namespace qlora {

struct AttnOut {
  uint16_t *o;  // [B, T, H, D] dense
  float *lse;   // [B, H, T], nullable
};

// The softmax state of a lane's row: the running maximum of the raw scores (both halves'), the sum of this half's
// weights, the unnormalized output.
template <int D>
struct RowState {
  float m, l;
  f32x16 o[D / 32];
  __device__ __forceinline__ void init() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o[d] = zero16();
  }
};

// One tile of kSub x 32 keys against a wave's 32 rows. `full`: every row sees every key.
template <int D, int kSub>
__device__ __forceinline__ void attn_tile(const AttnArgs &a, const TileReads<D> &rd, const uint8_t *kt,
                                          const uint8_t *vt, const u32x4 (&qf)[D / 16], int key0, int p, bool full,
                                          int half, RowState<D> &st) {
  f32x16 s[kSub];
#pragma unroll
  for (int b = 0; b < kSub; ++b) {
    s[b] = zero16();
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s[b] = mfma32(rd.rows(kt, b, i, half), qf[i], s[b]);
  }
  if (!full) {
#pragma unroll
    for (int b = 0; b < kSub; ++b) attn_mask(a, p, key0 + 32 * b, half, s[b]);
  }
  float mx = s[0][0];
#pragma unroll
  for (int b = 0; b < kSub; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[b][e]);
  mx = fmaxf(st.m, halves_max(mx));
  // rows that have seen nothing yet count from 0 (their weights are all exp2(-inf))
  const float from = mx == -INFINITY ? 0.f : mx;
  if (__any(mx > st.m)) {
    const float f = __builtin_amdgcn_exp2f((st.m - from) * a.c);
    st.l *= f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) st.o[d][e] *= f;
    st.m = mx;
  }
  const float mc = from * a.c;
  float sum = 0.f;
#pragma unroll
  for (int b = 0; b < kSub; ++b)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      s[b][e] = __builtin_amdgcn_exp2f(fmaf(s[b][e], a.c, -mc));
      sum += s[b][e];
    }
  st.l += sum;
#pragma unroll
  for (int b = 0; b < kSub; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 pf = pack_frag(s[b], i);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) st.o[d] = mfma32(rd.cols(vt, b, i, d), pf, st.o[d]);
    }
}

// A lane's query row: its 8-value runs as B fragments, zeros for rows past the last.
template <int D>
__device__ __forceinline__ void load_row(const AttnRows &x, int b, int t, int head, bool ok, int half,
                                         u32x4 (&f)[D / 16]) {
  const uint16_t *p = x.p + b * x.b + t * x.t + head * x.h + 8 * half;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) f[i] = ok ? ld16(p + 16 * i) : u32x4{0u, 0u, 0u, 0u};
}

// Output row and the logarithm of its sum. A row that sees nothing (`some` false) gives 0 and -inf; one whose scores are all
// -inf has a sum of 0 and gives NaN, as the formula does.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs &a, const AttnOut &out, int b, int t, int head, bool write,
                                          bool some, int half, float m, float l, f32x16 (&o)[D / 32]) {
  const float inv = 1.f / l;
  uint16_t *row = out.o + (((int64_t)b * a.T + t) * a.H + head) * D;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = some ? o[d][e] * inv : 0.f;
    u32x4 run[2];
    column_runs(o[d], run);
    if (write) {
      st16(row + 32 * d + 8 * half, run[0]);
      st16(row + 32 * d + 16 + 8 * half, run[1]);
    }
  }
  if (out.lse && write && half == 0)
    out.lse[((int64_t)b * a.H + head) * a.T + t] =
        some ? (m * a.c + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : -INFINITY;
}

// The softmax of a tile of 32 keys in 16 pieces of a few vector instructions. The running maximum moves only where a
// score lies more than 2^8 above it (`grow`, for the wave as a whole): weights up to 2^8 lose nothing in float32 or, being
// rounded relatively, in bf16, and the rescaling of the output becomes rare.
struct SoftmaxPieces {
  float t0, t1, mx, mc, old, sum0, sum1;
  bool grow;
  __device__ __forceinline__ void run(int k, f32x16 &s, float c, float &m, u32x4 (&pf)[2]) {
    if (k == 0) {
      t0 = fmaxf(fmaxf(s[0], s[1]), s[2]);
      t1 = fmaxf(fmaxf(s[3], s[4]), s[5]);
      t0 = fmaxf(fmaxf(t0, s[6]), s[7]);
      t1 = fmaxf(fmaxf(t1, s[8]), s[9]);
      pin(t0);
      pin(t1);
    } else if (k == 1) {
      t0 = fmaxf(fmaxf(t0, s[10]), s[11]);
      t1 = fmaxf(fmaxf(t1, s[12]), s[13]);
      t0 = fmaxf(fmaxf(t0, s[14]), s[15]);
      mx = fmaxf(t0, t1);
      pin(mx);
    } else if (k == 2) {
      mx = halves_max(mx);
      grow = __any((mx - m) * c > 8.f);
    } else if (k == 3) {
      old = m;
      const float to = fmaxf(m, mx);
      m = grow ? to : m;
      mc = (m == -INFINITY ? 0.f : m) * c;
      sum0 = sum1 = 0.f;
      pin(mc);
    } else if (k < 12) {
      const int e = 2 * (k - 4);
      s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -mc));
      s[e + 1] = __builtin_amdgcn_exp2f(fmaf(s[e + 1], c, -mc));
      sum0 += s[e];
      sum1 += s[e + 1];
      pin(sum0);
      pin(sum1);
    } else {
      const int w = 2 * (k - 12);
#pragma unroll
      for (int j = w; j < w + 2; ++j) {
        uint32_t x = pack_bf16x2(s[2 * j], s[2 * j + 1]);
        pin(x);
        pf[j >> 2][j & 3] = x;
      }
    }
  }
};

constexpr int kFwdThreads = 256, kFwdRows = 128;

template <int D>
__global__ __launch_bounds__(kFwdThreads, 2) void k_attn_fwd(AttnArgs a, AttnOut out, int tiles) {
  constexpr int kKeys = 32, kTileBytes = kKeys * kRowBytes<D>, kSlots = 4, kQk = D / 16, kPv = D / 16, kDt = D / 32;
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * kSlots * kTileBytes];  // keys, then values
  uint8_t *const kring = ring, *const vring = ring + kSlots * kTileBytes;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, ml = lane & 31;
  int bg, tile;
  attn_work(blockIdx.x, a.B * a.G, tiles, bg, tile);
  const int b = bg / a.G, g = bg - b * a.G;
  int n, off;
  attn_sequence(a, b, n, off);
  const int R = a.T * a.rep;
  const int wg0 = tile * kFwdRows, row0 = wg0 + 32 * wave;
  const int wg1 = wg0 + kFwdRows < R ? wg0 + kFwdRows - 1 : R - 1, row1 = row0 + 31 < R ? row0 + 31 : R - 1;
  const int c = row0 + ml, t = c / a.rep, head = g * a.rep + c - t * a.rep;
  const int p = c < R ? attn_position(t, off, n) : -1;
  u32x4 qf[D / 16];

  const int p0 = off + wg0 / a.rep > 0 ? off + wg0 / a.rep : 0, p1 = off + wg1 / a.rep < n ? off + wg1 / a.rep : n - 1;
  KeyTiles kts{0, 0, 0};
  if (p0 <= p1) kts = key_tiles(a, p0, p1, kKeys);
  const int count = kts.count;
  // the wave's own positions
  const int q0 = off + row0 / a.rep > 0 ? off + row0 / a.rep : 0, q1 = off + row1 / a.rep < n ? off + row1 / a.rep : n - 1;

  const TileReads<D> rd(lane);
  constexpr int kN = TileCopy<D, kKeys, 4>::kN;  // copies of a wave per tile
  RowState<D> st;
  st.init();
  auto mask = [&](int key0, f32x16 &s) {
    const int key1 = key0 + kKeys - 1;
    if (!(key1 <= q0 && (q1 - key0 < a.window || key1 < a.sinks))) attn_mask(a, p, key0, half, s);
  };
  if (count > 0) {
    // Tile i lies in slot i % 4. Step i, behind a barrier, issues keys i + 4 and values i + 2 (past the last tile that
    // one again: always the same number of copies) into slots whose tiles every wave has finished; those issued two
    // steps ago have come in: keys to i + 2 and values to i, which is as far as the reads go until the next barrier.
    // Values "-1" are zeros.
    TileStream<D, kKeys, 4> ks, vs;
    ks.set(a.k.p + b * a.k.b + g * a.k.h, a.k.t, kts, n, wave, lane);
    vs.set(a.v.p + b * a.v.b + g * a.v.h, a.v.t, kts, n, wave, lane);
    const uint32_t kto = lds_addr(kring) + 1024u * (uint32_t)(wave * kN), vto = kto + kSlots * kTileBytes;
#pragma unroll
    for (int i = 0; i < 3; ++i) ks.issue(kto + i * kTileBytes, true);
    vs.issue(vto, true);
    ks.issue(kto + 3 * kTileBytes, true);
    vs.issue(vto + kTileBytes, true);
    load_row<D>(a.q, b, t, head, c < R, half, qf);  // (behind the copies: one trip to memory for both)
    for (int i = tid; i < kTileBytes / 16; i += kFwdThreads) st16(vring + 3 * kTileBytes + 16 * i, u32x4{0u, 0u, 0u, 0u});
    wait_barrier<2 * kN>();
    RingReads<D> rr;
    rr.set_rows(kring, rd, half);
    rr.set_cols(vring, rd);
    u32x4 pf[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}}, kf[2], vf[2];
    auto load_k = [&](int slot, int k) { kf[k & 1] = rr.rows(slot * kTileBytes, k); };
    auto load_v = [&](int slot, int j) { vf[j & 1] = rr.cols(slot * kTileBytes, j / kDt, j % kDt); };
    f32x16 sc[2];  // scores; between steps those of tile i in sc[0]
    sc[0] = zero16();
    int key0 = kts.key0(0, kKeys);  // of the tile whose scores are formed
#pragma unroll
    for (int k = 0; k < kQk; ++k) sc[0] = mfma32(rr.rows(0, k), qf[k], sc[0]);
    mask(key0, sc[0]);
    load_k(1, 0);
    load_k(1, 1);
    load_v(3, 0);
    load_v(3, 1);
    // the products around tile i in slot S: scores of i in s, of i + 1 into next
    auto products = [&](const int S, f32x16 &s, f32x16 &next) {
      const int s1 = (S + 1) & 3, s2 = (S + 2) & 3, sb = (S + 3) & 3;
      u32x4 pn[2];
      SoftmaxPieces sp;
#pragma unroll
      for (int q = 0; q < kQk; ++q) {
        next = mfma32(kf[q & 1], qf[q], q ? next : zero16());
        QLORA_SCHED_FENCE();
        if (q + 2 < kQk)
          load_k(s1, q + 2);
        else
          load_k(s2, q + 2 - kQk);
#pragma unroll
        for (int k = 0; k < 8 / kQk; ++k) sp.run((16 / kQk) * q + k, s, a.c, st.m, pn);
        QLORA_SCHED_FENCE();
        st.o[q % kDt] = mfma32(vf[q & 1], pf[q / kDt], st.o[q % kDt]);
        QLORA_SCHED_FENCE();
        if (q + 2 < kPv)
          load_v(sb, q + 2);
        else
          load_v(S, q + 2 - kPv);
#pragma unroll
        for (int k = 0; k < 8 / kQk; ++k) sp.run((16 / kQk) * q + 8 / kQk + k, s, a.c, st.m, pn);
        QLORA_SCHED_FENCE();
      }
      if (sp.grow) {
        asm volatile("; rescale");  // (rare: a branch, no multiplication by 1)
        const float scale = __builtin_amdgcn_exp2f((sp.old - (st.m == -INFINITY ? 0.f : st.m)) * a.c);
        st.l *= scale;
#pragma unroll
        for (int d = 0; d < kDt; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) st.o[d][e] *= scale;
      }
      st.l += sp.sum0 + sp.sum1;
      pf[0] = pn[0];
      pf[1] = pn[1];
    };
    const int gap = (kts.w0 - kts.ns + 1) * kKeys;
    auto step = [&](int i, const int S) {
      wait_barrier<2 * kN>();
      ks.issue(kto + S * kTileBytes, true);
      vs.issue(vto + ((S + 2) & 3) * kTileBytes, true);
      // (the list is taken to an even length: nobody sees the tile behind it)
      key0 = i + 1 < count ? key0 + (i + 1 == kts.ns ? gap : kKeys) : 1 << 29;
      products(S, sc[S & 1], sc[(S + 1) & 1]);
      mask(key0, sc[(S + 1) & 1]);
    };
    for (int i = 0;; i += 4) {
      step(i, 0);
      step(i + 1, 1);
      if (i + 2 >= count) break;
      step(i + 2, 2);
      step(i + 3, 3);
      if (i + 4 >= count) break;
    }
    // the last tile's V P
    wait_barrier<0>();
    const int at = ((count - 1 | 1) & 3) * kTileBytes;
#pragma unroll
    for (int j = 0; j < kPv; ++j) st.o[j % kDt] = mfma32(rr.cols(at, j / kDt, j % kDt), pf[j / kDt], st.o[j % kDt]);
  }
  store_row<D>(a, out, b, t, head, c < R, p >= 0, half, st.m, halves_sum(st.l), st.o);
}

// ---------------------------------------------------------------------------
// few rows: the keys split over workgroups and waves
// ---------------------------------------------------------------------------
constexpr int kSplitWaves = 4, kSplitKeys = 32, kMaxSplits = 64;

// Partials of one (row tile, split): the output [32][D], then maxima and sums of 32 rows.
template <int D>
constexpr int kPartFloats = 32 * D + 64;

template <int D>
__global__ __launch_bounds__(64 * kSplitWaves) void k_attn_split(AttnArgs a, AttnOut out, int row_tiles, int splits,
                                                                 float *partial, uint32_t *counters) {
  constexpr int kTileBytes = kSplitKeys * kRowBytes<D>, kDt = D / 32;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // per wave [2][keys | values]; then the join
  __shared__ float ml_lds[2][kSplitWaves][64];
  __shared__ uint32_t last_lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, mlane = lane & 31;
  const int work = blockIdx.x / splits, split = blockIdx.x - work * splits;
  const int bg = work / row_tiles, tile = work - bg * row_tiles;
  const int b = bg / a.G, g = bg - b * a.G;
  int n, off;
  attn_sequence(a, b, n, off);
  const int R = a.T * a.rep, row0 = tile * 32, row1 = row0 + 31 < R ? row0 + 31 : R - 1;
  const int c = row0 + mlane, t = c / a.rep, head = g * a.rep + c - t * a.rep;
  const int p = c < R ? attn_position(t, off, n) : -1;
  u32x4 qf[D / 16];
  load_row<D>(a.q, b, t, head, c < R, half, qf);
  const int q0 = off + row0 / a.rep > 0 ? off + row0 / a.rep : 0, q1 = off + row1 / a.rep < n ? off + row1 / a.rep : n - 1;
  KeyTiles kts{0, 0, 0};
  if (q0 <= q1) kts = key_tiles(a, q0, q1, kSplitKeys);

  const TileReads<D> rd(lane);
  TileCopy<D, kSplitKeys, 1> kc, vc;
  kc.set(a.k.t, 0, lane);
  vc.set(a.v.t, 0, lane);
  const uint16_t *kp = a.k.p + b * a.k.b + g * a.k.h, *vp = a.v.p + b * a.v.b + g * a.v.h;
  uint8_t *mine = smem + wave * 4 * kTileBytes;
  RowState<D> st;
  st.init();
  wait_vmem();
  const int step = splits * kSplitWaves, first = split * kSplitWaves + wave;
  auto issue = [&](int i, int slot) {
    const int key0 = kts.key0(i, kSplitKeys);
    uint8_t *to = mine + slot * 2 * kTileBytes;
    kc.issue(kp + key0 * a.k.t, a.k.t, n - key0, to, 0);
    vc.issue(vp + key0 * a.v.t, a.v.t, n - key0, to + kTileBytes, 0);
  };
  if (first < kts.count) issue(first, 0);
  int slot = 0;
  for (int i = first; i < kts.count; i += step, slot ^= 1) {
    // this wave's reads of the other slot are done, then its next tile may land there
    if (i + step < kts.count) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      issue(i + step, slot ^ 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * TileCopy<D, kSplitKeys, 1>::kN) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    const int key0 = kts.key0(i, kSplitKeys), key1 = key0 + kSplitKeys - 1;
    const bool full = key1 <= q0 && (q1 - key0 < a.window || key1 < a.sinks);
    const uint8_t *kt = mine + slot * 2 * kTileBytes;
    attn_tile<D, 1>(a, rd, kt, kt + kTileBytes, qf, key0, p, full, half, st);
  }

  // The waves' states joined: wave w sums output tile w.
  const float lsum = halves_sum(st.l);
  ml_lds[0][wave][lane] = st.m;
  ml_lds[1][wave][lane] = lsum;
  float *join = reinterpret_cast<float *>(smem);
  __syncthreads();  // every wave is done with its ring
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4)
      *reinterpret_cast<f32x4 *>(join + (((wave * kDt + d) * 4 + e4) * 64 + lane) * 4) =
          f32x4{st.o[d][4 * e4], st.o[d][4 * e4 + 1], st.o[d][4 * e4 + 2], st.o[d][4 * e4 + 3]};
  __syncthreads();
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) m = fmaxf(m, ml_lds[0][w][lane]);
  const float from = m == -INFINITY ? 0.f : m;
  f32x16 o = zero16();
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) {
    const float f = __builtin_amdgcn_exp2f((ml_lds[0][w][lane] - from) * a.c);
    l += f * ml_lds[1][w][lane];
    if (wave < kDt) {
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(join + (((w * kDt + wave) * 4 + e4) * 64 + lane) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[4 * e4 + i] += f * v[i];
      }
    }
  }
  const auto final_lse = [&](float mx, float sum, bool some) {
    return some ? (mx * a.c + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f : -INFINITY;
  };
  if (splits == 1) {
    if (wave >= kDt) return;
    const bool some = p >= 0;
    const float inv = 1.f / l;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = some ? o[e] * inv : 0.f;
    u32x4 run[2];
    column_runs(o, run);
    if (c < R) {
      uint16_t *row = out.o + (((int64_t)b * a.T + t) * a.H + head) * D + 32 * wave + 8 * half;
      st16(row, run[0]);
      st16(row + 16, run[1]);
      if (out.lse && wave == 0 && half == 0) out.lse[((int64_t)b * a.H + head) * a.T + t] = final_lse(m, l, some);
    }
    return;
  }
  // This part out to memory (rows that exist); the last part to arrive joins them all, in their order.
  const rsrc_t pr = make_rsrc(partial + (size_t)work * splits * kPartFloats<D>, (int64_t)splits * kPartFloats<D> * 4);
  const auto at = [](int s) { return (uint32_t)(s * kPartFloats<D>) * 4u; };
  if (c < R && wave < kDt) {
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4)
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{__float_as_uint(o[4 * e4]), __float_as_uint(o[4 * e4 + 1]), __float_as_uint(o[4 * e4 + 2]),
                __float_as_uint(o[4 * e4 + 3])},
          pr, at(split) + (uint32_t)(mlane * D + 32 * wave + 8 * e4 + 4 * half) * 4u, 0, 16);
    if (wave == 0 && half == 0) {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), pr, at(split) + (uint32_t)(32 * D + mlane) * 4u, 0, 16);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(l), pr, at(split) + (uint32_t)(32 * D + 32 + mlane) * 4u, 0,
                                            16);
    }
  }
  wait_vmem();
  __syncthreads();
  uint32_t *counter = tile_counter(counters, work);
  if (tid == 0) last_lds = add_dev_u32(counter, 1u) == (uint32_t)(splits - 1) ? 1u : 0u;
  __syncthreads();
  if (!last_lds) return;
  if (tid == 0) st_dev_u32(counter, 0u);  // left as it was found
  // factors exp2((m_s - max m) c) of every part and row into LDS, the sums' total and the maximum beside them
  const int rows = R - row0 < 32 ? R - row0 : 32;
  float *fac = join, *part_l = join + kMaxSplits * 32, *tot = part_l + kMaxSplits * 32;  // [splits][32]; 1 / l (0: nothing seen)
#pragma unroll 4
  for (int i = tid; i < 32 * splits; i += 64 * kSplitWaves) {
    const uint32_t from = at(i >> 5) + (uint32_t)(32 * D + (i & 31)) * 4u;
    const bool row = (i & 31) < rows;
    const uint32_t mi = bld32_dev(pr, row ? from : kOOB), li = bld32_dev(pr, row ? from + 32 * 4 : kOOB);
    fac[i] = __uint_as_float(mi);
    part_l[i] = __uint_as_float(li);
  }
  __syncthreads();
  if (tid < rows) {
    float mx = -INFINITY, sum = 0.f;
    for (int s = 0; s < splits; ++s) mx = fmaxf(mx, fac[32 * s + tid]);
    const float base = mx == -INFINITY ? 0.f : mx;
    for (int s = 0; s < splits; ++s) {
      const float f = __builtin_amdgcn_exp2f((fac[32 * s + tid] - base) * a.c);
      sum += f * part_l[32 * s + tid];
      fac[32 * s + tid] = f;
    }
    const bool some = p >= 0;  // (tid < 32: this thread's own row)
    tot[tid] = some ? 1.f / sum : 0.f;
    if (out.lse) out.lse[((int64_t)b * a.H + head) * a.T + t] = final_lse(mx, sum, some);
  }
  __syncthreads();
  // 4 values of a row per thread and turn
  for (int i = tid; i < rows * (D / 4); i += 64 * kSplitWaves) {
    const int r = i / (D / 4), d4 = i % (D / 4);
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      const u32x4 v = bld16_dev(pr, at(s) + (uint32_t)(r * D + 4 * d4) * 4u);
      const float f = fac[32 * s + r];
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += f * __uint_as_float(v[k]);
    }
    const float inv = tot[r];
    u32x2 w = {0u, 0u};
    if (inv != 0.f) w = u32x2{pack_bf16x2(sum[0] * inv, sum[1] * inv), pack_bf16x2(sum[2] * inv, sum[3] * inv)};
    const int cc = row0 + r, tt = cc / a.rep, hh = g * a.rep + cc - tt * a.rep;
    *reinterpret_cast<u32x2 *>(out.o + (((int64_t)b * a.T + tt) * a.H + hh) * D + 4 * d4) = w;
  }
}

// Which kernel, and how many splits, by estimated time in us (steps and overheads measured at 1 x 5 heads x 1501, 3 x 16
// over 8 heads x 132 behind 1003, 24 x 1 and 1 x 1 tokens, D = 128):
//   tiles of 128 rows   8 us and 0.75 us per key tile where a unit has one workgroup, 0.43 us a workgroup where it has more
//   tiles of 32 rows    rounds of one workgroup a unit (two of D = 64), each 6 us (9 where parts are joined) and 2 us per key
//                       tile of a wave
AttnPlan attn_plan(int64_t B, int64_t T, int64_t S, int H, int G, int D, int window, int sinks) {
  AttnPlan p{};
  const int64_t R = T * (H / G), cus = device_cu_count(current_device());
  p.tiles = (int)((R + kFwdRows - 1) / kFwdRows);
  const auto key_tiles_of = [&](int64_t rows) {  // at most, of so many rows
    const int64_t span = (rows - 1) / (H / G) + 1;
    return (std::min<int64_t>(S, (int64_t)window + span + sinks + 2 * kSplitKeys) + kSplitKeys - 1) / kSplitKeys;
  };
  const int64_t row_tiles = (R + 31) / 32, work = B * G * row_tiles, nt = key_tiles_of(32), slots = D == 64 ? 2 * cus : cus;
  const int64_t most = work > kMaxTileCounters ? 1 : std::min<int64_t>(kMaxSplits, (nt + kSplitWaves - 1) / kSplitWaves);
  int64_t splits = 1;
  double cost = 0;
  for (int64_t s = 1; s <= most; ++s) {
    const double c = (double)((work * s + slots - 1) / slots) * ((s > 1 ? 9 : 6) + 2.0 * ((nt + kSplitWaves * s - 1) / (kSplitWaves * s)));
    if (s == 1 || c < cost) {
      cost = c;
      splits = s;
    }
  }
  if (R > 32 && 8 + key_tiles_of(kFwdRows) * std::max(0.75, 0.43 * (B * G * p.tiles) / cus) <= cost) return p;
  p.row_tiles = (int)row_tiles;
  p.splits = (int)splits;
  if (p.splits > 1) p.partial_floats = (size_t)work * p.splits * (D == 128 ? kPartFloats<128> : kPartFloats<64>);
  return p;
}

template <int D>
static hipError_t launch_split(const AttnArgs &a, const AttnOut &out, const AttnPlan &p, float *partial,
                               uint32_t *counters, hipStream_t st) {
  constexpr int lds = kSplitWaves * 4 * kSplitKeys * kRowBytes<D>;
  static DeviceOnce once;
  const hipError_t e = once.run(current_device(), [] {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(k_attn_split<D>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  });
  if (e != hipSuccess) return e;
  k_attn_split<D><<<dim3((unsigned)(a.B * a.G * p.row_tiles * p.splits)), 64 * kSplitWaves, lds, st>>>(
      a, out, p.row_tiles, p.splits, partial, counters);
  return hipGetLastError();
}

hipError_t launch_attn_fwd(const AttnArgs &a, int D, uint16_t *o, float *lse, float *partial, uint32_t *counters,
                           hipStream_t st) {
  const AttnPlan p = attn_plan(a.B, a.T, a.S, a.H, a.G, D, a.window, a.sinks);
  const AttnOut out{o, lse};
  if (p.row_tiles)
    return D == 128 ? launch_split<128>(a, out, p, partial, counters, st)
                    : launch_split<64>(a, out, p, partial, counters, st);
  const dim3 grid((unsigned)(a.B * a.G * p.tiles));
  if (D == 128)
    k_attn_fwd<128><<<grid, kFwdThreads, 0, st>>>(a, out, p.tiles);
  else
    k_attn_fwd<64><<<grid, kFwdThreads, 0, st>>>(a, out, p.tiles);
  return hipGetLastError();
}

}  // namespace qlora
