// Attention with a sliding window and sinks, backward (see attention.h).
//
// With P = softmax's weights from the saved logarithms, delta = rowsum(dO * O):
//     dS = scale P * (dO V^T - delta),  dQ = dS K,  dK = dS^T Q,  dV = P^T dO.
// Two kernels, neither with atomics, so that the sums have one order:
//
// k_attn_dq: 128 packed rows per workgroup, key tiles streamed as in the
// forward. delta from the bf16 O is off by O's rounding, which would be the
// largest error after the results' own; a row's sum of P (dO V^T - delta),
// which is 0 with the exact delta, says by how much, and the other kernel gets
// the corrected one (dQ too where rows see few keys, kFewKeys). dS enters dQ's product as two bf16 terms (the matrix unit
// has room beside the LDS reads): without them dQ's error was 1.55 times that
// of one rounding, with them 1.15 times; dK's is 1.43 times.
// 2 x 4096 tokens, 40 over 8 heads, window 1024: 308 to 317 us, the matrix unit busy half of the cycles, as in the large
// products over the base.
//
// k_attn_dkv: 128 keys of one key head per workgroup, 32 per wave, which holds
// their K and V rows and both sums in registers (one wave per SIMD); the rows of
// all the heads that share the keys, 32 at a time, go from memory straight into
// LDS, eight tiles in a ring. As in the forward the vector work of a tile stands
// between the matrix work of its neighbours: a step forms the scores and dO V^T
// of tile i + 1 and adds tile i - 1 to the sums. A row's logarithm and delta
// enter those products as one more K slice, each as three bf16 terms (24 bits)
// against ones: they arrive with the tile as 32 bytes a row that k_attn_dq left,
// and cost a matrix instruction instead of LDS reads by every lane.
// A step's 34 products (1088 cycles) and its 32 KB of LDS reads a wave (1024 cycles a CU) bound it together: 2 x 4096
// tokens, 40 over 8 heads, window 1024, 448 us; of an earlier form that took 454, without its copies 375, without LDS reads
// 410, without the sinks' shares 420, the products alone about 280. Of a wave's time 57 % are an instruction's of its own,
// 23 % it waits for its turn or a busy unit, 20 % for data.
// The rows that only see the sinks would make the first key tile's list many
// times as long as the others': they are shared out to workgroups of their own,
// whose float32 sums k_attn_sinks adds, in order, to the first tiles'.
#include "attention.h"
#include "kernels.h"

namespace qlora {

constexpr int kBwdThreads = 256, kBwdRows = 128, kBwdKeys = 128;
// Rows that see at most so many keys (and those that share a wave with one) have their delta corrected before dQ. The error
// that is left otherwise falls with the root of their number (dQ's error over that of one rounding: 2.5 with 2 keys, 1.7
// with 10, 1.3 with 64; corrected 1.0). Time, with the pass and without: 2 x 2048 tokens, 40 over 8 heads, window 16, where
// every row sees few, 111 and 95 us (reads from memory of tiles that are on their way into LDS as well); 8 x 512 tokens
// without a window 167 and 166.
constexpr int kFewKeys = 64;

struct AttnGrad {
  AttnRows o, dO;
  const float *lse;
  u32x4 *stats;            // [B, G, T rep][2]: -lse / scale and -delta as three bf16 terms each, then zeros
  uint16_t *dq, *dk, *dv;  // dense
};

// x as three bf16 terms and zeros: the K slice that adds it to a product with {1, 1, 1, 0, ...}.
__device__ __forceinline__ u32x4 three_terms(float x) {
  const uint32_t a = pack_bf16x2(x, 0.f);
  float rest = x - bf16_lo_to_f32(a);
  const uint32_t b = pack_bf16x2(rest, 0.f);
  rest -= bf16_lo_to_f32(b);
  return u32x4{(a & 0xffffu) | (b << 16), pack_bf16x2(rest, 0.f), 0u, 0u};
}

template <int D>
__device__ __forceinline__ void load_frags(const uint16_t *p, bool ok, int half, u32x4 (&f)[D / 16]) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) f[i] = ok ? ld16(p + 16 * i + 8 * half) : u32x4{0u, 0u, 0u, 0u};
}

template <int D>
__global__ __launch_bounds__(kBwdThreads, 2) void k_attn_dq(AttnArgs a, AttnGrad gr, int tiles) {
  constexpr int kKeys = 32, kTileBytes = kKeys * kRowBytes<D>, kSlots = 4, kRows = 2 * (D / 16), kDt = D / 32, kCols = 2 * kDt;
  constexpr int kAhead = 4;  // fragments read ahead of the products
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * kSlots * kTileBytes];  // keys, then values
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, ml = lane & 31;
  int bg, tile;
  attn_work(blockIdx.x, a.B * a.G, tiles, bg, tile);
  const int b = bg / a.G, g = bg - b * a.G;
  int n, off;
  attn_sequence(a, b, n, off);
  const int R = a.T * a.rep;
  const int wg0 = tile * kBwdRows, row0 = wg0 + 32 * wave;
  const int wg1 = wg0 + kBwdRows < R ? wg0 + kBwdRows - 1 : R - 1, row1 = row0 + 31 < R ? row0 + 31 : R - 1;
  const int c = row0 + ml, t = c / a.rep, head = g * a.rep + c - t * a.rep;
  const bool in = c < R;
  const int p = in ? attn_position(t, off, n) : -1;

  const int p0 = off + wg0 / a.rep > 0 ? off + wg0 / a.rep : 0, p1 = off + wg1 / a.rep < n ? off + wg1 / a.rep : n - 1;
  KeyTiles kts{0, 0, 0};
  if (p0 <= p1) kts = key_tiles(a, p0, p1, kKeys);
  const int count = kts.count;
  const int q0 = off + row0 / a.rep > 0 ? off + row0 / a.rep : 0, q1 = off + row1 / a.rep < n ? off + row1 / a.rep : n - 1;
  const TileReads<D> rd(lane);
  constexpr int kN = TileCopy<D, kKeys, 4>::kN;  // copies of a wave per tile of keys, and of values
  TileStream<D, kKeys, 4> ks, vs;
  const uint32_t kto = lds_addr(ring) + 1024u * (uint32_t)(wave * kN), vto = kto + kSlots * kTileBytes;
  if (count > 0) {
    ks.set(a.k.p + b * a.k.b + g * a.k.h, a.k.t, kts, n, wave, lane);
    vs.set(a.v.p + b * a.v.b + g * a.v.h, a.v.t, kts, n, wave, lane);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      ks.issue(kto + i * kTileBytes, true);
      vs.issue(vto + i * kTileBytes, true);
    }
  }
  // (behind the copies: one trip to memory for both)
  u32x4 qf[D / 16], gf[D / 16];
  load_frags<D>(a.q.p + b * a.q.b + t * a.q.t + head * a.q.h, in, half, qf);
  load_frags<D>(gr.dO.p + b * gr.dO.b + t * gr.dO.t + head * gr.dO.h, in, half, gf);
  float delta = 0.f;
  {
    u32x4 of[D / 16];
    load_frags<D>(gr.o.p + b * gr.o.b + t * gr.o.t + head * gr.o.h, in, half, of);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        delta += bf16_lo_to_f32(of[i][w]) * bf16_lo_to_f32(gf[i][w]) + bf16_hi_to_f32(of[i][w]) * bf16_hi_to_f32(gf[i][w]);
  }
  delta = halves_sum(delta);
  const int64_t at = ((int64_t)b * a.H + head) * a.T + t;
  float rest = 0.f;  // this half's sum of P (dO V^T - delta)
  const float lse = p >= 0 ? gr.lse[at] : 0.f, lse2 = lse * 1.4426950408889634f;
  // Of few keys that sum is no small part of dS: where the wave's first row sees few (a row at position p sees
  // min(p + 1, window + sinks)), it is formed in a pass over the wave's own tiles, and corrects delta for dQ too.
  if (q0 <= q1 && (q0 + 1 < a.window + a.sinks ? q0 + 1 : a.window + a.sinks) <= kFewKeys) {
    const KeyTiles own = key_tiles(a, q0, q1, kKeys);
    for (int i = 0; i < own.count; ++i) {
      const int key0 = own.key0(i, kKeys), key = key0 + ml;
      u32x4 f[D / 16];
      f32x16 s = zero16(), dp = zero16();
      load_frags<D>(a.k.p + b * a.k.b + g * a.k.h + (int64_t)key * a.k.t, key < n, half, f);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) s = mfma32(f[k], qf[k], s);
      load_frags<D>(a.v.p + b * a.v.b + g * a.v.h + (int64_t)key * a.v.t, key < n, half, f);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) dp = mfma32(f[k], gf[k], dp);
      attn_mask(a, p, key0, half, s);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        rest += s[e] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(fmaf(s[e], a.c, -lse2)) * (dp[e] - delta);
    }
    delta += halves_sum(rest);
    rest = 0.f;
  }
  f32x16 dq[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) dq[d] = zero16();
  wait_vmem();  // from here on only the copies count
  if (count > 0) {
    // Tile i lies in slot i % 4. A step forms the scores and dO V^T of its tile, then dS, then dQ's products; its barrier
    // stands before the last: tile i + 1 has come in (the next step's first fragments are read beside those products),
    // and tile i + 3 is issued over i - 1, which every wave has finished.
    wait_barrier<0>();
    RingReads<D> rr;
    rr.set_rows(ring, rd, half);
    rr.set_cols(ring, rd);
    u32x4 rf[kAhead], cf[kAhead];
    auto load_row = [&](int slot, int r) {  // slice r / 2 of the keys (r even) or values
      rf[r % kAhead] = rr.rows(((r & 1) * kSlots + slot) * kTileBytes, r >> 1);
    };
    auto load_col = [&](int slot, int j) { cf[j % kAhead] = rr.cols(slot * kTileBytes, j / kDt, j % kDt); };
#pragma unroll
    for (int r = 0; r < kAhead; ++r) load_row(0, r);
    int key0 = kts.key0(0, kKeys);
    const int gap = (kts.w0 - kts.ns + 1) * kKeys;
    auto step = [&](int i, const int S) {
      f32x16 s, dp;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r & 1)
          dp = mfma32(rf[r % kAhead], gf[r >> 1], r > 1 ? dp : zero16());
        else
          s = mfma32(rf[r % kAhead], qf[r >> 1], r > 1 ? s : zero16());
        QLORA_SCHED_FENCE();
        if (r + kAhead < kRows)
          load_row(S, r + kAhead);
        else
          load_col(S, r + kAhead - kRows);
        QLORA_SCHED_FENCE();
      }
      const int key1 = key0 + kKeys - 1;
      if (!(key1 <= q0 && (q1 - key0 < a.window || key1 < a.sinks))) {
        attn_mask(a, p, key0, half, s);
#pragma unroll
        for (int e = 0; e < 16; ++e) dp[e] = s[e] == -INFINITY ? 0.f : dp[e];  // (dO V^T may be anything there)
      }
      // (the list is taken to an even length: nobody sees the tile behind it)
      key0 = i + 1 < count ? key0 + (i + 1 == kts.ns ? gap : kKeys) : 1 << 29;
      u32x4 hi[2], lo[2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], a.c, -lse2)) * (dp[e] - delta);
        rest += s[e];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        hi[k] = pack_frag(s, k);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          s[8 * k + 2 * w] -= bf16_lo_to_f32(hi[k][w]);
          s[8 * k + 2 * w + 1] -= bf16_hi_to_f32(hi[k][w]);
        }
        lo[k] = pack_frag(s, k);
      }
      wait_barrier<2 * kN>();
      ks.issue(kto + ((S + 3) & 3) * kTileBytes, true);
      vs.issue(vto + ((S + 3) & 3) * kTileBytes, true);
#pragma unroll
      for (int j = 0; j < kCols; j += 2) {  // (two sums in turn)
#pragma unroll
        for (int u = 0; u < 2; ++u) dq[(j + u) % kDt] = mfma32(cf[(j + u) % kAhead], hi[j / kDt], dq[(j + u) % kDt]);
#pragma unroll
        for (int u = 0; u < 2; ++u) dq[(j + u) % kDt] = mfma32(cf[(j + u) % kAhead], lo[j / kDt], dq[(j + u) % kDt]);
        QLORA_SCHED_FENCE();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (j + u + kAhead < kCols)
            load_col(S, j + u + kAhead);
          else
            load_row((S + 1) & 3, j + u + kAhead - kCols);
        }
        QLORA_SCHED_FENCE();
      }
    };
    for (int i = 0;; i += 4) {
      step(i, 0);
      step(i + 1, 1);
      if (i + 2 >= count) break;
      step(i + 2, 2);
      step(i + 3, 3);
      if (i + 4 >= count) break;
    }
    wait_barrier<0>();
  }
  rest = halves_sum(rest);
  if (in)
    gr.stats[(((int64_t)bg * R + c) << 1) + half] =
        p >= 0 ? three_terms(half ? -(delta + rest) : -lse / a.scale) : u32x4{0u, 0u, 0u, 0u};
  uint16_t *row = gr.dq + (((int64_t)b * a.T + t) * a.H + head) * D;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
#pragma unroll
    for (int e = 0; e < 16; ++e) dq[d][e] = p >= 0 ? dq[d][e] * a.scale : 0.f;
    u32x4 run[2];
    column_runs(dq[d], run);
    if (in) {
      st16(row + 32 * d + 8 * half, run[0]);
      st16(row + 32 * d + 16 + 8 * half, run[1]);
    }
  }
}

// Work of k_attn_dkv: per (sequence, key head) and sink tile `far` workgroups each take a share of the rows past its
// window; those behind them take the key tiles with the rows of their windows. (The shares are short and come first:
// the last workgroups to start are then not the ones that end last.) Partials of the former, and of the sink tiles
// among the latter, are [far + 1][2 (dK, dV)][wave][D / 32][4][64 lanes] float4 per sink tile; a wave without sinks
// among its 32 keys has only those of its window.
struct DkvPlan {
  int tiles, sink_tiles, far, far_rows;
  float *partial;
};
template <int D>
constexpr int kSinkFloats = 2 * kBwdKeys * D;

// Tokens t0 .. t1 (none where t1 < t0) that a workgroup takes: those whose window reaches the tile, at positions key0
// .. key0 + 127 + window - 1 of the sequence (share -1; all from key0 on for sinks that are not shared out), or of those
// past them, which see its sinks alone, a share.
__device__ __forceinline__ void row_share(const AttnArgs &a, const DkvPlan &pl, int key0, int n, int off, int share,
                                          int &t0, int &t1) {
  const int first = key0 - off > 0 ? key0 - off : 0;
  const int last = n - 1 - off < a.T - 1 ? n - 1 - off : a.T - 1;  // the last token that sees anything
  const int end = key0 + kBwdKeys - 1 - off;                      // of the tile's last key
  const int wend = end < last - a.window + 1 && (pl.far > 0 || key0 >= a.sinks) ? end + a.window - 1 : last;
  t0 = first;
  t1 = wend;
  if (share >= 0) {
    t0 = (wend + 1 > first ? wend + 1 : first) + share * pl.far_rows;
    t1 = t0 + pl.far_rows - 1 < last ? t0 + pl.far_rows - 1 : last;
  }
  if (key0 >= n) t1 = t0 - 1;
}

// The block of 32 tokens that a list of `blocks` begins with. Workgroups of neighbouring key tiles run at the same time and
// read overlapping lists; each from its own first row, their reads of a row lie further apart than the L2 cache reaches.
// They read it together where block x (counted over the sequence, xf the list's first) comes at the time x mod the
// length of a window's list; with no window, where the 32 tiles that share an XCD begin with the last tile's first block.
// (2 x 4096 tokens: 1.49 GB fetched from memory without, 0.38 with; 466 -> 454 us.)
__device__ __forceinline__ int first_block(const AttnArgs &a, int tile, int blocks) {
  const int xf = tile * (kBwdKeys / 32);
  const int span = (a.window + kBwdKeys - 1 + 31) / 32, at = (span - xf % span) % span;
  if (at < blocks) return at;
  const int group = ((tile | 31) - tile) * (kBwdKeys / 32);
  return group < blocks ? group : 0;
}

template <int D>
__device__ __forceinline__ void store_keys(const AttnArgs &a, const AttnGrad &gr, int b, int g, int key, int half,
                                           f32x16 (&dk)[D / 32], f32x16 (&dv)[D / 32]) {
  const int64_t at = (((int64_t)b * a.S + key) * a.G + g) * D;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
#pragma unroll
    for (int e = 0; e < 16; ++e) dk[d][e] *= a.scale;
    u32x4 rk[2], rv[2];
    column_runs(dk[d], rk);
    column_runs(dv[d], rv);
    if (key < a.S)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        st16(gr.dk + at + 32 * d + 16 * r + 8 * half, rk[r]);
        st16(gr.dv + at + 32 * d + 16 * r + 8 * half, rv[r]);
      }
  }
}

// The row tiles of tokens t0 .. t1: blocks of 32 tokens, each once per head of the group; a tile is 32 rows of Q and of
// dO and their statistics. A lane's offsets never change and a tile's addresses move by two constants (with tiles of 32
// consecutive packed rows every lane had to follow its rows' tokens and heads). The blocks come in a cycle from `start`
// on (see first_block); past the last tile that one comes again.
template <int D>
struct RowStream {
  typedef TileCopy<D, 32, 4> Copy;
  static constexpr int kN = Copy::kN;
  Copy cq, cg;
  int row[kN];  // of the tile
  uint32_t vs;
  uint64_t q, g, st, qh, gh, qw, gw, sw;  // the next tile's addresses; to the next head; to the next block's first
  uint64_t qc, gc, sc;                    // from the last block to the first
  int rep, head, left, tokens, blocks;    // the next tile's head; tiles behind it; tokens from its block on; all blocks
  __device__ __forceinline__ void set(const AttnArgs &a, const AttnGrad &gr, int b, int grp, int t0, int t1, int start,
                                      int wave, int lane) {
    rep = a.rep;
    cq.set(a.q.t, wave, lane);
    cg.set(gr.dO.t, wave, lane);
#pragma unroll
    for (int i = 0; i < kN; ++i) row[i] = (wave * kN + i) * Copy::kRowsPer + lane / Copy::kChunks;
    vs = (uint32_t)(lane >> 1) * (uint32_t)rep * 32u + (uint32_t)(lane & 1) * 16u;
    q = (uint64_t)(uintptr_t)(a.q.p + b * a.q.b + (int64_t)grp * rep * a.q.h + t0 * a.q.t);
    g = (uint64_t)(uintptr_t)(gr.dO.p + b * gr.dO.b + (int64_t)grp * rep * gr.dO.h + t0 * gr.dO.t);
    st = (uint64_t)(uintptr_t)(gr.stats + ((((int64_t)b * a.G + grp) * a.T + t0) * rep << 1));
    qh = (uint64_t)(2 * a.q.h);
    gh = (uint64_t)(2 * gr.dO.h);
    qw = (uint64_t)(2 * (32 * a.q.t - (rep - 1) * a.q.h));
    gw = (uint64_t)(2 * (32 * gr.dO.t - (rep - 1) * gr.dO.h));
    sw = (uint64_t)(32 * (31 * rep + 1));
    head = 0;
    tokens = t1 - t0 + 1;
    blocks = (tokens + 31) / 32;
    left = blocks * rep - 1;
    qc = qw - (uint64_t)(64 * blocks * a.q.t);
    gc = gw - (uint64_t)(64 * blocks * gr.dO.t);
    sc = sw - (uint64_t)(1024 * (int64_t)blocks * rep);
    q += (uint64_t)(64 * start * a.q.t);
    g += (uint64_t)(64 * start * gr.dO.t);
    st += (uint64_t)(1024 * (int64_t)start * rep);
    tokens -= 32 * start;
  }
  // qto, gto: LDS addresses of the wave's parts of the tile; sto: of its statistics (every wave copies them all)
  __device__ __forceinline__ void issue(uint32_t qto, uint32_t gto, uint32_t sto) {
    const i32x4 qs{(int)(uint32_t)q, (int)(uint32_t)(q >> 32), 0x7fffffff, 0x00020000};
    const i32x4 gs{(int)(uint32_t)g, (int)(uint32_t)(g >> 32), 0x7fffffff, 0x00020000};
    const int valid = tokens < 32 ? tokens : 32;
    const i32x4 ss{(int)(uint32_t)st, (int)(uint32_t)(st >> 32), ((valid - 1) * rep + 1) * 32, 0x00020000};
    if (valid == 32) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        dma16_asm(qs, qto + 1024u * i, cq.voff[i], 0u);
        dma16_asm(gs, gto + 1024u * i, cg.voff[i], 0u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {  // rows past the list read zeros
        dma16_asm(qs, qto + 1024u * i, row[i] < valid ? cq.voff[i] : kOOB, 0u);
        dma16_asm(gs, gto + 1024u * i, row[i] < valid ? cg.voff[i] : kOOB, 0u);
      }
    }
    dma16_asm(ss, sto, vs, 0u);
    if (left == 0) return;
    --left;
    ++head;
    if (head < rep) {
      q += qh;
      g += gh;
      st += 32;
      return;
    }
    head = 0;
    const bool cycle = tokens <= 32;
    tokens += cycle ? 32 * blocks - 32 : -32;
    q += cycle ? qc : qw;
    g += cycle ? gc : gw;
    st += cycle ? sc : sw;
  }
};

// The vector work of a tile of 32 rows in 16 pieces: weights exp2(c s), rounded for their product; dS = weight times
// (dO V^T - delta), rounded.
struct GradPieces {
  uint32_t seen;  // bit 8 (e / 4) + e % 4: whether the lane's row of accumulator e sees its key
  __device__ __forceinline__ void run(int k, f32x16 &s, f32x16 &dp, float c, u32x4 (&pf)[2], u32x4 (&df)[2]) {
    const int e = 2 * (k >> 1);
    if ((k & 1) == 0) {
      // (two scores a piece: pieces 0, 2, .. form weights 0 .. 15 in pairs)
#pragma unroll
      for (int u = e; u < e + 2; ++u) {
        const int keep = __builtin_amdgcn_sbfe((int)seen, 8 * (u >> 2) + (u & 3), 1);
        s[u] = __int_as_float(__float_as_int(__builtin_amdgcn_exp2f(s[u] * c)) & keep);
        dp[u] = __int_as_float(__float_as_int(dp[u]) & keep);
      }
      uint32_t x = pack_bf16x2(s[e], s[e + 1]);
      pin(x);
      pf[k >> 3][(k >> 1) & 3] = x;
    } else {
      uint32_t x = pack_bf16x2(s[e] * dp[e], s[e + 1] * dp[e + 1]);
      pin(x);
      df[k >> 3][(k >> 1) & 3] = x;
    }
  }
};

template <int D>
__global__ __launch_bounds__(kBwdThreads, 1) void k_attn_dkv(AttnArgs a, AttnGrad gr, DkvPlan pl) {
  constexpr int kTileBytes = 32 * kRowBytes<D>, kSlots = 8, kQk = D / 16, kDt = D / 32;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // [kSlots] Q, [kSlots] dO, [kSlots][32 rows][2] statistics
  uint8_t *const qring = smem, *const gring = smem + kSlots * kTileBytes, *const sring = smem + 2 * kSlots * kTileBytes;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, ml = lane & 31;
  const int heads = a.B * a.G, far = heads * pl.sink_tiles * pl.far;
  int bg, tile, share = -1;
  if ((int)blockIdx.x >= far) {
    // (counted down again: with no window the first keys are seen by the most rows)
    attn_work(blockIdx.x - far, heads, pl.tiles, bg, tile);
    tile = pl.tiles - 1 - tile;
  } else {
    const int j = blockIdx.x;
    share = j % pl.far;
    bg = j / pl.far / pl.sink_tiles;
    tile = j / pl.far % pl.sink_tiles;
  }
  const int b = bg / a.G, g = bg - b * a.G;
  int n, off;
  attn_sequence(a, b, n, off);
  const int key0 = tile * kBwdKeys;
  int t0, t1;
  row_share(a, pl, key0, n, off, share, t0, t1);
  const int tokens = t1 >= t0 ? t1 - t0 + 1 : 0, count = (tokens + 31) / 32 * a.rep;
  if (share >= 0 && count == 0) return;  // (k_attn_sinks knows)

  const int kw0 = key0 + 32 * wave, key = kw0 + ml;
  const bool kin = key < n;
  f32x16 dk[kDt], dv[kDt];
#pragma unroll
  for (int d = 0; d < kDt; ++d) {
    dk[d] = zero16();
    dv[d] = zero16();
  }
  if (count > 0) {
    u32x4 kf[kQk], vf[kQk];
    load_frags<D>(a.k.p + b * a.k.b + g * a.k.h + (int64_t)key * a.k.t, kin, half, kf);
    load_frags<D>(a.v.p + b * a.v.b + g * a.v.h + (int64_t)key * a.v.t, kin, half, vf);
    const TileReads<D> rd(lane);
    RowStream<D> rs;
    const int blocks = (tokens + 31) / 32, start = share < 0 ? first_block(a, tile, blocks) : 0;
    rs.set(a, gr, b, g, t0, t1, start, wave, lane);
    constexpr int kCopies = 2 * RowStream<D>::kN + 1;  // of a wave per tile
    const uint32_t qto = lds_addr(qring) + 1024u * (uint32_t)(wave * RowStream<D>::kN), gto = qto + kSlots * kTileBytes;
    const uint32_t sto = lds_addr(sring);
    wait_vmem();  // K and V are in: from here on only the copies count
    // Tile i lies in slot i % 8. Step i, behind a barrier, issues tile i + 5; those up to i + 2 have come in, which is as
    // far as the reads go until the next barrier. Tile "-1" is zeros.
#pragma unroll
    for (int i = 0; i < 5; ++i) rs.issue(qto + i * kTileBytes, gto + i * kTileBytes, sto + i * 1024);
    for (int i = tid; i < kTileBytes / 16; i += kBwdThreads) {
      st16(qring + 7 * kTileBytes + 16 * i, u32x4{0u, 0u, 0u, 0u});
      st16(gring + 7 * kTileBytes + 16 * i, u32x4{0u, 0u, 0u, 0u});
    }
    wait_barrier<2 * kCopies>();
    RingReads<D> qr, dr;
    qr.set_rows(qring, rd, half);
    qr.set_cols(qring, rd);
    dr.set_rows(gring, rd, half);
    dr.set_cols(gring, rd);
    uint32_t sat = sto + 32u * ml;
    pin(sat);
    const u32x4 ones = half ? u32x4{0u, 0u, 0u, 0u} : u32x4{0x3f803f80u, 0x00003f80u, 0u, 0u};
    auto stat = [&](int slot, int k) {
      typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
      return *(lds_u32x4 *)((__attribute__((address_space(3))) const uint8_t *)(uintptr_t)sat + slot * 1024 + 16 * k);
    };
    // A key is seen by the list's tokens from `lo` to below `hi`: not by those before it, past its window, or past the list.
    const int64_t first = (int64_t)key - off - t0, last = key < a.sinks ? INT32_MAX : first + a.window;
    int lo = (int)(first < 0 ? 0 : first < tokens ? first : tokens), hi = (int)(last < 0 ? 0 : last < tokens ? last : tokens);
    lo -= 32 * start;
    hi -= 32 * start;
    int seen_head = 0, seen_cycle = (blocks - start) * a.rep, seen_left = count;  // tiles to the cycle's, to the list's end
    // The rows of a tile that see the key, as bits; each call is for the tile behind the last one's. Bits and two ANDs an
    // accumulator cost the same for every tile and hide behind the products; a branch around the masks of whole tiles
    // made them wait for the scores (an earlier form of this kernel, 2 x 4096 tokens as above: 750 us without any masks, 800
    // with the branch).
    auto seen_rows = [&] {
      const auto from = [](int x) { return x > 31 ? 0u : 0xffffffffu << (x < 0 ? 0 : x); };
      const uint32_t m = (from(lo) & ~from(hi)) >> (4 * half);
      const bool wrap = ++seen_head == a.rep;  // the next tile begins a block
      seen_head = wrap ? 0 : seen_head;
      int by = wrap ? 32 : 0;
      by = --seen_cycle == 0 ? 32 - 32 * blocks : by;
      hi -= by;
      lo = --seen_left == 0 ? 1 << 30 : lo - by;  // (nobody sees the tile behind the list)
      return m;
    };
    f32x16 s[2], dp[2];  // of tile i in [i & 1]
    u32x4 pf[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}}, df[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    u32x4 fq[2], fg[2], cq[2], cg[2];  // fragments: rows of Q and dO, columns of Q and dO
    // A step has kQk + 1 rounds: slice k of the next tile's scores and dO V^T (slice 0 are the statistics), and in all but
    // the last one product of each sum.
    auto load_next = [&](int slot, int k, int S) {  // slice k of the scores and of dO V^T (an odd number: they take turns)
      fq[(k + S) & 1] = k == 0 ? stat(slot, 0) : qr.rows(slot * kTileBytes, k - 1);
      fg[(k + S) & 1] = k == 0 ? stat(slot, 1) : dr.rows(slot * kTileBytes, k - 1);
    };
    auto load_sum = [&](int slot, int j) {  // j-th products of both sums
      cq[j & 1] = qr.cols(slot * kTileBytes, j / kDt, j % kDt);
      cg[j & 1] = dr.cols(slot * kTileBytes, j / kDt, j % kDt);
    };
    s[0] = zero16();
    dp[0] = zero16();
#pragma unroll
    for (int k = 0; k <= kQk; ++k) {
      s[0] = mfma32(k == 0 ? stat(0, 0) : qr.rows(0, k - 1), k == 0 ? ones : kf[k - 1], s[0]);
      dp[0] = mfma32(k == 0 ? stat(0, 1) : dr.rows(0, k - 1), k == 0 ? ones : vf[k - 1], dp[0]);
    }
    load_next(1, 0, 0);
    load_next(1, 1, 0);
    load_sum(7, 0);
    load_sum(7, 1);
    auto step = [&](const int S) {
      wait_barrier<2 * kCopies>();
      rs.issue(qto + ((S + 5) & 7) * kTileBytes, gto + ((S + 5) & 7) * kTileBytes, sto + ((S + 5) & 7) * 1024);
      const int s1 = (S + 1) & 7, s2 = (S + 2) & 7, sb = (S + 7) & 7;
      f32x16 &sc = s[S & 1], &dc = dp[S & 1], &sn = s[(S + 1) & 1], &dn = dp[(S + 1) & 1];
      u32x4 pn[2], dfn[2];
      GradPieces gp{seen_rows()};
#pragma unroll
      for (int k = 0; k <= kQk; ++k) {
        sn = mfma32(fq[(k + S) & 1], k == 0 ? ones : kf[k - 1], k ? sn : zero16());
        QLORA_SCHED_FENCE();
        if (k < kQk) {
#pragma unroll
          for (int u = 0; u < 8 / kQk; ++u) gp.run(2 * (8 / kQk) * k + 2 * u, sc, dc, a.c, pn, dfn);
        }
        QLORA_SCHED_FENCE();
        if (k < kQk) dv[k % kDt] = mfma32(cg[k & 1], pf[k / kDt], dv[k % kDt]);
        QLORA_SCHED_FENCE();
        if (k < kQk) {
#pragma unroll
          for (int u = 0; u < 8 / kQk; ++u) gp.run(2 * (8 / kQk) * k + 2 * u + 1, sc, dc, a.c, pn, dfn);
        }
        QLORA_SCHED_FENCE();
        dn = mfma32(fg[(k + S) & 1], k == 0 ? ones : vf[k - 1], k ? dn : zero16());
        QLORA_SCHED_FENCE();
        if (k + 2 <= kQk)
          load_next(s1, k + 2, S);
        else
          load_next(s2, k + 1 - kQk, S + 1);
        QLORA_SCHED_FENCE();
        if (k < kQk) dk[k % kDt] = mfma32(cq[k & 1], df[k / kDt], dk[k % kDt]);
        QLORA_SCHED_FENCE();
        if (k < kQk) {
          if (k + 2 < kQk)
            load_sum(sb, k + 2);
          else
            load_sum(S, k + 2 - kQk);
        }
        QLORA_SCHED_FENCE();
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        pf[u] = pn[u];
        df[u] = dfn[u];
      }
    };
    // (the list is taken to an even length: the tile behind it is masked whole)
    const int steps = count + (count & 1);
    if (kw0 >= n || (share >= 0 && kw0 >= a.sinks)) {  // no row of the list sees these keys: the copies alone
      for (int i = 0; i < steps; ++i) {
        wait_barrier<2 * kCopies>();
        const int to = (i + 5) & 7;
        rs.issue(qto + to * kTileBytes, gto + to * kTileBytes, sto + to * 1024);
      }
      wait_barrier<0>();
    } else {
      for (int i = 0;; i += 8) {
        step(0);
        step(1);
        if (i + 2 >= steps) break;
        step(2);
        step(3);
        if (i + 4 >= steps) break;
        step(4);
        step(5);
        if (i + 6 >= steps) break;
        step(6);
        step(7);
        if (i + 8 >= steps) break;
      }
      wait_barrier<0>();
      const int at = ((steps - 1) & 7) * kTileBytes;
#pragma unroll
      for (int j = 0; j < kQk; ++j) {
        dv[j % kDt] = mfma32(dr.cols(at, j / kDt, j % kDt), pf[j / kDt], dv[j % kDt]);
        dk[j % kDt] = mfma32(qr.cols(at, j / kDt, j % kDt), df[j / kDt], dk[j % kDt]);
      }
    }
  }
  if (pl.far > 0 && tile < pl.sink_tiles) {
    if (share >= 0 && kw0 >= a.sinks) return;
    float *to = pl.partial + (((size_t)bg * pl.sink_tiles + tile) * (pl.far + 1) + share + 1) * kSinkFloats<D> +
                wave * 32 * D + lane * 4;
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        *reinterpret_cast<f32x4 *>(to + (d * 4 + e4) * 256) =
            f32x4{dk[d][4 * e4], dk[d][4 * e4 + 1], dk[d][4 * e4 + 2], dk[d][4 * e4 + 3]};
        *reinterpret_cast<f32x4 *>(to + kBwdKeys * D + (d * 4 + e4) * 256) =
            f32x4{dv[d][4 * e4], dv[d][4 * e4 + 1], dv[d][4 * e4 + 2], dv[d][4 * e4 + 3]};
      }
    return;
  }
  store_keys<D>(a, gr, b, g, key, half, dk, dv);
}

// The sink tiles' sums: one workgroup per (sequence, key head, sink tile, 32 keys, 32 columns, dK or dV); its waves take
// the shares in turn and are joined in their order.
template <int D>
__global__ __launch_bounds__(kBwdThreads) void k_attn_sinks(AttnArgs a, AttnGrad gr, DkvPlan pl) {
  __shared__ __attribute__((aligned(16))) float join[4][16 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  int j = blockIdx.x;
  const int which = j & 1, part = (j >> 1) & 3, d = (j >> 3) % (D / 32), bt = (j >> 3) / (D / 32);
  const int bg = bt / pl.sink_tiles, tile = bt - bg * pl.sink_tiles;
  const int b = bg / a.G, g = bg - b * a.G;
  int n, off;
  attn_sequence(a, b, n, off);
  const int kw0 = tile * kBwdKeys + 32 * part, key = kw0 + (lane & 31);
  const float *from = pl.partial + (size_t)bt * (pl.far + 1) * kSinkFloats<D> + which * kBwdKeys * D + part * 32 * D +
                      d * 1024 + lane * 4;
  int shares = 1;  // the window's, then those that have rows
  if (kw0 < a.sinks)
    for (; shares <= pl.far; ++shares) {
      int t0, t1;
      row_share(a, pl, tile * kBwdKeys, n, off, shares - 1, t0, t1);
      if (t1 < t0) break;
    }
  f32x16 sum = zero16();
#pragma unroll 4
  for (int s = wave; s < shares; s += 4)
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const f32x4 x = *reinterpret_cast<const f32x4 *>(from + (size_t)s * kSinkFloats<D> + e4 * 256);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[4 * e4 + i] += x[i];
    }
#pragma unroll
  for (int e = 0; e < 16; ++e) join[wave][e * 64 + lane] = sum[e];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    sum[e] = (join[0][e * 64 + lane] + join[1][e * 64 + lane]) + (join[2][e * 64 + lane] + join[3][e * 64 + lane]);
    if (which == 0) sum[e] *= a.scale;
  }
  u32x4 run[2];
  column_runs(sum, run);
  uint16_t *to = (which ? gr.dv : gr.dk) + (((int64_t)b * a.S + key) * a.G + g) * D + 32 * d + 8 * half;
  if (key < a.S) {
    st16(to, run[0]);
    st16(to + 16, run[1]);
  }
}

// The rows past the sink tiles' windows in about one share per compute unit, of 64 tokens at least (a share's waves
// without sinks idle, and a workgroup has a unit to itself): 2 x 4096 tokens 448 us with them; a list of their own kept
// whole is four times as long as the others'. Where the sink tiles fill half of the units by themselves, or fewer than
// kFarRows rows would be shared out (a step of 32 takes about 1 us, the second kernel 7), their lists stay whole.
constexpr int kFarRows = 512;
static DkvPlan dkv_plan(int64_t B, int64_t T, int64_t S, int rep, int G, int window, int sinks) {
  DkvPlan p{};
  p.tiles = (int)((S + kBwdKeys - 1) / kBwdKeys);
  if (sinks > 0 && S > window) {
    const int sink_tiles = std::min<int>((sinks + kBwdKeys - 1) / kBwdKeys, p.tiles);
    const int64_t most = std::min<int64_t>(device_cu_count(current_device()) / (B * G * sink_tiles), 64);
    // (offsets lie on the device; whatever they are, the tokens past a window are at positions from it to S)
    const int64_t tokens = std::min<int64_t>(T, S - window);
    if (most < 2 || tokens * rep < kFarRows) return p;
    p.sink_tiles = sink_tiles;
    p.far_rows = (int)std::max<int64_t>(64, ((tokens + most - 1) / most + 31) / 32 * 32);  // whole blocks
    p.far = (int)((tokens + p.far_rows - 1) / p.far_rows);
  }
  return p;
}

size_t attn_bwd_workspace_floats(int64_t B, int64_t T, int64_t S, int H, int G, int D, int window, int sinks,
                                 size_t *partial_at) {
  const DkvPlan p = dkv_plan(B, T, S, H / G, G, window, sinks);
  const size_t stats = (size_t)B * H * T * 8;  // 32 bytes a row
  if (partial_at) *partial_at = stats;
  return stats + (p.far ? (size_t)B * G * p.sink_tiles * (p.far + 1) * 2 * kBwdKeys * D : 0);
}

template <int D>
static hipError_t launch_as(const AttnArgs &a, AttnGrad gr, DkvPlan pl, hipStream_t st) {
  const int64_t R = (int64_t)a.T * a.rep;
  const int tiles = (int)((R + kBwdRows - 1) / kBwdRows), heads = a.B * a.G;
  constexpr int lds = 8 * (2 * 32 * kRowBytes<D> + 1024);
  static DeviceOnce once;
  hipError_t e = once.run(current_device(), [] {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(k_attn_dkv<D>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  });
  if (e != hipSuccess) return e;
  k_attn_dq<D><<<dim3((unsigned)(heads * tiles)), kBwdThreads, 0, st>>>(a, gr, tiles);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_attn_dkv<D><<<dim3((unsigned)(heads * (pl.tiles + pl.sink_tiles * pl.far))), kBwdThreads, lds, st>>>(a, gr, pl);
  e = hipGetLastError();
  if (e != hipSuccess || !pl.far) return e;
  k_attn_sinks<D><<<dim3((unsigned)(heads * pl.sink_tiles * 8 * (D / 32))), kBwdThreads, 0, st>>>(a, gr, pl);
  return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnArgs &a, int D, const AttnRows &o, const AttnRows &dO, const float *lse,
                           uint16_t *dq, uint16_t *dk, uint16_t *dv, float *ws, hipStream_t st) {
  size_t at = 0;
  (void)attn_bwd_workspace_floats(a.B, a.T, a.S, a.H, a.G, D, a.window, a.sinks, &at);
  DkvPlan pl = dkv_plan(a.B, a.T, a.S, a.rep, a.G, a.window, a.sinks);
  pl.partial = ws + at;
  const AttnGrad gr{o, dO, lse, reinterpret_cast<u32x4 *>(ws), dq, dk, dv};
  return D == 128 ? launch_as<128>(a, gr, pl, st) : launch_as<64>(a, gr, pl, st);
}

}  // namespace qlora
