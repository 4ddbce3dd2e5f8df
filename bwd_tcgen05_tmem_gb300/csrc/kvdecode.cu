// kvdecode.cu -- attention of a few query tokens over the 4-bit cache.
//
// Per (sequence b, query token i, query head): pos = len_b - seqlen_q + i,
// visible keys j <= pos with (no window, or j >= pos - window_left, or
// j < sinks);  O = softmax(scale q k) v and LSE = ln sum exp.
//
// The work is a stream of codes (d / 2 + d / 16 bytes a token and side), so it
// is bound by HBM if the codes can be turned into matrix operands fast enough:
// an SM's share of the memory rate is about 47 codes a clock.  Hence
//   * products on the tensor cores with the CACHE as the 16-row operand and the
//     query rows as the 8-column one (mma.m16n8k16): a decode step has 1 to 16
//     rows for each kv head, and this side wastes the least;
//   * codes go from shared memory to operand registers without a detour: the
//     cache is laid out (see kvcache.cu) so that a lane's vectors hold exactly
//     the codes of its operand registers.  One mask makes two fp16 numbers of two
//     codes: below fp16's normal range a number's bits are its value in units of
//     2^-24, and the products take such numbers.  Every other code stays four bits
//     up, in units 16 times as large, which saves its shift: q is held divided by
//     16 there, O is multiplied by 16 at the end (head dim 256 differs, see KCodes).
//     K: pairs of one register are dims n, n + 4 of a word of one token.
//     V: they are the same dim of two tokens (one byte permute joins the
//     half-words of both);
//   * the codes' offset of 8: K's enters as the start value of the products,
//     -8 times the sum of q, worked out once for each piece; V's is taken off
//     the codes, exactly, by one packed add.  (As a start value it would have
//     to cancel in O, and the tensor cores' sums do not hold enough bits.)
//   * both products are in fp16, which holds q and the probabilities better
//     than bf16 where the range allows: a bf16 q row is held times a power of
//     two that brings its largest element to 2^13 .. 2^14 (exact, but for
//     elements 2^27 times smaller), and a warp keeps a power of two that brings
//     the largest probability times V scale of its tokens to 2^13 .. 2^15;
//   * scales stay out of the operands: K's multiply the FP32 products of each
//     32-dim group, V's multiply the probabilities before these are rounded.
//
// S^T = K Q^T leaves probabilities with tokens along the operand's rows; the
// second product O^T = V^T P^T wants them along its depth: movmatrix
// transposes 8 x 8 blocks in registers.
//
// Split: every (sequence, kv head, block of 8 or 16 query rows) is an item, its
// tiles of 64 tokens are a stretch of one list, and the list is cut into equal
// runs, one for each warp of a grid that fills the card, so ragged lengths
// balance; an item counts kItemCost tiles more than it has, for what comes once
// for each.  Lengths are read on the device, so a captured graph serves any
// lengths.  Warps wait for nobody but their own copies.  A warp holds a piece's
// running sum and O in registers and writes the result, or, where the item is
// shared with other warps, a partial result that a second kernel joins in the
// order of the runs.
//
// Measured on a GB300 (graph replays, 8 kv heads, 4 query heads each, bf16):
// 16 x 32768 tokens of head dim 128 118.5 us = 5.1 TB/s (75% of a plain copy's
// rate), 48 ragged ones up to 32768 94 us, 512 x 1023 140 us, 2048 x 250 192 us (an
// item's start and end weigh about two tiles); head dim 64 74 us, 192 / 128 157 us,
// 256 (8 requests) 130 us; 16 query rows a kv head 176 us; pages of 16 tokens 142
// us, of 32 129 us.
// What bounds the long ones: the instructions of a tile (about 1180 a warp for
// 64 tokens of head dim 128, half of them on the ALU pipe; 62% of the issue
// slots are taken) beside the copies: when the whole took 121 us, the tiles' work
// without copies took 115 us and the copies alone 99 us.  Short requests wait for
// instructions too (the loop and what surrounds it do not fit the first instruction
// cache).  From 9 rows a kv head on 8 warps an SM are left to hide latencies.
// Every 16 rows a kv head are an item of their own, which reads and converts the
// cache again: 4 x 8192 tokens, 4 query heads a kv head, 1, 8, 32, 128, 256 query
// tokens 20, 35, 100, 331, 647 us, where reading the cache back and attn_fwd take
// 90, 90, 90, 92, 140 us.
// Tiles of 64 tokens against 32: 16 x 32K tokens 121 / 131 us, head dim 64 75 /
// 94 us, 16 query rows 187 / 219 us; a window of 4095 (24 requests, 4 new tokens,
// 192 / 128) 35.3 / 33.0 us, where the tiles that the window's ends cut weigh
// more.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kcommon.cuh"
#include "kv.h"
#include "kvtile.cuh"

namespace attn {

constexpr int kWarps = 4;     // of a block
constexpr int kTile = 64;     // tokens of a warp's tile
constexpr int kItemCost = 2;  // in tiles: what an item costs a warp besides them (q, the list, the result)
constexpr int kExpMin = -80, kExpMax = 100;  // exponents of V's scales told apart

// Whether a lane's share is to fit 128 registers (four blocks an SM, two otherwise).
// Not all of it does: of head dims 192 / 128 156 bytes a thread spill, of 64 with 16
// rows 144, of 128 32.
__host__ __device__ constexpr bool light(int dv, int nt) { return dv * nt <= 128; }

template <int DQK, int DV, int NT>
struct DecShape {
  static constexpr int GK = DQK / 32, GV = DV / 32;
  static constexpr int kRows = 8 * NT;
  // a tile's codes and scales in shared memory, K and V apart
  static constexpr int kKc = kTile * DQK / 2, kVc = kTile * DV / 2;
  static constexpr int kKslot = kKc + kTile * GK * 2, kVslot = kVc + kTile * GV * 2;
  // blocks of an SM: as many as its registers hold
  static constexpr int kBlocks = light(DV, NT) ? 4 : 2;
  static constexpr int kDepth = DQK == 64 && NT == 1 ? 2 : 1;  // slots of each
  static constexpr int kRing = kWarps * kDepth * (kKslot + kVslot);
  static constexpr int kPart = kRows * (DV + 2);  // floats of a partial result
};

// ----------------------------------------------------------------- geometry
struct SeqRange {
  int len;      // tokens held
  int lo;       // first tile of the window part
  int n_sink;   // tiles before it that hold sinks
  int tiles;    // all tiles of the sequence that some query sees
};

__device__ __forceinline__ int seq_len(const DecodeParams& p, int b) {
  const int len = p.seq_lens[b], cap = p.cols << p.c.page_shift;
  if (len >= 0 && len <= cap) return len;
  if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
  return 0;
}
__device__ __forceinline__ SeqRange seq_range(const DecodeParams& p, int b) {
  SeqRange s;
  s.len = seq_len(p, b);
  // the first query's window starts at len - seqlen_q - window_left
  const int64_t w = p.window_left < 0 ? 0 : (int64_t)s.len - p.seqlen_q - p.window_left;
  s.lo = w > 0 ? (int)(w / kTile) : 0;
  if (p.starts) s.lo = min(p.starts[b], s.len) / kTile;  // (a call without window and first tokens)
  const int sink_tiles = (int)(((int64_t)p.sinks + kTile - 1) / kTile);
  s.n_sink = min(sink_tiles, s.lo);
  s.tiles = s.n_sink + (s.len + kTile - 1) / kTile - s.lo;
  return s;
}
// An item's share of the list of work: its tiles, and what it costs besides them.
__device__ __forceinline__ int units_of(int tiles) { return tiles ? tiles + kItemCost : 0; }
// u / n, u >= 0 (64-bit quotients are slow)
__device__ __forceinline__ long long quotient(long long u, int n) {
  return u <= INT32_MAX ? (int)u / n : u / n;
}
// tiles before position u of a sequence's items
__device__ __forceinline__ long long tiles_before(int tiles, long long u) {
  if (tiles == 0) return 0;
  const int n = units_of(tiles);
  const long long item = quotient(u, n);
  const int x = (int)(u - item * n) - kItemCost;
  return item * tiles + (x > 0 ? x : 0);
}
// first token of the v-th tile
__device__ __forceinline__ int tile_token(const SeqRange& s, int v) {
  return (v < s.n_sink ? v : s.lo + v - s.n_sink) * kTile;
}
// Runs that a call's work is cut into: one for each warp, but none without a tile.
__host__ __device__ inline long long used_runs(long long tiles, int blocks) {
  return tiles < (long long)blocks * kWarps ? tiles : (long long)blocks * kWarps;
}

// ----------------------------------------------------------------- operands
// V's, less 8 each (exact), in units of 2^-24, those of odd n 16 fold: their sums
// keep 18 bits, the probabilities have 11.
__device__ __forceinline__ void signed8(uint32_t w, uint32_t (&p)[4]) {
  p[0] = w & 0x000f000fu;
  p[1] = w & 0x00f000f0u;
  w >>= 8;
  p[2] = w & 0x000f000fu;
  p[3] = w & 0x00f000f0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t o = i & 1 ? 0x80808080u : 0x80088008u;  // -8
    const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&p[i]), *reinterpret_cast<const __half2*>(&o));
    p[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Token of row r (of 8) of a tile's block of 8: the four tokens of rows 2c and
// the four of rows 2c + 1 are neighbours, so a warp's V loads (rows 2c of all
// four c) cover 256 bytes in a row, and rows 2q, 2q + 1 lie in different
// halves of the banks, so its K loads do not collide either.
__device__ __forceinline__ int row_token(int r) {
  return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1;
}

// ----------------------------------------------------------------- a tile
// What a lane holds of its warp's piece: the query operand, O^T, and for its
// columns 2c, 2c + 1 (query rows) of each block of 8 the running statistics.
template <int DQK, int DV, int NT>
struct Piece {
  using S = DecShape<DQK, DV, NT>;
  // dims (8c + i, 8c + i + 4) of group g; those of odd i in KCodes' unit for them
  uint32_t qf[NT][S::GK][4];
  float xs[NT][2];               // from products to scores in base 2
  float o[NT][S::GV][2][4];      // dims 32 g + 4 r + {0,1}, {2,3} (odd ones 16 fold)
  // A score x (base 2) counts as 2^(x + ref), ref = kf - m: m is the column's
  // reference, kf = 14 - e with 2^e above V's scales so far.  l: this lane's
  // share of the sum; O is held times 2^-24.
  float ref[NT][2], l[NT][2];
  float lim, vlim;               // kf + 1; 2^e
};

// S^T of a tile, in units of the products: blocks of 16 tokens, rows r, r + 8.
// lows: what the codes' offset of 8 adds up to, for each group and column pair.
// (Past the last token and in pages out of range the slot's bytes are whatever
// they were: the mask hides what comes of them.)
template <int DQK, int DV, int NT>
__device__ __forceinline__ void tile_scores(const Piece<DQK, DV, NT>& z, const uint8_t* st, const float4* lows, int r,
                                            int c, float (&x)[kTile / 16][NT][4]) {
  using S = DecShape<DQK, DV, NT>;
#pragma unroll
  for (int m = 0; m < kTile / 16; ++m) {
    uint32_t sa[S::GK / 2], sb[S::GK / 2], ka[S::GK], kb[S::GK];
    const int ta = m * 16 + row_token(r), tb = ta + 8;
    lds_words<S::GK>(st + ta * (DQK / 2) + c * 4 * S::GK, ka);
    lds_words<S::GK>(st + tb * (DQK / 2) + c * 4 * S::GK, kb);
    lds_words<S::GK / 2>(st + S::kKc + ta * 2 * S::GK, sa);
    lds_words<S::GK / 2>(st + S::kKc + tb * 2 * S::GK, sb);
#pragma unroll
    for (int g = 0; g < S::GK; ++g) {
      uint32_t a[4], b[4];
      KCodes<DQK>::of(ka[g], a);
      KCodes<DQK>::of(kb[g], b);
      const float fa = scale_of(sa, g), fb = scale_of(sb, g);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t* q = z.qf[t][g];
        float acc[4];
        float(&y)[4] = x[m][t];
        const float4 lv = lows[(t * S::GK + g) * 4 + c];
        const float low[4] = {lv.x, lv.y, lv.z, lv.w};
        mma16816(acc, a[0], b[0], a[1], b[1], q[0], q[1], low);
        mma16816(acc, a[2], b[2], a[3], b[3], q[2], q[3]);
        y[0] = g ? fmaf(acc[0], fa, y[0]) : acc[0] * fa;
        y[1] = g ? fmaf(acc[1], fa, y[1]) : acc[1] * fa;
        y[2] = g ? fmaf(acc[2], fb, y[2]) : acc[2] * fb;
        y[3] = g ? fmaf(acc[3], fb, y[3]) : acc[3] * fb;
      }
    }
  }
}

// Hides what the lane's columns do not see.
template <int DQK, int DV, int NT>
__device__ __forceinline__ void tile_mask(const DecodeParams& p, int len, int row0, int t0, int r, int c,
                                          float (&x)[kTile / 16][NT][4]) {
  using S = DecShape<DQK, DV, NT>;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = row0 + t * 8 + 2 * c + e;
      const int pos = len - p.seqlen_q + (int)p.by_group.div(row);
      const int hi = row < p.rows ? pos : -1;
      const int lo = p.window_left < 0 ? 0 : max(0, pos - p.window_left);
#pragma unroll
      for (int i = 0; i < kTile / 8; ++i) {
        const int j = t0 + i * 8 + row_token(r);
        if (j > hi || (j < lo && j >= p.sinks)) x[i >> 1][t][2 * (i & 1) + e] = -INFINITY;
      }
    }
}

// What tile_top says without the infinite scales: those make the products
// infinite anyway, and must not take the others' precision.  (Rare: not inlined,
// which leaves the loop its registers: 16 x 32K tokens 116 us, inlined 121 us.)
__device__ __noinline__ float tile_top_finite(const DecodeParams& p, const uint8_t* scales, int groups, int rows,
                                              int len, int row0, int t0) {
  const int hi = len - p.seqlen_q + (int)p.by_group.div(min(row0 + rows, p.rows) - 1);
  const int lo = p.window_left < 0 ? 0 : len - p.seqlen_q + (int)p.by_group.div(row0) - p.window_left;
  float top = 0.0f;
  for (int i = threadIdx.x & 31; i < kTile; i += 32) {
    const int j = t0 + i;
    if (j > hi || (j < lo && j >= p.sinks)) continue;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(scales + i * 2 * groups);
    for (int g = 0; g < groups; ++g)
      if (scale_of(w, g) <= 3.40282347e38f) top = fmaxf(top, scale_of(w, g));
  }
  return top;
}

// Scores to probabilities, in base 2.  The reference of a column moves only when
// a score passes it by more than 1: probabilities stay below 2 (times 2^kf, and
// times V's scales below 2^15), and most tiles need no exchange between lanes.
// top: the largest V scale of this lane's tokens; st: the tile's V.
template <int DQK, int DV, int NT>
__device__ __forceinline__ void tile_softmax(const DecodeParams& p, Piece<DQK, DV, NT>& z, const uint8_t* st,
                                             int len, int row0, int t0, float top,
                                             float (&x)[kTile / 16][NT][4]) {
  using S = DecShape<DQK, DV, NT>;
  bool move = top >= z.vlim;
  float mx[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y = fmaxf(x[0][t][e], x[0][t][2 + e]);
#pragma unroll
      for (int m = 1; m < kTile / 16; ++m) y = fmax3(y, x[m][t][e], x[m][t][2 + e]);
      mx[t][e] = z.xs[t][e] * y;
      move |= mx[t][e] + z.ref[t][e] > z.lim;
    }
  bool any = __any_sync(0xffffffffu, move);
  if (any && __any_sync(0xffffffffu, top > 3.40282347e38f)) {
    top = tile_top_finite(p, st + S::kVc, S::GV, S::kRows, len, row0, t0);
    move = top >= z.vlim;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) move |= mx[t][e] + z.ref[t][e] > z.lim;
    any = __any_sync(0xffffffffu, move);
  }
  if (any) {
    const float kf_old = z.lim - 1.0f;
    float f0 = 1.0f, f1 = 1.0f;  // 2^(e_old - e), whose exponent may be below a number's
    {
      // (positive numbers: their bits are ordered)
      const uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(top, 0.0f)));
      const int e = min(max((int)(u >> 23) - 126, kExpMin), kExpMax), e_old = 15 - (int)z.lim;
      if (e > e_old) {
        f0 = pow2(max(e_old - e, -126));
        f1 = pow2(e_old - e - max(e_old - e, -126));
        z.lim = (float)(15 - e);
        z.vlim = pow2(e);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float m = kf_old - z.ref[t][e];
        float y = mx[t][e];
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
        y = fmaxf(y, m);
        const float b = ex2(m - y), a = b * f0 * f1;
        z.ref[t][e] = z.lim - 1.0f - y;
        z.l[t][e] = z.l[t][e] * b * f0 * f1;  // (the sum is up to 2^95: a alone may be 0)
#pragma unroll
        for (int g = 0; g < S::GV; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            z.o[t][g][h][e] *= a;
            z.o[t][g][h][2 + e] *= a;
          }
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint64_t xs = f2_pack(z.xs[t][0], z.xs[t][1]), ref = f2_pack(z.ref[t][0], z.ref[t][1]);
    uint64_t sum = f2_pack(z.l[t][0], z.l[t][1]);
#pragma unroll
    for (int m = 0; m < kTile / 16; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float& y0 = x[m][t][2 * h];
        float& y1 = x[m][t][2 * h + 1];
        f2_unpack(f2_fma(f2_pack(y0, y1), xs, ref), y0, y1);
        y0 = ex2(y0);
        y1 = ex2(y1);
        sum = f2_add(sum, f2_pack(y0, y1));
      }
    f2_unpack(sum, z.l[t][0], z.l[t][1]);
  }
}

// The largest V scale (NaN apart) of this lane's tokens (every 32nd) of a tile.
// Where some query does not see all of it: tokens that no query sees do not
// count, their scales may be anything; those past the last token are set to
// zero in the slot, and `odd` is set if a scale of the others is not finite.
template <int DQK, int DV, int NT>
__device__ __forceinline__ float tile_top(const DecodeParams& p, uint8_t* st, bool whole, int len, int row0,
                                          int t0, int lane, bool& odd) {
  using S = DecShape<DQK, DV, NT>;
  float top[kTile / 32];
#pragma unroll
  for (int h = 0; h < kTile / 32; ++h) {
    uint32_t w[S::GV / 2];
    lds_words<S::GV / 2>(st + S::kVc + (h * 32 + lane) * 2 * S::GV, w);
    __nv_bfloat162 y = *reinterpret_cast<__nv_bfloat162*>(&w[0]);
#pragma unroll
    for (int i = 1; i < S::GV / 2; ++i) y = __hmax2(y, *reinterpret_cast<__nv_bfloat162*>(&w[i]));
    const uint32_t u = *reinterpret_cast<uint32_t*>(&y);
    top[h] = fmaxf(scale_of(&u, 0), scale_of(&u, 1));
  }
  if (!whole) {
    const int hi = len - p.seqlen_q + (int)p.by_group.div(min(row0 + S::kRows, p.rows) - 1);
    const int lo = p.window_left < 0 ? 0 : len - p.seqlen_q + (int)p.by_group.div(row0) - p.window_left;
#pragma unroll
    for (int h = 0; h < kTile / 32; ++h) {
      const int j = t0 + h * 32 + lane;
      uint32_t* w = reinterpret_cast<uint32_t*>(st + S::kVc + (h * 32 + lane) * 2 * S::GV);
#pragma unroll
      for (int i = 0; i < S::GV / 2; ++i) {
        if (j >= len) w[i] = 0u;
        odd |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
      }
      if (j > hi || (j < lo && j >= p.sinks)) top[h] = 0.0f;
    }
    __syncwarp();
  }
  return fmaxf(top[0], top[1]);
}

// O^T += V^T P^T.  ODD: a scale is not finite, and hidden pairs must not see it.
template <bool ODD, int DQK, int DV, int NT>
__device__ __forceinline__ void tile_values(Piece<DQK, DV, NT>& z, const uint8_t* st, int r, int c,
                                            const float (&x)[kTile / 16][NT][4]) {
  using S = DecShape<DQK, DV, NT>;
#pragma unroll
  for (int mt = 0; mt < kTile / 16; ++mt) {
    uint32_t vs[2][S::GV / 2];  // scales of tokens r and r + 8
#pragma unroll
    for (int h = 0; h < 2; ++h)
      lds_words<S::GV / 2>(st + S::kVc + (mt * 16 + h * 8 + row_token(r)) * 2 * S::GV, vs[h]);
    uint32_t v0[S::GV / 2], v1[S::GV / 2], v2[S::GV / 2], v3[S::GV / 2];
    const uint8_t* vb = st + r * 2 * S::GV;
    const int te = mt * 16 + row_token(2 * c), to = mt * 16 + row_token(2 * c + 1);
    lds_words<S::GV / 2>(vb + te * (DV / 2), v0);
    lds_words<S::GV / 2>(vb + to * (DV / 2), v1);
    lds_words<S::GV / 2>(vb + (te + 8) * (DV / 2), v2);
    lds_words<S::GV / 2>(vb + (to + 8) * (DV / 2), v3);
#pragma unroll
    for (int g = 0; g < S::GV; ++g) {
      const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
      uint32_t a[4], b[4];
      signed8(__byte_perm(v0[g >> 1], v1[g >> 1], sel), a);
      signed8(__byte_perm(v2[g >> 1], v3[g >> 1], sel), b);
      const float fa = scale_of(vs[0], g), fb = scale_of(vs[1], g);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float p0, p1, p2, p3;
        f2_unpack(f2_mul(f2_pack(x[mt][t][0], x[mt][t][2]), f2_pack(fa, fb)), p0, p2);
        f2_unpack(f2_mul(f2_pack(x[mt][t][1], x[mt][t][3]), f2_pack(fa, fb)), p1, p3);
        if (ODD) {
          p0 = x[mt][t][0] == 0.0f ? 0.0f : p0;
          p1 = x[mt][t][1] == 0.0f ? 0.0f : p1;
          p2 = x[mt][t][2] == 0.0f ? 0.0f : p2;
          p3 = x[mt][t][3] == 0.0f ? 0.0f : p3;
        }
        const uint32_t b0 = transpose8x8(Pack<false>::two(p0, p1));
        const uint32_t b1 = transpose8x8(Pack<false>::two(p2, p3));
        mma16816(z.o[t][g][0], a[0], a[1], b[0], b[1], b0, b1);
        mma16816(z.o[t][g][1], a[2], a[3], b[2], b[3], b0, b1);
      }
    }
  }
}

// Where a finished row goes: O = acc / sum, LSE = (mx + log2 sum) ln 2.
struct RowOut {
  int64_t o, lse;
  __device__ __forceinline__ RowOut(const DecodeParams& p, int b, int kvh, int row) {
    const int qi = (int)p.by_group.div(row), qh = kvh * p.group + row - qi * p.group;
    o = b * p.o_b + qi * p.o_t + qh * p.o_h;
    lse = ((int64_t)b * p.heads_q + qh) * p.seqlen_q + qi;
  }
  // dims 4 d4 .. + 3
  template <bool BF16>
  __device__ __forceinline__ void write(const DecodeParams& p, int d4, const float4& y) const {
    if (p.o_f32)
      *reinterpret_cast<float4*>((float*)p.o + o + d4 * 4) = y;
    else
      *reinterpret_cast<uint2*>((uint16_t*)p.o + o + d4 * 4) =
          make_uint2(Pack<BF16>::two(y.x, y.y), Pack<BF16>::two(y.z, y.w));
  }
  __device__ __forceinline__ void write_lse(const DecodeParams& p, float mx, float sum) const {
    p.lse[lse] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
  }
};
// 1 / sum; 0 where no token is visible (sum is NaN where a score is, and O with it)
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
// Four dims of a row, and with the first of them its LSE.
template <bool BF16>
__device__ __forceinline__ void write_row(const DecodeParams& p, int b, int kvh, int row, int d4,
                                          const float4& acc, float mx, float sum) {
  const RowOut out(p, b, kvh, row);
  const float inv = inverse(sum);
  out.write<BF16>(p, d4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (d4 == 0) out.write_lse(p, mx, sum);
}

// ----------------------------------------------------------------- the kernel
// A place in the list of tiles: tile v of an item of a sequence.
struct Cursor {
  int b, item, v;
  SeqRange sr;
};
// Tiles in a row that a warp copies next.
struct __align__(16) Strip {
  const int32_t* row;  // of the block table
  int token, left;     // of the tile looked up last; tiles after it
  int head_row, len;   // first row of the kv head in a page; tokens of the sequence
};
// Moves `n` tiles on.  Past the end of the list (lengths that changed under the
// call): b = batch.
__device__ __forceinline__ void advance(const DecodeParams& p, int per_seq, Cursor& k, int n) {
  k.v += n;
  while (k.b < p.batch && k.v >= k.sr.tiles) {
    k.v -= k.sr.tiles;
    if (k.sr.tiles == 0 || ++k.item == per_seq) {
      k.item = 0;
      if (++k.b < p.batch) k.sr = seq_range(p, k.b);
    }
  }
}

template <bool BF16, int DQK, int DV, int NT>
__global__ void __launch_bounds__(kWarps * 32, DecShape<DQK, DV, NT>::kBlocks)
    attn_kv_decode_kernel(const __grid_constant__ DecodeParams p) {
  using S = DecShape<DQK, DV, NT>;
  constexpr int kThreads = kWarps * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Cursor copy_at[kWarps], work_at[kWarps];
  __shared__ Strip strip[kWarps];
  __shared__ float4 lows[kWarps][NT * S::GK * 4];
  __shared__ long long s_sum[2 * kWarps], s_tiles[kWarps][2], s_before[kWarps];
  __shared__ int s_b[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");  // (the join waits for the whole grid)
  // Beside a shared prefix this grid starts before the prefix kernel ends, and must
  // not end before it does, since the joins wait for this one alone: one block more does
  // nothing but wait.  (A wait wherever a block returns cost 16 x 32K tokens without a
  // prefix 121 us against 117; one at the start of a block that works 5 of 4 requests' 31.)
  if (p.starts && blockIdx.x == gridDim.x - 1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (tid < kWarps) {
    s_b[tid] = p.batch;
    s_before[tid] = s_tiles[tid][0] = s_tiles[tid][1] = 0;
  }
  // ---- the list of work, and its warps' runs of it.  Each thread takes the
  // sequences b = tid, tid + kThreads, ..: units and tiles are added up over
  // chunks of kThreads sequences, first all of them for the totals (where there
  // are more than one chunk), then as prefix sums.
  const int per_seq = p.c.heads * p.row_blocks;  // items of a sequence
  long long before_u = 0, before_t = 0;  // of the chunks so far
  int nt = 0;                      // this thread's sequence of the chunk
  long long u0 = 0, t0 = 0;        // units and tiles before it (of one item of each sequence)
  auto chunk = [&](int b0) {
    nt = b0 + tid < p.batch ? seq_range(p, b0 + tid).tiles : 0;
    const int mine = units_of(nt);
    long long ju = mine, jt = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, ju, o), y = __shfl_up_sync(0xffffffffu, jt, o);
      if (lane >= o) ju += x, jt += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = ju, s_sum[kWarps + warp] = jt;
    __syncthreads();
    u0 = before_u + ju - mine;
    t0 = before_t + jt - nt;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) u0 += s_sum[w], t0 += s_sum[kWarps + w];
      before_u += s_sum[w];
      before_t += s_sum[kWarps + w];
    }
  };
  chunk(0);
  for (int b0 = kThreads; b0 < p.batch; b0 += kThreads) chunk(b0);
  const long long all = before_u * per_seq;
  const long long n_runs = used_runs(before_t * per_seq, (int)gridDim.x - (p.starts ? 1 : 0));
  const long long run0 = (long long)blockIdx.x * kWarps;
  // blocks without a run: nothing to join there
  if (tid < kWarps && run0 + tid >= n_runs) p.ends[run0 + tid] = -1;
  if (run0 >= n_runs) return;
  // run k has units [bound(k), bound(k + 1))
  const long long each = quotient(all, (int)n_runs), more = all - each * n_runs;
  auto bound = [&](long long k) { return each * k + min(k, more); };
  // the sequences that hold the runs' first units, and the tiles before both ends
  if (p.batch > kThreads) before_u = before_t = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    if (p.batch > kThreads) chunk(b0);
    const long long n = (long long)units_of(nt) * per_seq, first_u = u0 * per_seq;
    for (int w = 0; w < kWarps && run0 + w < n_runs; ++w) {
      const long long first = bound(run0 + w), last = bound(run0 + w + 1);
      if (first >= first_u && first < first_u + n) {
        s_b[w] = b0 + tid;
        s_before[w] = first_u;
        s_tiles[w][0] = t0 * per_seq + tiles_before(nt, first - first_u);
      }
      if (last > first_u && last <= first_u + n)
        s_tiles[w][1] = t0 * per_seq + tiles_before(nt, last - first_u);
    }
    if (before_u * per_seq >= bound(min(run0 + kWarps, n_runs))) break;
  }
  __syncthreads();
  // From here on the warps go their own ways.
  const long long run = run0 + warp;
  const int first_b = s_b[warp];
  const int n_run = (int)min(max(s_tiles[warp][1] - s_tiles[warp][0], 0ll), (long long)INT32_MAX);
  if (run >= n_runs) return;
  if (first_b >= p.batch || n_run == 0) {
    if (lane == 0) p.ends[run] = -1;
    return;
  }

  const int r = lane >> 2, c = lane & 3;
  uint8_t* k_ring = smem + warp * (S::kDepth * (S::kKslot + S::kVslot));
  uint8_t* v_ring = k_ring + S::kDepth * S::kKslot;
  // ---- copies.  A warp feeds its own slots, across the items of its run, by
  // 16-byte asynchronous copies of all its lanes (a tile of one array is one
  // run of bytes); it waits for its own copies alone.  K and V have slots of
  // their own: the next K is on its way while V is used, and the other way
  // round.  Where the next tile lies is looked up one tile ahead.
  if (lane == 0) {
    Cursor k;
    k.b = first_b;
    k.sr = seq_range(p, first_b);
    const long long u = bound(run) - s_before[warp];
    const int n = max(units_of(k.sr.tiles), 1);
    const long long i = quotient(u, n);
    k.item = (int)min(i, (long long)INT32_MAX);
    k.v = max((int)(u - i * n) - kItemCost, 0);
    if (k.item >= per_seq) k.b = p.batch;  // lengths that changed under the call
    advance(p, per_seq, k, 0);
    copy_at[warp] = work_at[warp] = k;
    strip[warp].left = 0;
  }
  // Page of the tile to copy next: lane i's is that of its tokens
  // 16 (i % (kTile / 16)) .. (all the same for pages of a tile or more).
  int next_page = 0;
  auto look_up = [&]() {
    __syncwarp();
    if (strip[warp].left == 0) {
      __syncwarp();
      if (lane == 0) {
        Cursor k = copy_at[warp];
        Strip t{p.table, 0, 1, 0, 0};  // no tile (lengths that changed under the call)
        if (k.b < p.batch) {
          const int stop = k.v < k.sr.n_sink ? k.sr.n_sink : k.sr.tiles;
          t.row = p.table + (int64_t)k.b * p.table_stride;
          t.token = tile_token(k.sr, k.v) - kTile;
          t.left = stop - k.v;
          t.head_row = ((int)p.by_blocks.div(k.item)) * p.c.page_size;
          t.len = k.sr.len;
          advance(p, per_seq, k, t.left);
          copy_at[warp] = k;
        }
        strip[warp] = t;
      }
      __syncwarp();
    }
    const int token = strip[warp].token + kTile, left = strip[warp].left - 1;
    const int len = strip[warp].len;
    if (token < len) next_page = strip[warp].row[min(token + 16 * (lane % (kTile / 16)), len - 1) >> p.c.page_shift];
    __syncwarp();
    if (lane == 0) strip[warp].token = token, strip[warp].left = left;
  };
  // Tokens first .. first + ROWS of the tile looked up last, its K or its V:
  // they lie in one page.
  auto copy_rows = [&](auto is_k, auto rows, uint8_t* slot, int page, int first) {
    constexpr bool K = decltype(is_k)::value;
    constexpr int ROWS = decltype(rows)::value, W = K ? DQK / 2 : DV / 2, G = K ? S::GK : S::GV;
    if ((unsigned)page >= (unsigned)p.c.num_pages) return;
    const int row = strip[warp].head_row + ((strip[warp].token + first) & (p.c.page_size - 1));
    const int64_t at = (int64_t)page * (p.c.heads * p.c.page_size) + row;
    auto run = [&](uint32_t dst, const uint8_t* src, auto bytes_of) {
      constexpr int N = ROWS * decltype(bytes_of)::value;
      dst += first * decltype(bytes_of)::value + lane * 16;
      src += at * decltype(bytes_of)::value + lane * 16;
#pragma unroll
      for (int i = 0; i < N; i += 512)
        if (N - i >= 512 || lane * 16 < N - i) copy16(dst + i, src + i);
    };
    run(smem_u32(slot), K ? p.c.k_codes : p.c.v_codes, std::integral_constant<int, W>());
    run(smem_u32(slot) + kTile * W, reinterpret_cast<const uint8_t*>(K ? p.c.k_scales : p.c.v_scales),
        std::integral_constant<int, 2 * G>());
  };
  auto copy = [&](auto is_k, uint8_t* slot) {
    __syncwarp();
    const int left = strip[warp].len - strip[warp].token;
    if (left <= 0) return;
    if (decltype(is_k)::value && (unsigned)next_page >= (unsigned)p.c.num_pages && p.status) {
      // A page outside the cache is not copied.  One that no query looks into,
      // between the first tokens and the window, may be gone: what the slot held
      // before is masked like any hidden token.
      const int i = 16 * (lane % (kTile / 16)), t = strip[warp].token + i;
      if (i < left && (p.window_left < 0 || t < p.sinks || t + 16 > strip[warp].len - p.seqlen_q - p.window_left))
        atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    }
    auto pieces = [&](auto rows) {
      constexpr int ROWS = decltype(rows)::value;
#pragma unroll
      for (int i = 0; i < kTile; i += ROWS)
        if (i < left) copy_rows(is_k, rows, slot, __shfl_sync(0xffffffffu, next_page, i / 16), i);
    };
    if (p.c.page_size >= kTile)
      copy_rows(is_k, std::integral_constant<int, kTile>(), slot, next_page, 0);
    else if (p.c.page_size == 32)
      pieces(std::integral_constant<int, 32>());
    else
      pieces(std::integral_constant<int, 16>());
  };
  int used = 0;
  look_up();
  for (int i = 0; i < S::kDepth; ++i) {
    if (i < n_run) copy(std::true_type(), k_ring + i * S::kKslot);
    copies_end();
    if (i < n_run) copy(std::false_type(), v_ring + i * S::kVslot);
    copies_end();
    if (i + 1 < n_run) look_up();
  }
  for (int pieces = 0; used < n_run; ++pieces) {
    // the piece: the run's tiles of one item
    const Cursor k = work_at[warp];
    if (k.b >= p.batch) {  // lengths that changed under the call
      if (pieces == 0 && lane == 0) p.ends[run] = -1;
      break;
    }
    const SeqRange sr = k.sr;
    const int b = k.b, item = k.item, v0 = k.v, v1 = min(sr.tiles, v0 + n_run - used);
    const int kvh = (int)p.by_blocks.div(item), rb = item - kvh * p.row_blocks;
    __syncwarp();
    if (lane == 0) {
      // for the join: the first and the last run that work on an item, and
      // the items that a run ends for others
      int* info = p.info + 2 * ((int64_t)b * per_seq + item);
      if (v0 == 0) info[0] = (int)run;
      if (v1 == sr.tiles) info[1] = (int)run;
      if (pieces == 0) p.ends[run] = v0 > 0 && v1 == sr.tiles ? (int)(b * per_seq + item) : -1;
      Cursor n = k;
      advance(p, per_seq, n, v1 - v0);
      work_at[warp] = n;
    }

    Piece<DQK, DV, NT> z;
    const int row0 = rb * S::kRows;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = row0 + t * 8 + r;
      const int qi = (int)p.by_group.div(row), qh = kvh * p.group + row - qi * p.group;
      const uint16_t* src = (const uint16_t*)p.q + b * p.q_b + qi * p.q_t + qh * p.q_h + 8 * c;
      uint4 qv[S::GK];
      uint32_t top = 0;  // largest magnitude: as bits they are ordered
#pragma unroll
      for (int g = 0; g < S::GK; ++g) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.rows) v = *reinterpret_cast<const uint4*>(src + 32 * g);
        qv[g] = v;
        const uint32_t mx = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        top = max(top, max(mx & 0xffffu, mx >> 16));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t tf = __float_as_uint(Pack<BF16>::to_f((uint16_t)top));
      const int ex = min(max((int)(tf >> 23) - 127 - 13, -100), 100);  // largest at 2^13 .. 2^14
      const float inv = pow2(-ex);
#pragma unroll
      for (int g = 0; g < S::GK; ++g) {
        const uint32_t w[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = Pack<BF16>::to_f((uint16_t)(w[i >> 1] >> (16 * (i & 1)))) * ((i & 1) ? inv * KCodes<DQK>::kOdd : inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) z.qf[t][g][i] = Pack<false>::two(f[i], f[i + 4]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // (not 0, whatever the scale: times -inf that would be NaN)
        z.xs[t][e] = fmaxf(p.scale_log2 * KCodes<DQK>::kUnit * __shfl_sync(0xffffffffu, pow2(ex), (2 * c + e) * 4),
                           1.17549435e-38f);
        z.ref[t][e] = 1e30f;  // nothing seen yet: a reference below any score
        z.l[t][e] = 0.0f;
      }
#pragma unroll
      for (int g = 0; g < S::GV; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) z.o[t][g][h][e] = 0.0f;
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int g = 0; g < S::GK; ++g) {
        const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float low[4];
        constexpr uint32_t even = KCodes<DQK>::kEven8, odd = KCodes<DQK>::kOdd8;
        mma16816(low, even, even, odd, odd, z.qf[t][g][0], z.qf[t][g][1], zero);
        mma16816(low, even, even, odd, odd, z.qf[t][g][2], z.qf[t][g][3]);
        if (r == 0) lows[warp][(t * S::GK + g) * 4 + c] = make_float4(low[0], low[1], low[2], low[3]);
      }
    __syncwarp();
    z.lim = (float)(15 - kExpMin);
    z.vlim = pow2(kExpMin);
    // every query of the item sees token j if j <= pos_lo and (j >= pos_hi -
    // window_left or j < sinks); columns past the last row hold zeros, and what
    // they sum up is not written
    const int pos_lo = sr.len - p.seqlen_q + (int)p.by_group.div(row0);
    const int pos_hi = sr.len - p.seqlen_q + (int)p.by_group.div(min(row0 + S::kRows, p.rows) - 1);

    const int whole_hi = pos_lo - (kTile - 1);
    const int whole_lo = p.window_left < 0 ? 0 : pos_hi - p.window_left;
    for (int v = v0; v < v1; ++v) {
      const int s = used % S::kDepth;
      const bool more = used + S::kDepth < n_run;
      ++used;
      const int t0 = tile_token(sr, v);
      const bool whole = t0 <= whole_hi && (t0 >= whole_lo || t0 + kTile <= p.sinks);
      uint8_t *ks = k_ring + s * S::kKslot, *vs = v_ring + s * S::kVslot;
      float x[kTile / 16][NT][4];
      copies_wait<2 * S::kDepth - 1>();
      __syncwarp();
      tile_scores(z, ks, lows[warp], r, c, x);
      if (!whole) tile_mask<DQK, DV, NT>(p, sr.len, row0, t0, r, c, x);
      if (more) copy(std::true_type(), ks);
      copies_end();
      copies_wait<2 * S::kDepth - 1>();
      __syncwarp();
      bool odd = false;
      const float top = tile_top<DQK, DV, NT>(p, vs, whole, sr.len, row0, t0, lane, odd);
      tile_softmax(p, z, vs, sr.len, row0, t0, top, x);
      if (__any_sync(0xffffffffu, odd))
        tile_values<true>(z, vs, r, c, x);
      else
        tile_values<false>(z, vs, r, c, x);
      if (more) {
        copy(std::false_type(), vs);
        if (used + S::kDepth < n_run) look_up();
      }
      copies_end();
    }

    // ---- the result, or a partial one: O and the sum relative to the reference m.
    // (2^-kf is taken off a partial one: the join's weights are differences of
    // references, and two warps' units may be 2^180 apart.)
    const bool done = v0 == 0 && v1 == sr.tiles;
    const float unit = pow2(1 - (int)z.lim);
    float* part = p.partial + (run * 2 + (v0 == 0 ? 1 : 0)) * S::kPart;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = z.l[t][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = t * 8 + 2 * c + e, row_all = row0 + row;
        if (row_all >= p.rows) continue;
        // dims 32 g + 4 r .. + 3 times f
        auto dims = [&](int g, float f) {
          const float lo = f * 16777216.0f, hi = f * 1048576.0f;
          return make_float4(z.o[t][g][0][e] * lo, z.o[t][g][0][2 + e] * hi, z.o[t][g][1][e] * lo,
                             z.o[t][g][1][2 + e] * hi);
        };
        if (done) {
          const RowOut out(p, b, kvh, row_all);
          const float inv = inverse(sum);
#pragma unroll
          for (int g = 0; g < S::GV; ++g) out.write<BF16>(p, 8 * g + r, dims(g, inv));
          if (r == 0) out.write_lse(p, -z.ref[t][e], sum);
        } else {
#pragma unroll
          for (int g = 0; g < S::GV; ++g)
            *reinterpret_cast<float4*>(part + row * DV + 32 * g + 4 * r) = dims(g, unit);
          if (r == 0) {
            part[S::kRows * DV + row] = z.lim - 1.0f - z.ref[t][e];
            part[S::kRows * (DV + 1) + row] = sum * unit;
          }
        }
      }
  }
  copies_wait<0>();
}

// ----------------------------------------------------------------- the join
// A thread takes four dims of a row.  Rows of sequences without a visible key
// get O = 0 and LSE = -inf here.
//
// By item: a block for each row of each item, whose pieces are shared out over
// groups of threads; the groups' sums are added in their order.  It spreads the
// work best where few items are cut into many pieces; where they are cut into very
// many, the blocks are larger (one request of 65536 tokens, 8 kv heads: 256
// threads 34.8 us, 1024 29.7 us; 10^6 tokens, one kv head: 111 and 63 us; 16 x 32K
// tokens: 117 and 125 us).  By run: 128 threads look
// at a run, and join the item that it ends for others (the whole block does
// where that has many pieces): no more blocks than the runs need, however many
// items there are.  Measured, whole call: 128 items (16 x 32K tokens) by item
// 131 us, by run 137 us; 4096 items (512 x 1K) by item 170 us, by run 148 us.
constexpr int kByItemPieces = 4;  // of an item on average: from there on by item
constexpr int kTeamPieces = 8;    // joined by one team after another
constexpr int kManyPieces = 64;   // of an item on average: from there on by item in larger blocks
constexpr int kByItemThreads = 256, kManyThreads = 1024, kTeam = 128, kByRunThreads = kTeam * kWarps;

// Adds a piece of a row (reference m, sum l, O y) to what a thread holds.
__device__ __forceinline__ void add_piece(float4& acc, float& sum, float& mx, float m, float l,
                                          const float4& y) {
  const float to = fmaxf(mx, m), f = ex2(m - to), a = mx == -INFINITY ? 0.0f : ex2(mx - to);
  mx = to;
  sum = fmaf(sum, a, l * f);
  acc.x = fmaf(acc.x, a, y.x * f), acc.y = fmaf(acc.y, a, y.y * f);
  acc.z = fmaf(acc.z, a, y.z * f), acc.w = fmaf(acc.w, a, y.w * f);
}

// Sequences blockIdx.x, + gridDim.x, ..: this comes before the wait, since it
// needs nothing of the first kernel.
template <bool BF16>
__device__ __forceinline__ void empty_rows(const DecodeParams& p, int threads) {
  const int q = p.c.d_v / 4, lanes = threads / q;  // rows at a time
  const int r0 = threadIdx.x / q, d4 = threadIdx.x - r0 * q;
  for (int64_t b0 = blockIdx.x; b0 < p.batch; b0 += (int64_t)threads * gridDim.x) {
    const int64_t mine = b0 + (int64_t)threadIdx.x * gridDim.x;
    const bool empty = mine < p.batch && seq_len(p, (int)mine) == 0;
    if (!__syncthreads_or(empty)) continue;
    for (int64_t b = b0; b < p.batch && b < b0 + (int64_t)threads * gridDim.x; b += gridDim.x) {
      if (seq_len(p, (int)b)) continue;
      for (int64_t i = r0; i < (int64_t)p.c.heads * p.rows; i += lanes) {
        const int kvh = (int)(i / p.rows), row = (int)(i - (int64_t)kvh * p.rows);
        write_row<BF16>(p, (int)b, kvh, row, d4, make_float4(0.f, 0.f, 0.f, 0.f), 0.0f, 0.0f);
      }
    }
  }
}

template <bool BF16, int DV, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) attn_kv_join_items_kernel(
    const __grid_constant__ DecodeParams p, int runs) {
  constexpr int kPart = ROWS * (DV + 2), kLanes = DV / 4, kGroups = THREADS / kLanes;
  __shared__ float4 sm_o[kGroups][kLanes];
  __shared__ float sm_l[kGroups], sm_m[kGroups];
  const int per_seq = p.c.heads * p.row_blocks, tid = threadIdx.x;
  const int rows = min(ROWS, p.rows);
  const int at = blockIdx.x / rows, row = blockIdx.x - at * rows;
  const int b = at / per_seq, item = at - b * per_seq;
  const int kvh = (int)p.by_blocks.div(item), row_all = (item - kvh * p.row_blocks) * ROWS + row;
  asm volatile("griddepcontrol.launch_dependents;");  // (a kernel that joins this with other parts)
  empty_rows<BF16>(p, THREADS);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row_all >= p.rows || seq_len(p, b) == 0) return;
  const int k0 = p.info[2 * (int64_t)at], k1 = p.info[2 * (int64_t)at + 1];
  // (equal: one run finished it; out of range: lengths that changed under the call)
  if (k0 < 0 || k1 <= k0 || k1 >= runs) return;
  const int np = k1 - k0 + 1;
  const int g = tid / kLanes, d4 = tid % kLanes;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.0f, mx = -INFINITY;
#pragma unroll 8
  for (int i = g; i < np; i += kGroups) {
    const float* pc = p.partial + ((int64_t)(k0 + i) * 2 + (i == 0 ? 1 : 0)) * kPart;
    add_piece(acc, sum, mx, pc[ROWS * DV + row], pc[ROWS * (DV + 1) + row],
              *reinterpret_cast<const float4*>(pc + row * DV + d4 * 4));
  }
  sm_o[g][d4] = acc;
  if (d4 == 0) sm_l[g] = sum, sm_m[g] = mx;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k)
    if (k < np) add_piece(acc, sum, mx, sm_m[k], sm_l[k], sm_o[k][d4]);
  write_row<BF16>(p, b, kvh, row_all, d4, acc, mx, sum);
}

template <bool BF16, int DV, int ROWS>
__global__ void __launch_bounds__(kByRunThreads) attn_kv_join_runs_kernel(
    const __grid_constant__ DecodeParams p) {
  constexpr int kPart = ROWS * (DV + 2), kLanes = DV / 4, kEach = ROWS * kLanes / kTeam;
  __shared__ float4 sm_o[kByRunThreads];
  __shared__ float sm_l[kByRunThreads], sm_m[kByRunThreads];
  __shared__ int s_at[kWarps], s_k0[kWarps], s_np[kWarps];
  const int per_seq = p.c.heads * p.row_blocks, tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  empty_rows<BF16>(p, kByRunThreads);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < kWarps) {
    const int run = blockIdx.x * kWarps + tid, at = p.ends[run];
    const int k0 = at < 0 ? 0 : p.info[2 * (int64_t)at];
    s_at[tid] = at;
    s_k0[tid] = k0;
    s_np[tid] = at < 0 || k0 < 0 || k0 >= run ? 0 : run - k0 + 1;
  }
  __syncthreads();
  auto piece = [&](int k0, int i) { return p.partial + ((int64_t)(k0 + i) * 2 + (i == 0 ? 1 : 0)) * kPart; };
  // ---- items of many pieces: by the whole block, in groups
  for (int w = 0; w < kWarps; ++w) {
    const int np = s_np[w];
    if (np <= kTeamPieces) continue;
    const int b = s_at[w] / per_seq, item = s_at[w] - b * per_seq;
    const int kvh = (int)p.by_blocks.div(item), row0 = (item - kvh * p.row_blocks) * ROWS;
    const int need = min(ROWS, p.rows - row0) * kLanes, groups = kByRunThreads / need;
    const int g = tid / need, i0 = tid - g * need, row = i0 / kLanes, d4 = i0 % kLanes;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.0f, mx = -INFINITY;
    if (g < groups) {
#pragma unroll 4
      for (int i = g; i < np; i += groups) {
        const float* pc = piece(s_k0[w], i);
        add_piece(acc, sum, mx, pc[ROWS * DV + row], pc[ROWS * (DV + 1) + row],
                  *reinterpret_cast<const float4*>(pc + row * DV + d4 * 4));
      }
    }
    __syncthreads();
    sm_o[tid] = acc;
    sm_l[tid] = sum;
    sm_m[tid] = mx;
    __syncthreads();
    if (g > 0) continue;
    for (int k = 1; k < groups; ++k)
      add_piece(acc, sum, mx, sm_m[k * need + tid], sm_l[k * need + tid], sm_o[k * need + tid]);
    write_row<BF16>(p, b, kvh, row0 + row, d4, acc, mx, sum);
  }
  // ---- the others: by a team each
  const int w = tid / kTeam, t = tid % kTeam, np = s_np[w];
  if (np < 2 || np > kTeamPieces) return;
  const int b = s_at[w] / per_seq, item = s_at[w] - b * per_seq;
  const int kvh = (int)p.by_blocks.div(item), row0 = (item - kvh * p.row_blocks) * ROWS;
  float4 acc[kEach];
  float sum[kEach], mx[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f), sum[j] = 0.0f, mx[j] = -INFINITY;
#pragma unroll 2
  for (int i = 0; i < np; ++i) {
    const float* pc = piece(s_k0[w], i);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {  // (rows past the last one are read too: they lie in the workspace)
      const int at4 = j * kTeam + t, row = at4 / kLanes;
      add_piece(acc[j], sum[j], mx[j], pc[ROWS * DV + row], pc[ROWS * (DV + 1) + row],
                *reinterpret_cast<const float4*>(pc + at4 * 4));
    }
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int at4 = j * kTeam + t, row = at4 / kLanes;
    if (row0 + row < p.rows) write_row<BF16>(p, b, kvh, row0 + row, at4 % kLanes, acc[j], mx[j], sum[j]);
  }
}

// ----------------------------------------------------------------- launches
// (At d_v 256 a lane's share of O for 16 rows would not fit its registers.)
int decode_col_tiles(int rows, int d_v) { return rows > 8 && d_v < 256 ? 2 : 1; }

int decode_blocks(const DecodeParams& p, int num_sms) {
  // no more than the longest possible list of tiles keeps busy
  const int64_t tiles = (((int64_t)p.cols << p.c.page_shift) + kTile - 1) / kTile;
  const int most = num_sms * (light(p.c.d_v, decode_col_tiles(p.rows, p.c.d_v)) ? 4 : 2);
  const int64_t runs = used_runs(tiles * p.batch * p.c.heads * p.row_blocks, most);
  return (int)std::max<int64_t>((runs + kWarps - 1) / kWarps, 1);
}

size_t decode_runs(int blocks) { return (size_t)blocks * kWarps; }

size_t decode_partial_floats(int blocks, int rows_per_block, int d_v) {
  return (size_t)blocks * kWarps * 2 * rows_per_block * (d_v + 2);
}

namespace {

// Dynamic shared memory beyond what every kernel may take, asked for once on
// each device (`done`: a bit for each, of this kernel).
template <typename F>
cudaError_t allow_smem(F* f, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <bool BF16, int DQK, int DV, int NT>
cudaError_t dec_launch(const DecodeParams& p, int blocks, cudaStream_t st) {
  using S = DecShape<DQK, DV, NT>;
  auto* main = attn_kv_decode_kernel<BF16, DQK, DV, NT>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(main, S::kRing, done);
  if (e != cudaSuccess) return e;
  // the join is launched while the first kernel runs, and waits for its end (beside a
  // shared prefix the first kernel is launched like that too)
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = p.starts ? 1 : 0;
  cfg.gridDim = dim3((unsigned)blocks + (p.starts ? 1 : 0));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = S::kRing;
  e = cudaLaunchKernelEx(&cfg, main, p);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = 0;
  const int64_t items = (int64_t)p.batch * p.c.heads * p.row_blocks;
  const int runs = blocks * kWarps;
  if (items * kByItemPieces <= runs) {
    cfg.gridDim = dim3((unsigned)(items * std::min(8 * NT, p.rows)));
    const bool many = items * kManyPieces <= runs;
    cfg.blockDim = dim3(many ? kManyThreads : kByItemThreads);
    return many ? cudaLaunchKernelEx(&cfg, attn_kv_join_items_kernel<BF16, DV, 8 * NT, kManyThreads>, p, runs)
                : cudaLaunchKernelEx(&cfg, attn_kv_join_items_kernel<BF16, DV, 8 * NT, kByItemThreads>, p, runs);
  }
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kByRunThreads);
  return cudaLaunchKernelEx(&cfg, attn_kv_join_runs_kernel<BF16, DV, 8 * NT>, p);
}

template <bool BF16, int NT>
cudaError_t dec_dims(const DecodeParams& p, int blocks, cudaStream_t st) {
  if constexpr (NT == 1)
    if (p.c.d_qk == 256 && p.c.d_v == 256) return dec_launch<BF16, 256, 256, 1>(p, blocks, st);
  if (p.c.d_qk == 64 && p.c.d_v == 64) return dec_launch<BF16, 64, 64, NT>(p, blocks, st);
  if (p.c.d_qk == 128 && p.c.d_v == 128) return dec_launch<BF16, 128, 128, NT>(p, blocks, st);
  if (p.c.d_qk == 192 && p.c.d_v == 128) return dec_launch<BF16, 192, 128, NT>(p, blocks, st);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_kv4_decode(const DecodeParams& p, bool bf16, int blocks, cudaStream_t st) {
  const bool wide = decode_col_tiles(p.rows, p.c.d_v) == 2;
  if (bf16) return wide ? dec_dims<true, 2>(p, blocks, st) : dec_dims<true, 1>(p, blocks, st);
  return wide ? dec_dims<false, 2>(p, blocks, st) : dec_dims<false, 1>(p, blocks, st);
}

}  // namespace attn
