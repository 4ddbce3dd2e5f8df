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
//     the codes of its operand registers.  Two codes become two fp16 numbers by
//     one mask into the mantissa of 1024 and one exact fused multiply-add
//     (1024 + c - 1032, or (1024 + 16 c) / 16 - 72: the second form saves the
//     shift of every other code).
//     K: pairs of one register are dims n, n + 4 of a word of one token.
//     V: they are the same dim of two tokens (one byte permute joins the
//     half-words of both);
//   * both products are in fp16, which holds q and the probabilities better
//     than bf16 where the range allows: a bf16 q row is held times a power of
//     two that brings its largest element to 2^13 .. 2^14 (exact, but for
//     elements 2^27 times smaller), and a warp keeps a power of two that brings
//     the largest probability times V scale of its tokens to 2^13 .. 2^14;
//   * scales stay out of the operands: K's multiply the FP32 products of each
//     32-dim group, V's multiply the probabilities before these are rounded.
//
// S^T = K Q^T leaves probabilities with tokens along the operand's rows; the
// second product O^T = V^T P^T wants them along its depth: movmatrix
// transposes 8 x 8 blocks in registers.
//
// Split: every (sequence, kv head, block of query rows) is an item of
// ceil(tiles / 8) units (a unit: 8 tiles of 32 tokens, one for each warp).  The
// call's units are one list, cut into equal runs, one for each block of a grid
// that fills the card, so ragged lengths balance; lengths are read on the
// device, so a captured graph serves any lengths.  A block keeps a piece's
// running maximum, sum and O in registers of its 8 warps, joins them through
// shared memory at the end of the piece, and writes the result, or, where the
// item is shared with other blocks, a partial result that a second kernel
// joins in the order of the blocks.
#include <algorithm>

#include "kcommon.cuh"
#include "kv.h"

namespace attn {

constexpr int kTile = 32;   // tokens of a warp's tile
constexpr int kWarps = 8;   // warps of a block
constexpr int kUnit = kTile * kWarps;
constexpr int kExpMin = -100, kExpMax = 100;  // exponents of V's scales told apart

template <int DQK, int DV, int NT>
struct DecShape {
  static constexpr int GK = DQK / 32, GV = DV / 32;
  static constexpr int kRows = 8 * NT;
  // a tile's codes and scales in shared memory
  static constexpr int kKc = kTile * DQK / 2, kVc = kTile * DV / 2;
  static constexpr int kKs = kTile * GK * 2, kVs = kTile * GV * 2;
  static constexpr int kStage = kKc + kVc + kKs + kVs;  // a multiple of 128
  // blocks of an SM: as many as its registers hold
  static constexpr int kBlocks = (NT == 1 && DV <= 128) || DV == 64 ? 2 : 1;
  static constexpr int kStages = kBlocks == 2 || DQK > 192 ? 2 : 3;
  static constexpr int kRing = kWarps * kStages * kStage;
  // the join of the warps: O [row][dim] of 8 warps, and their maxima and sums
  static constexpr int kJoin = kWarps * kRows * (DV + 2) * 4;
  static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + 1024;
};

// ----------------------------------------------------------------- geometry
struct SeqRange {
  int len;      // tokens held
  int lo;       // first tile of the window part
  int n_sink;   // tiles before it that hold sinks
  int tiles;    // all tiles of the sequence that some query sees
};

__device__ __forceinline__ SeqRange seq_range(const DecodeParams& p, int b) {
  SeqRange s;
  s.len = p.seq_lens[b];
  const int cap = p.cols << p.c.page_shift;
  if (s.len < 0 || s.len > cap) {
    if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    s.len = 0;
  }
  // the first query's window starts at len - seqlen_q - window_left
  const int64_t w = p.window_left < 0 ? 0 : (int64_t)s.len - p.seqlen_q - p.window_left;
  s.lo = w > 0 ? (int)(w / kTile) : 0;
  if (s.len == 0) s.lo = 0;
  const int sink_tiles = (int)(((int64_t)p.sinks + kTile - 1) / kTile);
  s.n_sink = min(sink_tiles, s.lo);
  s.tiles = s.n_sink + (s.len + kTile - 1) / kTile - s.lo;
  return s;
}
__device__ __forceinline__ int units_of(const SeqRange& s) { return (s.tiles + kWarps - 1) / kWarps; }
// first token of the v-th tile
__device__ __forceinline__ int tile_token(const SeqRange& s, int v) {
  return (v < s.n_sink ? v : s.lo + v - s.n_sink) * kTile;
}

// ----------------------------------------------------------------- operands
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 codes of a word as fp16 numbers -8 .. 7: pair n is codes n (low half)
// and n + 4 (high half).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&p)[4]) {
  const __half2 low = __half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));       // 1032
  const __half2 sixteenth = __half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00));
  const __half2 high = __half2(__ushort_as_half(0xd480), __ushort_as_half(0xd480));      // -72
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i ? w >> 8 : w;
    uint32_t x, y;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xEA;" : "=r"(x) : "r"(v));  // 1024 + code
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xEA;" : "=r"(y) : "r"(v));  // 1024 + 16 code
    const __half2 f = __hsub2(*reinterpret_cast<__half2*>(&x), low);
    const __half2 g = __hfma2(*reinterpret_cast<__half2*>(&y), sixteenth, high);
    p[2 * i] = *reinterpret_cast<const uint32_t*>(&f);
    p[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&g);
  }
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// N words from shared memory, in the widest loads their alignment allows
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* s, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(s)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2*>(s)[i];
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(s)[i];
  }
}
// scale g of the pairs in w
__device__ __forceinline__ float scale_of(const uint32_t* w, int g) {
  return __uint_as_float((g & 1) ? (w[g >> 1] & 0xffff0000u) : (w[g >> 1] << 16));
}

// Token of row r (of 8) of a tile's block of 8: the four tokens of rows 2c and
// the four of rows 2c + 1 are neighbours, so a warp's V loads (rows 2c of all
// four c) cover 256 bytes in a row, and rows 2q, 2q + 1 lie in different
// halves of the banks, so its K loads do not collide either.
__device__ __forceinline__ int row_token(int r) {
  return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1;
}

// ----------------------------------------------------------------- the kernel
template <bool BF16, int DQK, int DV, int NT>
__global__ void __launch_bounds__(kWarps * 32, DecShape<DQK, DV, NT>::kBlocks) attn_kv_decode_kernel(
    const __grid_constant__ DecodeParams p) {
  using S = DecShape<DQK, DV, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps][S::kStages];
  __shared__ int abort_flag;
  __shared__ long long s_sum[kWarps];
  __shared__ long long s_before;  // units before s_b
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const Abort ab{&abort_flag, p.status, kWaitLimitNs};
  if (tid == 0) {
    abort_flag = 0;
    s_b = p.batch;
    s_before = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < S::kStages; ++s) mbar_init(&full[w][s], 1);
    fence_barrier_init();
  }
  // ---- the list of units, and this block's run of it
  const int per_seq = p.c.heads * p.row_blocks;  // items of a sequence
  long long mine = 0;
  for (int b = tid; b < p.batch; b += kWarps * 32) mine += units_of(seq_range(p, b));
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += s_sum[w];
  all *= per_seq;
  const long long nblk = all < (long long)gridDim.x ? all : (long long)gridDim.x;
  if (blockIdx.x == 0 && tid == 0) *p.total = all;
  if ((long long)blockIdx.x >= nblk) return;
  const long long first = all * blockIdx.x / nblk, last = all * (blockIdx.x + 1) / nblk;
  // the sequence that holds unit `first`
  long long before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kWarps * 32) {
    const int b = b0 + tid;
    const long long n = b < p.batch ? (long long)units_of(seq_range(p, b)) * per_seq : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long off = before;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) off += s_sum[w];
      before += s_sum[w];
    }
    if (first >= off + inc - n && first < off + inc) {
      s_b = b;
      s_before = off + inc - n;
    }
    __syncthreads();
    if (s_b < p.batch) break;
  }
  int b = s_b;
  if (b >= p.batch) return;  // lengths that changed under the call
  long long at = first;              // next unit
  long long seq_first = s_before;    // first unit of sequence b

  uint8_t* ring = smem + warp * (S::kStages * S::kStage);
  uint32_t phase = 0;  // of this warp's stages: fills so far
  bool ok = true;
  while (at < last) {
    SeqRange sr = seq_range(p, b);
    int nu = units_of(sr);
    while (at >= seq_first + (long long)nu * per_seq) {  // sequences without units
      seq_first += (long long)nu * per_seq;
      if (++b >= p.batch) return;
      sr = seq_range(p, b);
      nu = units_of(sr);
    }
    const int item = (int)((at - seq_first) / nu);
    const int kvh = item / p.row_blocks, rb = item - kvh * p.row_blocks;
    const long long item_first = seq_first + (long long)item * nu;
    const int u0 = (int)(at - item_first);
    const int u1 = (int)(last - item_first < nu ? last - item_first : nu);
    at = item_first + u1;
    if (u0 == 0 && tid == 0) {  // where the item lies, for the join
      long long* info = reinterpret_cast<long long*>(p.info);
      info[(int64_t)b * per_seq + item] = item_first;
    }

    // ---- query operand: qf[nt][g][i] holds dims (8c + i, 8c + i + 4) of group g
    uint32_t qf[NT][S::GK][4];
    float xs[NT][2];  // from products to scores in base 2, of columns 2c, 2c + 1
    int jhi[NT][2], jlo[NT][2];  // visible keys of the lane's columns 2c, 2c + 1
    const int row0 = rb * S::kRows;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = row0 + t * 8 + r;
      const int qi = row / p.group, qh = kvh * p.group + row % p.group;
      const uint16_t* src = (const uint16_t*)p.q + b * p.q_b + qi * p.q_t + qh * p.q_h + 8 * c;
      uint4 qv[S::GK];
      uint32_t top = 0;
#pragma unroll
      for (int g = 0; g < S::GK; ++g) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.rows) v = *reinterpret_cast<const uint4*>(src + 32 * g);
        if (BF16) {
          qv[g] = v;
          // magnitudes as bits are ordered
          uint32_t mx = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                 __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
          top = max(top, max(mx & 0xffffu, mx >> 16));
        } else {
          qf[t][g][0] = __byte_perm(v.x, v.z, 0x5410);
          qf[t][g][1] = __byte_perm(v.x, v.z, 0x7632);
          qf[t][g][2] = __byte_perm(v.y, v.w, 0x5410);
          qf[t][g][3] = __byte_perm(v.y, v.w, 0x7632);
        }
      }
      float unit = 1.0f;  // q is held times 1 / unit
      if (BF16) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = min(max((int)(top >> 7) - 127 - 13, -100), 100);  // largest at 2^13 .. 2^14
        unit = __uint_as_float((uint32_t)(127 + ex) << 23);
        const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
        for (int g = 0; g < S::GK; ++g) {
          const uint32_t w[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[i] = inv * __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[t][g][i] = Pack<false>::two(f[i], f[i + 4]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        xs[t][e] = p.scale_log2 * __shfl_sync(0xffffffffu, unit, (2 * c + e) * 4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int cr = row0 + t * 8 + 2 * c + e;
        const int pos = sr.len - p.seqlen_q + cr / p.group;
        jhi[t][e] = cr < p.rows ? pos : -1;
        jlo[t][e] = p.window_left < 0 ? 0 : max(0, pos - p.window_left);
      }
    }
    // every query of the item sees token j if j <= pos_lo and (j >= pos_hi -
    // window_left or j < sinks)
    const int pos_lo = sr.len - p.seqlen_q + row0 / p.group;
    const int pos_hi = sr.len - p.seqlen_q + (min(row0 + S::kRows, p.rows) - 1) / p.group;

    float o[NT][S::GV][2][4];  // O^T: dims 32 g + 4 r + {0,1}, {2,3}; columns 2c, 2c + 1
    float m[NT][2], l[NT][2];
    int vexp = kExpMin;  // O is held times 2^(14 - vexp)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) m[t][e] = -INFINITY, l[t][e] = 0.0f;
#pragma unroll
      for (int g = 0; g < S::GV; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][g][h][e] = 0.0f;
    }

    // ---- this warp's tiles of the piece: v = (u0 + k) * 8 + warp, k < u1 - u0
    const int n = u1 - u0;
    int pages[2] = {-1, -1};  // of tile 32 * (k / 32) + lane; a tile spans one or two pages
    auto issue = [&](int k) {  // whole warp
      if ((k & 31) == 0) {
        const int v = (u0 + k + lane) * kWarps + warp;
        pages[0] = pages[1] = -1;
        if (k + lane < n && v < sr.tiles) {
          const int t0 = tile_token(sr, v);
          const int32_t* row = p.table + (int64_t)b * p.table_stride;
          pages[0] = row[t0 >> p.c.page_shift];
          if (p.c.page_size < kTile && t0 + p.c.page_size < sr.len)
            pages[1] = row[(t0 >> p.c.page_shift) + 1];
          if ((unsigned)pages[0] >= (unsigned)p.c.num_pages ||
              (p.c.page_size < kTile && t0 + p.c.page_size < sr.len &&
               (unsigned)pages[1] >= (unsigned)p.c.num_pages)) {
            if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
          }
        }
      }
      const int v = (u0 + k) * kWarps + warp;
      const int pg0 = __shfl_sync(0xffffffffu, pages[0], k & 31);
      const int pg1 = __shfl_sync(0xffffffffu, pages[1], k & 31);
      if (lane == 0) {
        const int s = (int)(phase % S::kStages);
        uint8_t* st = ring + s * S::kStage;
        const int t0 = v < sr.tiles ? tile_token(sr, v) : 0;
        const int tok = min(p.c.page_size, kTile);  // tokens of a copy
        const bool a0 = (unsigned)pg0 < (unsigned)p.c.num_pages;
        const bool a1 = tok < kTile && (unsigned)pg1 < (unsigned)p.c.num_pages;
        const uint32_t bytes = (uint32_t)tok * (DQK / 2 + DV / 2 + 2 * S::GK + 2 * S::GV);
        mbar_arrive_tx(&full[warp][s], bytes * ((a0 ? 1 : 0) + (a1 ? 1 : 0)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(h ? a1 : a0)) continue;
          const int64_t row = ((int64_t)(h ? pg1 : pg0) * p.c.heads + kvh) * p.c.page_size +
                              (h ? 0 : t0 & (p.c.page_size - 1));
          bulk_load(st + h * tok * (DQK / 2), p.c.k_codes + row * (DQK / 2), tok * (DQK / 2), &full[warp][s]);
          bulk_load(st + S::kKc + h * tok * (DV / 2), p.c.v_codes + row * (DV / 2), tok * (DV / 2), &full[warp][s]);
          bulk_load(st + S::kKc + S::kVc + h * tok * 2 * S::GK, p.c.k_scales + row * S::GK, tok * 2 * S::GK, &full[warp][s]);
          bulk_load(st + S::kKc + S::kVc + S::kKs + h * tok * 2 * S::GV, p.c.v_scales + row * S::GV, tok * 2 * S::GV, &full[warp][s]);
        }
      }
      ++phase;
    };
    int issued = 0;
    uint32_t used = phase;  // stage of the next tile to use
    for (; issued < n && issued < S::kStages; ++issued) issue(issued);

    for (int k = 0; k < n && ok; ++k, ++used) {
      const int s = (int)(used % S::kStages);
      ok = mbar_wait_warp(&full[warp][s], (used / S::kStages) & 1u, ab);
      if (!ok) break;
      const uint8_t* st = ring + s * S::kStage;
      const int v = (u0 + k) * kWarps + warp;
      if (v < sr.tiles) {
        const int t0 = tile_token(sr, v);
        // (columns past the last row hold zeros: what they sum up is not written)
        const bool whole = t0 + kTile - 1 <= pos_lo &&
                           (p.window_left < 0 || t0 >= pos_hi - p.window_left || t0 + kTile <= p.sinks);
        float x[2][NT][4];  // S^T of two blocks of 16 tokens: rows r, r + 8
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int ta = mt * 16 + row_token(r), tb = ta + 8;
          uint32_t ka[S::GK], kb[S::GK], sa[S::GK / 2], sb[S::GK / 2];
          lds_words<S::GK>(st + ta * (DQK / 2) + c * 4 * S::GK, ka);
          lds_words<S::GK>(st + tb * (DQK / 2) + c * 4 * S::GK, kb);
          lds_words<S::GK / 2>(st + S::kKc + S::kVc + ta * 2 * S::GK, sa);
          lds_words<S::GK / 2>(st + S::kKc + S::kVc + tb * 2 * S::GK, sb);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][t][e] = 0.0f;
#pragma unroll
          for (int g = 0; g < S::GK; ++g) {
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[t][e] = 0.0f;
            uint32_t a[4], bk[4];
            codes8(ka[g], a);
            codes8(kb[g], bk);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma16816(acc[t], a[2 * h], bk[2 * h], a[2 * h + 1], bk[2 * h + 1],
                         qf[t][g][2 * h], qf[t][g][2 * h + 1]);
            const float fa = scale_of(sa, g), fb = scale_of(sb, g);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              x[mt][t][0] = fmaf(acc[t][0], fa, x[mt][t][0]);
              x[mt][t][1] = fmaf(acc[t][1], fa, x[mt][t][1]);
              x[mt][t][2] = fmaf(acc[t][2], fb, x[mt][t][2]);
              x[mt][t][3] = fmaf(acc[t][3], fb, x[mt][t][3]);
            }
          }
        }
        // ---- running softmax in base 2
        float alpha[NT][2];
        bool moved = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float& y = x[mt][t][2 * h + e];
                y *= xs[t][e];
                if (!whole) {
                  const int j = t0 + mt * 16 + h * 8 + row_token(r);
                  if (j > jhi[t][e] || (j < jlo[t][e] && j >= p.sinks)) y = -INFINITY;
                }
                mx = fmaxf(mx, y);
              }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[t][e], mx);
            const float ms = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet
            alpha[t][e] = ex2(m[t][e] - ms);
            moved |= mn != m[t][e];
            m[t][e] = mn;
            float sum = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float& y = x[mt][t][2 * h + e];
                y = ex2(y - ms);
                sum += y;
              }
            l[t][e] = fmaf(l[t][e], alpha[t][e], sum);
          }
        // ---- V's scales, and the power of two that fits their largest
        uint32_t vs[2][2][S::GV / 2];  // of tokens r and r + 8 of both blocks
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            lds_words<S::GV / 2>(st + S::kKc + S::kVc + S::kKs +
                                     (mt * 16 + h * 8 + row_token(r)) * 2 * S::GV, vs[mt][h]);
        float kf;
        {
          float mx = 0.0f;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              bool seen = whole;  // a token no query sees: its scales may be anything
#pragma unroll
              for (int t = 0; t < NT; ++t) seen |= x[mt][t][2 * h] != 0.0f || x[mt][t][2 * h + 1] != 0.0f;
              float sm = 0.0f;
#pragma unroll
              for (int g = 0; g < S::GV; ++g) sm = fmaxf(sm, scale_of(vs[mt][h], g));
              if (seen) mx = fmaxf(mx, sm);
            }
          // positive numbers: their bits are ordered
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
          const int e = min(max((int)(top >> 23) - 126, kExpMin), kExpMax);
          if (e > vexp) {
            const float f = __uint_as_float((uint32_t)(127 + max(vexp - e, -126)) << 23);
#pragma unroll
            for (int t = 0; t < NT; ++t) alpha[t][0] *= f, alpha[t][1] *= f;
            moved = true;
            vexp = e;
          }
          kf = __uint_as_float((uint32_t)(127 + 14 - vexp) << 23);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int g = 0; g < S::GV; ++g)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][g][h][e] *= alpha[t][e & 1];
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t v0[S::GV / 2], v1[S::GV / 2], v2[S::GV / 2], v3[S::GV / 2];
          const uint8_t* vb = st + S::kKc + r * 2 * S::GV;
          const int te = mt * 16 + row_token(2 * c), to = mt * 16 + row_token(2 * c + 1);
          lds_words<S::GV / 2>(vb + te * (DV / 2), v0);
          lds_words<S::GV / 2>(vb + to * (DV / 2), v1);
          lds_words<S::GV / 2>(vb + (te + 8) * (DV / 2), v2);
          lds_words<S::GV / 2>(vb + (to + 8) * (DV / 2), v3);
#pragma unroll
          for (int g = 0; g < S::GV; ++g) {
            const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
            const uint32_t z0 = __byte_perm(v0[g >> 1], v1[g >> 1], sel);
            const uint32_t z1 = __byte_perm(v2[g >> 1], v3[g >> 1], sel);
            const float fa = scale_of(vs[mt][0], g) * kf, fb = scale_of(vs[mt][1], g) * kf;
            uint32_t a[4], bq[4];
            codes8(z0, a);
            codes8(z1, bq);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              // a masked token's scale is not looked at: it may be anything
              float p0 = x[mt][t][0] * fa, p1 = x[mt][t][1] * fa;
              float p2 = x[mt][t][2] * fb, p3 = x[mt][t][3] * fb;
              if (!whole) {
                p0 = x[mt][t][0] == 0.0f ? 0.0f : p0;
                p1 = x[mt][t][1] == 0.0f ? 0.0f : p1;
                p2 = x[mt][t][2] == 0.0f ? 0.0f : p2;
                p3 = x[mt][t][3] == 0.0f ? 0.0f : p3;
              }
              const uint32_t b0 = transpose8x8(Pack<false>::two(p0, p1));
              const uint32_t b1 = transpose8x8(Pack<false>::two(p2, p3));
              mma16816(o[t][g][0], a[0], a[1], bq[0], bq[1], b0, b1);
              mma16816(o[t][g][1], a[2], a[3], bq[2], bq[3], b0, b1);
            }
          }
        }
      }
      __syncwarp();
      if (issued < n) issue(issued), ++issued;
    }
    if (!ok) {  // let the copies in flight land before the block ends
      for (; used != phase; ++used)
        mbar_wait_quiet(&full[warp][used % S::kStages], (used / S::kStages) & 1u, ab.limit_ns);
    }
    // ---- join the warps through the (drained) ring
    if (__syncthreads_or(!ok)) return;
    float* jo = reinterpret_cast<float*>(smem);                      // [warp][row][DV]
    float* jm = jo + kWarps * S::kRows * DV;                         // [warp][row]
    float* jl = jm + kWarps * S::kRows;                              // [warp][row]
    const float back = __uint_as_float((uint32_t)(127 - 14 + vexp) << 23);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[t][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = t * 8 + 2 * c + e;
        if (r == 0) jm[warp * S::kRows + row] = m[t][e], jl[warp * S::kRows + row] = sum;
#pragma unroll
        for (int g = 0; g < S::GV; ++g)
          *reinterpret_cast<float4*>(jo + (warp * S::kRows + row) * DV + 32 * g + 4 * r) =
              make_float4(o[t][g][0][e] * back, o[t][g][0][2 + e] * back, o[t][g][1][e] * back,
                          o[t][g][1][2 + e] * back);
      }
    __syncthreads();
    const bool done = u0 == 0 && u1 == nu;  // the whole item: no partial result
    float* part = p.partial + ((int64_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * (S::kRows * (DV + 2));
    for (int i = tid; i < S::kRows * (DV / 4); i += kWarps * 32) {
      const int row = i / (DV / 4), d4 = i % (DV / 4);
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, jm[w * S::kRows + row]);
      const float ms = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(jm[w * S::kRows + row] - ms);
        const float4 y = *reinterpret_cast<const float4*>(jo + (w * S::kRows + row) * DV + d4 * 4);
        sum = fmaf(jl[w * S::kRows + row], f, sum);
        acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y);
        acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
      }
      if (!done) {
        *reinterpret_cast<float4*>(part + row * DV + d4 * 4) = acc;
        if (d4 == 0) part[S::kRows * DV + row] = mx, part[S::kRows * (DV + 1) + row] = sum;
      } else if (row0 + row < p.rows) {
        const int qi = (row0 + row) / p.group, qh = kvh * p.group + (row0 + row) % p.group;
        const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        const int64_t off = b * p.o_b + qi * p.o_t + qh * p.o_h + d4 * 4;
        if (p.o_f32)
          *reinterpret_cast<float4*>((float*)p.o + off) = acc;
        else
          *reinterpret_cast<uint2*>((uint16_t*)p.o + off) =
              make_uint2(Pack<BF16>::two(acc.x, acc.y), Pack<BF16>::two(acc.z, acc.w));
        if (d4 == 0)
          p.lse[((int64_t)b * p.heads_q + qh) * p.seqlen_q + qi] =
              mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
      }
    }
    fence_proxy_async();  // these plain accesses come before the next copies into the ring
    __syncthreads();
  }
}

// ----------------------------------------------------------------- the join
// One block for each item.  Items without a visible key get O = 0 and LSE =
// -inf here; items that one block finished are left alone.  The pieces of the
// others (in the order of the blocks) are shared out over the 8 warps, whose
// sums are then added in warp order.
template <bool BF16, int DV, int ROWS>
__global__ void __launch_bounds__(256) attn_kv_join_kernel(const __grid_constant__ DecodeParams p,
                                                            int blocks) {
  __shared__ float sm_m[8][ROWS], sm_l[8][ROWS];
  extern __shared__ float so[];  // [8][ROWS * DV]
  const int per_seq = p.c.heads * p.row_blocks;
  const int b = (int)(blockIdx.x / per_seq), item = (int)(blockIdx.x % per_seq);
  const int kvh = item / p.row_blocks, row0 = (item - kvh * p.row_blocks) * ROWS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nu = units_of(seq_range(p, b));
  int k0 = 0, np = 0;
  if (nu > 0) {
    const long long all = *p.total;
    const long long nblk = all < blocks ? all : blocks;
    const long long a = reinterpret_cast<const long long*>(p.info)[blockIdx.x], z = a + nu - 1;
    // block k has units [all k / nblk, all (k + 1) / nblk): the block of unit u
    auto block_of = [&](long long u) {
      long long k = u * nblk / all;
      while (k > 0 && all * k / nblk > u) --k;
      while (all * (k + 1) / nblk <= u) ++k;
      return (int)k;
    };
    if (all <= 0 || a < 0 || z >= all) return;
    k0 = block_of(a);
    np = block_of(z) - k0 + 1;
    if (np == 1) return;
  }
  constexpr int kFloats = ROWS * (DV + 2);
  const float* part = p.partial;
  auto piece = [&](int i) { return part + ((int64_t)(k0 + i) * 2 + (i == 0 ? 1 : 0)) * kFloats; };
  for (int row = warp; row < ROWS; row += 8) {  // the row's maximum over all pieces
    float mx = -INFINITY;
    for (int i = lane; i < np; i += 32) mx = fmaxf(mx, piece(i)[ROWS * DV + row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) sm_m[0][row] = mx;
  }
  __syncthreads();
  constexpr int kVec = ROWS * DV / 4 / 32;  // float4 of a lane
  float4 acc[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.0f;  // lane < ROWS: of row `lane`
  for (int i = warp; i < np; i += 8) {
    const float* pc = piece(i);
    float f = 0.0f;
    if (lane < ROWS) {
      const float mx = sm_m[0][lane];
      f = ex2(pc[ROWS * DV + lane] - (mx == -INFINITY ? 0.0f : mx));
      sum = fmaf(pc[ROWS * (DV + 1) + lane], f, sum);
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(pc + (j * 32 + lane) * 4);
      const float fr = __shfl_sync(0xffffffffu, f, (j * 32 + lane) * 4 / DV);
      acc[j].x = fmaf(y.x, fr, acc[j].x), acc[j].y = fmaf(y.y, fr, acc[j].y);
      acc[j].z = fmaf(y.z, fr, acc[j].z), acc[j].w = fmaf(y.w, fr, acc[j].w);
    }
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    *reinterpret_cast<float4*>(so + warp * (ROWS * DV) + (j * 32 + lane) * 4) = acc[j];
  if (lane < ROWS) sm_l[warp][lane] = sum;
  __syncthreads();
  for (int i = tid; i < ROWS * DV / 4; i += 256) {
    const int row = i * 4 / DV, d4 = i % (DV / 4);
    if (row0 + row >= p.rows) continue;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float4 z = *reinterpret_cast<const float4*>(so + w * (ROWS * DV) + i * 4);
      y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
      s += sm_l[w][row];
    }
    const float mx = sm_m[0][row];
    const float inv = mx == -INFINITY ? 0.0f : 1.0f / s;
    y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
    const int qi = (row0 + row) / p.group, qh = kvh * p.group + (row0 + row) % p.group;
    const int64_t off = b * p.o_b + qi * p.o_t + qh * p.o_h + d4 * 4;
    if (p.o_f32)
      *reinterpret_cast<float4*>((float*)p.o + off) = y;
    else
      *reinterpret_cast<uint2*>((uint16_t*)p.o + off) =
          make_uint2(Pack<BF16>::two(y.x, y.y), Pack<BF16>::two(y.z, y.w));
    if (d4 == 0)
      p.lse[((int64_t)b * p.heads_q + qh) * p.seqlen_q + qi] =
          mx == -INFINITY ? -INFINITY : (mx + log2f(s)) * 0.6931471805599453f;
  }
}

// ----------------------------------------------------------------- launches
int decode_col_tiles(int rows, int d_v) {
  (void)d_v;
  return rows > 8 ? 2 : 1;
}

int decode_blocks(const DecodeParams& p, int num_sms) {
  // no more than the longest possible lists of units
  const int64_t cap = ((int64_t)p.cols << p.c.page_shift) / kUnit + 2;
  const int64_t units = cap * p.batch * p.c.heads * p.row_blocks;
  const int per_sm = (decode_col_tiles(p.rows, p.c.d_v) == 1 && p.c.d_v <= 128) || p.c.d_v == 64 ? 2 : 1;
  return (int)std::min<int64_t>((int64_t)num_sms * per_sm, std::max<int64_t>(units, 1));
}

size_t decode_partial_floats(int rows_per_block, int d_v) {
  return (size_t)rows_per_block * (d_v + 2);
}

namespace {

template <typename F>
cudaError_t allow_smem(F* f, int bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <bool BF16, int DQK, int DV, int NT>
cudaError_t dec_launch(const DecodeParams& p, int blocks, cudaStream_t st) {
  using S = DecShape<DQK, DV, NT>;
  auto* main = attn_kv_decode_kernel<BF16, DQK, DV, NT>;
  auto* join = attn_kv_join_kernel<BF16, DV, 8 * NT>;
  const int join_smem = 8 * 8 * NT * DV * 4;
  cudaError_t e = allow_smem(main, S::kSmem);
  if (e == cudaSuccess) e = allow_smem(join, join_smem);
  if (e != cudaSuccess) return e;
  main<<<blocks, kWarps * 32, S::kSmem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  join<<<p.batch * p.c.heads * p.row_blocks, 256, join_smem, st>>>(p, blocks);
  return cudaGetLastError();
}

template <bool BF16, int NT>
cudaError_t dec_dims(const DecodeParams& p, int blocks, cudaStream_t st) {
  if (p.c.d_qk == 64 && p.c.d_v == 64) return dec_launch<BF16, 64, 64, NT>(p, blocks, st);
  if (p.c.d_qk == 128 && p.c.d_v == 128) return dec_launch<BF16, 128, 128, NT>(p, blocks, st);
  if (p.c.d_qk == 192 && p.c.d_v == 128) return dec_launch<BF16, 192, 128, NT>(p, blocks, st);
  if (p.c.d_qk == 256 && p.c.d_v == 256) return dec_launch<BF16, 256, 256, NT>(p, blocks, st);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_kv4_decode(const DecodeParams& p, bool bf16, int blocks, cudaStream_t st) {
  const bool wide = decode_col_tiles(p.rows, p.c.d_v) == 2;
  if (bf16) return wide ? dec_dims<true, 2>(p, blocks, st) : dec_dims<true, 1>(p, blocks, st);
  return wide ? dec_dims<false, 2>(p, blocks, st) : dec_dims<false, 1>(p, blocks, st);
}

}  // namespace attn
