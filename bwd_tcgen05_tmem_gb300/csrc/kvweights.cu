// kvweights.cu -- the attention weights that cached tokens receive.
//
// For every sequence b, kv head h and token j:
//     w[b, h, j] (+)= sum over the queries i and the query heads a of h that see j
//                     of exp(scale q_{i,a} k_j - LSE_{i,a}),
// LSE the log-sum-exp of those queries' attention (what attn_kv_decode returns), so
// each query head hands out 1 in all.
//
// A stream of K's codes (d / 2 + d / 16 bytes a token and head) and of the sums (4
// bytes in, 4 out).  No token depends on another, so there is nothing to join: the
// sequences' units of 128 tokens are one list, cut into equal runs for the blocks of
// a grid that fills the card; lengths are read on the device.  A warp takes 32 of a
// unit's tokens.  Its lanes load the codes of their operand registers straight from
// the cache (its layout gives a lane whole vectors, and a warp whole lines), one
// unit ahead of what they compute with, and the pages one unit ahead of those.  More
// than 16 query rows take turns, 64 at a time, at a tile that is converted once for them.
//
// What bounds it: the instructions of a tile, 411 a warp for 32 tokens of head dim 128
// and 4 query rows (unpacking 80, scales on the sums 50, exponentials and sums 60,
// addresses and pages 60); the schedulers issue in 60 % of the cycles, the ALU pipe is
// busy in 47 %.  16 x 32K tokens of 8 kv heads, head dim 128, one GB300: 84 us,
// 4.0 TB/s of the 6.7 that a copy reaches; head dim 64 56, 192 102, 256 128, 16 query
// rows 102.  128 rows a head (the last 32 queries of 8 prompts of 32K tokens) take 276:
// a block of 8 rows costs 8 products, 16 scalings, 8 exponentials and their sums.
//
// The products are those of attention over the cache: the cache as the 16-row
// operand, 8 query rows as the other, in fp16 (q is held times a power of two that
// brings its row's largest element to 2^13 .. 2^14), the scales of the 32-dim groups on
// the FP32 sums.  Up to 16 query rows the codes are operands as they are, and their
// offset of 8 is the products' start value, as in kvdecode.cu; for more rows, which
// share the operand, 8 is taken off first.
#include <algorithm>

#include "kcommon.cuh"
#include "kv.h"
#include "kvtile.cuh"

namespace attn {

namespace {
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 32;               // tokens of a warp's tile
constexpr int kUnit = kWarps * kTile;   // of a block's unit
constexpr int kManyBlocks = 8;          // blocks of 8 query rows held at a time where there are many

// Blocks an SM.  A lane holds two tiles of codes, the query operand and (of few rows)
// its start values, 128 registers at four blocks of 128 threads, 168 at three, 255 at
// two: where they do not fit, a block more costs more than it hides.  16 x 32K tokens,
// 8 kv heads, one GB300, us, more blocks against two: head dim 64 56 / 66 (four), 128
// with 4 rows 84 / 149 (four), 192 102 / 114 (three), 256 224 / 128 (three / two), 128
// with 16 rows 151 / 102 (three / two), with 128 rows (8 x 32K) 286 / 276 (three / two),
// 9 prompts of 32 query tokens of head dim 64 29 / 35 (four).
constexpr int blocks_of(int dqk, int nb) {
  return dqk == 64 || (dqk == 128 && nb == 1) ? 4 : dqk == 192 && nb == 1 ? 3 : 2;
}
}  // namespace

// The units of a sequence that its call looks at: those that hold first tokens,
// then those from the window's first on (all of them where the weights are set).
struct UnitRange {
  int len, lo, n_sink, units;
};
__device__ __forceinline__ UnitRange unit_range(const WeightsParams& p, int b) {
  UnitRange s;
  s.len = p.seq_lens[b];
  const int most = min(p.cols << p.c.page_shift, p.capacity);
  if (s.len < 0 || s.len > most) {
    if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    s.len = 0;
  }
  const int64_t w = p.window_left < 0 || !p.add ? 0 : (int64_t)s.len - p.seqlen_q - p.window_left;
  s.lo = w > 0 ? (int)(w / kUnit) : 0;
  s.n_sink = min((int)(((int64_t)p.sinks + kUnit - 1) / kUnit), s.lo);
  s.units = s.n_sink + (s.len + kUnit - 1) / kUnit - s.lo;
  return s;
}

// The 8 codes of a word, less 8 each, as pairs of fp16 numbers: pair n holds dims n
// and n + 4.  1024 + code and 64 + code (16 times a code, times 1/16) have their
// codes in the low bits, so that both subtractions are exact.
__device__ __forceinline__ void signed_codes(uint32_t w, uint32_t (&p)[4]) {
  const __half2 o1 = __half2half2(__ushort_as_half(0xe408)), o16 = __half2half2(__ushort_as_half(0xd480));  // -1032, -72
  const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));                                                // 1 / 16
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    uint32_t lo, hi;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xEA;" : "=r"(lo) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xEA;" : "=r"(hi) : "r"(w));
    const __half2 x = __hadd2(*reinterpret_cast<__half2*>(&lo), o1);
    const __half2 y = __hfma2(*reinterpret_cast<__half2*>(&hi), r16, o16);
    p[i] = *reinterpret_cast<const uint32_t*>(&x);
    p[i + 1] = *reinterpret_cast<const uint32_t*>(&y);
    w >>= 8;
  }
}

template <int N>
__device__ __forceinline__ void ldg_words(const uint8_t* s, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(s) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(s) + i);
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  }
}

// What a warp holds of a tile: lane (r, c)'s words of tokens r + 8 i, and the sum so
// far of token r + 8 c.
template <int G>
struct KTile {
  uint32_t k[4][G], s[4][G / 2];
  float old;
};

// NB: blocks of 8 query rows that the lanes hold (1, 2), or that shared memory holds
// while a pass over the tokens is made for every kManyBlocks of them (kManyBlocks).
template <bool BF16, int DQK, int NB>
__global__ void __launch_bounds__(kThreads, blocks_of(DQK, NB)) attn_kv_weights_kernel(
    const __grid_constant__ WeightsParams p) {
  constexpr int G = DQK / 32;
  constexpr bool kMany = NB == kManyBlocks;
  constexpr bool kHold = NB * G <= 8, kHoldLow = NB * G <= 4;  // the query operand, and the start values, stay in registers
  __shared__ uint4 s_q[NB][G][32];            // operand registers of a lane
  __shared__ float s_xs[NB * 8], s_lse[NB * 8];  // from products to base-2 scores; LSE in base 2
  __shared__ float4 s_low[kWarps][kMany || kHoldLow ? 1 : NB][kHoldLow ? 1 : G][4];
  __shared__ long long s_sum[kWarps];
  __shared__ int s_b;
  __shared__ long long s_before;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  // ---- this block's run of the list (b, kv head, unit): units are added up over
  // chunks of kThreads sequences, first for the total, then to find the first one
  long long before = 0, mine0 = 0;
  int mine = 0;
  auto chunk = [&](int b0) {
    mine = b0 + tid < p.batch ? unit_range(p, b0 + tid).units : 0;
    long long j = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, j, o);
      if (lane >= o) j += x;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = j;
    __syncthreads();
    mine0 = before + j - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) mine0 += s_sum[w];
      before += s_sum[w];
    }
  };
  if (tid == 0) s_b = p.batch;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) chunk(b0);
  const long long all = before * p.c.heads;
  const long long each = all / gridDim.x, more = all - each * gridDim.x;
  const long long first = each * blockIdx.x + min((long long)blockIdx.x, more);
  long long left = each + (blockIdx.x < more ? 1 : 0);
  if (left == 0) return;
  if (p.batch > kThreads) before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    if (p.batch > kThreads) chunk(b0);
    const long long f = mine0 * p.c.heads;
    if (first >= f && first < f + (long long)mine * p.c.heads) s_b = b0 + tid, s_before = f;
    if (before * p.c.heads > first) break;
  }
  __syncthreads();
  int b = s_b;
  if (b >= p.batch) return;  // lengths that changed under the call
  UnitRange ur = unit_range(p, b);
  int kvh = (int)((first - s_before) / max(ur.units, 1)), v = (int)((first - s_before) - (long long)kvh * ur.units);

  for (; left > 0;) {
    // ---- a segment: units v .. v + n - 1 of one sequence and kv head
    const int n = (int)min(left, (long long)(ur.units - v));
    const int32_t* row = p.table + (int64_t)b * p.table_stride;
    float* w = p.w + (int64_t)b * p.w_b + (int64_t)kvh * p.w_h;
    const int pos0 = ur.len - p.seqlen_q;  // position of query 0
    // first token of the warp's tile of unit u of the segment
    constexpr int kPast = INT32_MAX - (2 * kTile - 1);  // a tile past any length, on a tile's boundary as all are
    static_assert(kPast % kTile == 0, "its rows in page 0 are read");
    auto token_of = [&](int u) {
      const int x = u + v;
      return u < n ? (x < ur.n_sink ? x : ur.lo + x - ur.n_sink) * kUnit + warp * kTile : kPast;
    };
    // the lane's part of the head's first row in page 0 (pages of a side take less than 2^31 bytes)
    const int64_t row0_of = (int64_t)kvh * p.c.page_size + r;
    const uint8_t* const my_codes = p.c.k_codes + row0_of * (DQK / 2) + c * 4 * G;
    const uint8_t* const my_scales = reinterpret_cast<const uint8_t*>(p.c.k_scales) + row0_of * (2 * G);
    const uint32_t rows_of = (uint32_t)(p.c.heads * p.c.page_size), page_codes = rows_of * (DQK / 2), page_scales = rows_of * (2 * G);
    for (int row0 = 0; row0 < p.rows; row0 += NB * 8) {
      const int nb = min(NB, (p.rows - row0 + 7) / 8);
      // ---- the query rows
      __syncthreads();
      for (int i = warp; i < nb; i += kWarps) {
        const int qrow = row0 + i * 8 + r;
        const int qi = (int)p.by_group.div(qrow), qh = kvh * p.group + qrow - qi * p.group;
        const uint16_t* src = (const uint16_t*)p.q + b * p.q_b + qi * p.q_t + qh * p.q_h + 8 * c;
        uint4 qv[G];
        uint32_t top = 0;  // largest magnitude: as bits they are ordered
#pragma unroll
        for (int g = 0; g < G; ++g) {
          qv[g] = make_uint4(0u, 0u, 0u, 0u);
          if (qrow < p.rows) qv[g] = *reinterpret_cast<const uint4*>(src + 32 * g);
          const uint32_t mx = __vmaxu2(__vmaxu2(qv[g].x & 0x7fff7fffu, qv[g].y & 0x7fff7fffu),
                                       __vmaxu2(qv[g].z & 0x7fff7fffu, qv[g].w & 0x7fff7fffu));
          top = max(top, max(mx & 0xffffu, mx >> 16));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t tf = __float_as_uint(Pack<BF16>::to_f((uint16_t)top));
        const int ex = min(max((int)(tf >> 23) - 127 - 13, -100), 100);  // largest at 2^13 .. 2^14
        const float inv = pow2(-ex);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t x[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f[e] = Pack<BF16>::to_f((uint16_t)(x[e >> 1] >> (16 * (e & 1)))) * (kMany || !(e & 1) ? inv : inv * KCodes<DQK>::kOdd);
          s_q[i][g][lane] = make_uint4(Pack<false>::two(f[0], f[4]), Pack<false>::two(f[1], f[5]),
                                       Pack<false>::two(f[2], f[6]), Pack<false>::two(f[3], f[7]));
        }
        if (c == 0) {
          s_xs[i * 8 + r] = p.scale_log2 * (kMany ? 1.0f : KCodes<DQK>::kUnit) * pow2(ex);
          const float lse = qrow < p.rows ? p.lse[((int64_t)b * p.heads_q + qh) * p.seqlen_q + qi] : 0.0f;
          s_lse[i * 8 + r] = lse * 1.4426950408889634f;
        }
      }
      __syncthreads();
      uint4 qf[kHold ? NB : 1][G];
      float4 low[kHoldLow ? NB : 1][G];  // what the codes' offset adds up to
      float xs[kMany ? 1 : NB][2], ls[kMany ? 1 : NB][2];
      if constexpr (!kMany) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
#pragma unroll
          for (int g = 0; g < G; ++g)
            if (kHold) qf[i][g] = s_q[i][g][lane];
#pragma unroll
          for (int e = 0; e < 2; ++e) xs[i][e] = s_xs[i * 8 + 2 * c + e], ls[i][e] = s_lse[i * 8 + 2 * c + e];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            constexpr uint32_t even = KCodes<DQK>::kEven8, odd = KCodes<DQK>::kOdd8;
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const uint4 q = s_q[i][g][lane];
            mma16816(x, even, even, odd, odd, q.x, q.y);
            mma16816(x, even, even, odd, odd, q.z, q.w);
            if (kHoldLow)
              low[i][g] = make_float4(x[0], x[1], x[2], x[3]);
            else if (r == 0)
              s_low[warp][i][g][c] = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
        __syncwarp();
      }
      // every query of these rows sees tokens whole_lo .. pos_lo; none sees one above
      // pos_hi, or below any_lo but the first `sinks`
      const int pos_lo = pos0 + (int)p.by_group.div(row0);
      const int pos_hi = pos0 + (int)p.by_group.div(min(row0 + NB * 8, p.rows) - 1);
      const int any_lo = p.window_left < 0 ? 0 : max(0, pos_lo - p.window_left);
      const int whole_lo = p.window_left < 0 ? 0 : max(0, pos_hi - p.window_left);
      // sums of other rows, or of earlier calls, are added to
      const bool later = row0 > 0;
      const int set_from = later ? INT32_MAX : p.add ? max(pos0, 0) : 0;

      // Pages of the two halves (16 tokens) of the tile at token t0.  A half that no query
      // sees a token of is not looked at, and page 0 is read in its place; of one that some do
      // all 16 rows are read.  Whatever hidden rows hold, their weights are 0.
      const int seen_end = min(ur.len, pos_hi + 1);
      int page[2];
      auto pages_of = [&](int t0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = t0 + 16 * h;
          page[h] = 0;
          if (t < seen_end && (t + 15 >= any_lo || t < p.sinks)) page[h] = __ldg(row + (t >> p.c.page_shift));
        }
      };
      auto load = [&](int t0, KTile<G>& z) {  // (of the pages looked up last)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pg = (uint32_t)page[h];
          if (pg >= (uint32_t)p.c.num_pages) {
            if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
            pg = 0;
          }
          const uint32_t in_page = (uint32_t)(t0 + 16 * h) & (uint32_t)(p.c.page_size - 1);
          const uint8_t* codes = my_codes + (uint64_t)pg * page_codes + in_page * (DQK / 2);
          const uint8_t* scales = my_scales + (uint64_t)pg * page_scales + in_page * (2 * G);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ldg_words<G>(codes + i * 8 * (DQK / 2), z.k[2 * h + i]);
            ldg_words<G / 2>(scales + i * 8 * (2 * G), z.s[2 * h + i]);
          }
        }
        const int t = t0 + 8 * c + r;
        z.old = 0.0f;
        if (t < ur.len && t < set_from) z.old = w[t];
      };
      const bool full_cols = row0 + nb * 8 <= p.rows;
      bool col[kMany ? 1 : NB][2];
      if constexpr (!kMany) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) col[i][e] = row0 + i * 8 + 2 * c + e < p.rows;
      }
      // 16 tokens times 8 query rows: their products with the scales on them (a lane has tokens
      // r, r + 8 in y[0 .. 1], y[2 .. 3], rows 2c, 2c + 1), and what those add to the tokens' sums
      auto products = [&](const uint32_t (&ka)[G][4], const uint32_t (&kb)[G][4], const uint32_t (&sa)[G / 2],
                          const uint32_t (&sb)[G / 2], const uint4 (&q)[G], const float4* start, float (&y)[4]) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float fa = scale_of(sa, g), fb = scale_of(sb, g);
          const float4 l = kMany ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : start[g];
          const float first[4] = {l.x, l.y, l.z, l.w};
          float acc[4];
          mma16816(acc, ka[g][0], kb[g][0], ka[g][1], kb[g][1], q[g].x, q[g].y, first);
          mma16816(acc, ka[g][2], kb[g][2], ka[g][3], kb[g][3], q[g].z, q[g].w);
          y[0] = g ? fmaf(acc[0], fa, y[0]) : acc[0] * fa;
          y[1] = g ? fmaf(acc[1], fa, y[1]) : acc[1] * fa;
          y[2] = g ? fmaf(acc[2], fb, y[2]) : acc[2] * fb;
          y[3] = g ? fmaf(acc[3], fb, y[3]) : acc[3] * fb;
        }
      };
      // (i: block of 8 rows; see0, see1: whether 2c, 2c + 1 of it are query rows; m: half of the tile)
      auto add = [&](float (&y)[4], int t0, int m, bool whole, int i, float xs0, float xs1, float ls0, float ls1, bool see0,
                     bool see1, float (&sum)[4]) {
        y[0] = ex2(fmaf(y[0], xs0, -ls0));
        y[1] = ex2(fmaf(y[1], xs1, -ls1));
        y[2] = ex2(fmaf(y[2], xs0, -ls0));
        y[3] = ex2(fmaf(y[3], xs1, -ls1));
        if (!whole) {  // (whatever a hidden token's scale is, its weight is 0)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int pos = pos0 + (int)p.by_group.div(row0 + i * 8 + 2 * c + e);
            const int lo = p.window_left < 0 ? 0 : pos - p.window_left;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int t = t0 + 16 * m + 8 * h + r;
              if (t > pos || (t < lo && t >= p.sinks)) y[2 * h + e] = 0.0f;
            }
          }
        }
        if (!full_cols) {  // columns past the last row
          y[0] = see0 ? y[0] : 0.0f, y[2] = see0 ? y[2] : 0.0f;
          y[1] = see1 ? y[1] : 0.0f, y[3] = see1 ? y[3] : 0.0f;
        }
        sum[2 * m] += y[0] + y[1];
        sum[2 * m + 1] += y[2] + y[3];
      };
      auto is_whole = [&](int t0) { return t0 + kTile - 1 <= pos_lo && (t0 >= whole_lo || t0 + kTile <= p.sinks); };
      auto store = [&](int t0, const float (&sum)[4], float old) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = sum[i];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          if (c == i) total = x;
        }
        const int t = t0 + 8 * c + r;
        if (t < ur.len) w[t] = t < set_from ? old + total : total;
      };

      if constexpr (kMany) {
        // The tile's operands serve all row blocks, so they are made first, and the next
        // tile comes into the codes' registers; both halves of the tile go through a row block together.
        KTile<G> z;
        int here = token_of(0);
        pages_of(here);
        load(here, z);
        pages_of(token_of(1));
        for (int u = 0; u < n; ++u) {
          uint32_t k[4][G][4], s[4][G / 2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int g = 0; g < G; ++g) signed_codes(z.k[i][g], k[i][g]);
#pragma unroll
            for (int g = 0; g < G / 2; ++g) s[i][g] = z.s[i][g];
          }
          const float old = z.old;
          const int t0 = here;
          here = token_of(u + 1);
          load(here, z);
          pages_of(token_of(u + 2));
          if (t0 >= ur.len) continue;
          const bool whole = is_whole(t0);
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int i = 0; i < nb; ++i) {
            const float2 x = *reinterpret_cast<const float2*>(s_xs + i * 8 + 2 * c);
            const float2 l = *reinterpret_cast<const float2*>(s_lse + i * 8 + 2 * c);
            const bool see0 = row0 + i * 8 + 2 * c < p.rows, see1 = row0 + i * 8 + 2 * c + 1 < p.rows;
            uint4 qi[G];
#pragma unroll
            for (int g = 0; g < G; ++g) qi[g] = s_q[i][g][lane];
            float y[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
              products(k[2 * m], k[2 * m + 1], s[2 * m], s[2 * m + 1], qi, nullptr, y[m]);
#pragma unroll
            for (int m = 0; m < 2; ++m) add(y[m], t0, m, whole, i, x.x, x.y, l.x, l.y, see0, see1, sum);
          }
          store(t0, sum, old);
        }
      } else {
        auto tile = [&](int t0, const KTile<G>& z) {
          if (t0 >= ur.len) return;
          const bool whole = is_whole(t0);
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t ka[G][4], kb[G][4];
#pragma unroll
            for (int g = 0; g < G; ++g) {
              KCodes<DQK>::of(z.k[2 * m][g], ka[g]);
              KCodes<DQK>::of(z.k[2 * m + 1][g], kb[g]);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              uint4 qi[G];
              float4 start[G];
#pragma unroll
              for (int g = 0; g < G; ++g) {
                qi[g] = kHold ? qf[kHold ? i : 0][g] : s_q[i][g][lane];
                start[g] = kHoldLow ? low[kHoldLow ? i : 0][g] : s_low[warp][kHoldLow ? 0 : i][kHoldLow ? 0 : g][c];
              }
              float y[4];
              products(ka, kb, z.s[2 * m], z.s[2 * m + 1], qi, start, y);
              add(y, t0, m, whole, i, xs[i][0], xs[i][1], ls[i][0], ls[i][1], col[i][0], col[i][1], sum);
            }
          }
          store(t0, sum, z.old);
        };
        // two tiles in registers: one is computed with while the other one comes
        KTile<G> ping, pong;
        int here = token_of(0), next = token_of(1);  // (past the segment: past any length)
        pages_of(here);
        load(here, ping);
        pages_of(next);
        for (int u = 0; u < n; u += 2) {
          load(next, pong);
          const int after = token_of(u + 2);
          pages_of(after);
          tile(here, ping);
          load(after, ping);
          here = after;
          const int last = next;
          next = token_of(u + 3);
          pages_of(next);
          tile(last, pong);
        }
      }
    }
    left -= n;
    v += n;
    if (left > 0 && v == ur.units) {
      v = 0;
      if (++kvh == p.c.heads) {
        kvh = 0;
        do ++b;
        while (b < p.batch && (ur = unit_range(p, b)).units == 0);
        if (b >= p.batch) return;
      }
    }
  }
}

// No query at all: what is set is 0.
__global__ void __launch_bounds__(256) attn_kv_weights_clear_kernel(const __grid_constant__ WeightsParams p) {
  const int64_t all = (int64_t)p.batch * p.c.heads;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int b = (int)(i / p.c.heads), h = (int)(i - (int64_t)b * p.c.heads), n = unit_range(p, b).len;
    float* w = p.w + b * p.w_b + h * p.w_h;
    for (int t = threadIdx.x; t < n; t += 256) w[t] = 0.0f;
  }
}

namespace {
template <bool BF16, int DQK, int NB>
cudaError_t weights_launch(const WeightsParams& p, int num_sms, cudaStream_t st) {
  // no more blocks than the longest possible list has units
  const int64_t units = (((int64_t)p.cols << p.c.page_shift) + kUnit - 1) / kUnit * p.batch * p.c.heads;
  const int64_t most = (int64_t)num_sms * blocks_of(DQK, NB);
  const unsigned blocks = (unsigned)std::max<int64_t>(std::min(most, units), 1);
  attn_kv_weights_kernel<BF16, DQK, NB><<<blocks, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}
template <bool BF16, int DQK>
cudaError_t weights_dims(const WeightsParams& p, int num_sms, cudaStream_t st) {
  if (p.rows <= 8) return weights_launch<BF16, DQK, 1>(p, num_sms, st);
  if (p.rows <= 16) return weights_launch<BF16, DQK, 2>(p, num_sms, st);
  return weights_launch<BF16, DQK, kManyBlocks>(p, num_sms, st);
}
template <bool BF16>
cudaError_t weights_type(const WeightsParams& p, int num_sms, cudaStream_t st) {
  switch (p.c.d_qk) {
    case 64: return weights_dims<BF16, 64>(p, num_sms, st);
    case 128: return weights_dims<BF16, 128>(p, num_sms, st);
    case 192: return weights_dims<BF16, 192>(p, num_sms, st);
    case 256: return weights_dims<BF16, 256>(p, num_sms, st);
    default: return cudaErrorNotSupported;
  }
}
}  // namespace

cudaError_t launch_kv4_weights(const WeightsParams& p, bool bf16, int num_sms, cudaStream_t st) {
  if (p.rows == 0) {
    const unsigned blocks = (unsigned)std::min<int64_t>((int64_t)p.batch * p.c.heads, 8 * num_sms);
    attn_kv_weights_clear_kernel<<<blocks, 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  return bf16 ? weights_type<true>(p, num_sms, st) : weights_type<false>(p, num_sms, st);
}

}  // namespace attn
