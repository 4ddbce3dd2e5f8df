// kvshared.cu -- attention of a few query tokens over the 4-bit cache for batches
// whose requests share their first tokens.
//
// The keys of a request are two disjoint sets: the group's prefix, and its own.
//   * prefix: the query rows of ALL of a group's requests (members * seqlen_q * query
//     heads of a kv head) against one copy of the prefix: a matrix-shaped problem, on
//     tcgen05.  O, the running maximum m and sum l of every row go to the workspace;
//   * own tokens: attn_kv_decode_kernel, from each sequence's first own token on;
//   * join: O = sum of the parts' weights, by their maxima and sums, and the LSE.
// attn_kv_decode alone reads and converts the prefix once for every request and every
// 16 query rows; here every 256 rows share a conversion.
//
// The prefix kernel.  One block an SM, 20 warps:
//   warps 0..7   softmax: two groups of 128 threads, one TMEM lane (query row) each;
//   warps 8..11  K's codes to the fp16 operand, warps 12..15 V's: two of the four take the
//                even tiles, two the odd ones, half of the tile's tokens each, four lanes a
//                row, the next tile's codes on their way in registers; no warp waits for
//                another one;
//   warps 16, 19 issue S = Q K^T, one for each softmax group, warp 17 O += P V;
//   warp 18      looks up where the tokens of the tiles to come lie, and asks for them in L2.
// A block's run of work is a stretch of the list (group, kv head, 256 query rows, tile
// of 64 keys), cut into equal runs.  With more than 128 rows the two softmax groups have
// 128 rows each and share every converted tile; with fewer they take turns at the tiles
// for the same rows, each with its own O (two parts for the join).  Each group reads its
// scores into registers at once, so that the next ones are computed while it works, and
// has two P buffers in TMEM.  At head dim 256
// O fills half of TMEM: one softmax group, 128 rows.
//
// Numbers: code - 8 is exact in fp16 and so is its product with a bf16 scale (4 + 8
// bits), times a power of two that makes the largest scale of half a tile 2^11 .. 2^12.
// K's comes back with the scores; V's goes into the probabilities, in units that the row's
// largest probability times V's largest scale of half a tile sets: O's reference follows it
// when it grows, the sum's follows the largest probability alone.
// q is held as in kvdecode.cu.  Probabilities are FP32 in the sum and rounded to fp16 for
// the second product, times 2^11: a reference moves when what it follows passes it by 2^4, so
// they stay below 2^15, and those 2^-35 below the largest are still told from 0.
//
// What bounds it: instructions (60 % issue, the ALU pipe at 45 %, the tensor pipe at 44 %)
// and the wait of each softmax row for its scores.  256 requests of 4 rows over 32K tokens, 8 kv
// heads of 128, one GB300: 182 us, the prefix kernel 142 of them (0.97 PFLOP/s); plan 4,
// own tokens 20, the two joins 14.  64 requests over 8K tokens 64.5 us.  The first
// instruction cache is what K's and V's conversion in one loop, and loops that are not
// unrolled, are for: apart they took 233 us.  Tiles of 128 keys 250, four softmax groups of
// half a row 269.
//
// In a row of 8 dims the operand's order is 0 4 1 5 2 6 3 7 (a mask of a word of codes
// makes pairs n, n + 4): Q is stored the same way, O's columns are put back at the end.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kcommon.cuh"
#include "kv.h"
#include "kvtile.cuh"

namespace attn {

namespace {

constexpr int KT = 64;  // keys of a tile: prefixes are taken in whole ones, the rest is the requests' own
constexpr float kLag = 4.0f, kBias = 15.0f - kLag;  // a row's reference may lag its maximum; probabilities are held times 2^kBias
constexpr int kXRing = 16;  // factors of tiles on their way to the softmax groups
// Parts of an item on average above which a block joins a row: 256 requests over 32K take
// 185 us with 12 and with 40 (one build), 205 with 3 (few parts, many rows); 4 samples of 1K tokens 31 with
// 12, 42 with 40.
constexpr int kJoinParts = 12;
constexpr int kRowRing = 8;  // tiles that are looked up ahead
constexpr int kThreads = 640;
// Registers of a thread: 96 at the launch; the softmax groups, which hold a row of
// scores, take what the issuing warps give up (2 * 112 + 2 * 96 + 56 <= 5 * 96).
constexpr int kSoftmaxRegs = 112, kIssueRegs = 56;

template <int DQK, int DV>
struct ShShape {
  static constexpr bool kWide = DV > 128;
  static constexpr int kSlots = kWide ? 1 : 2;     // softmax groups
  static constexpr int kRT = 128 * kSlots;         // query rows of an item
  static constexpr int kKSlot = KT * 128;          // 64 dims of a tile
  static constexpr int kKTile = kKSlot * (DQK / 64), kVTile = kKSlot * (DV / 64);
  static constexpr int kQTile = kSlotBytes * (DQK / 64);
  static constexpr int kKS = kWide ? 2 : DQK == 192 ? 3 : 4, kVS = kKS;  // stages
  static constexpr int kSmem = kSlots * kQTile + kKS * kKTile + kVS * kVTile + 1024;
  static constexpr int kTmemO = 256;
};

}  // namespace

// ----------------------------------------------------------------- the list of work
// What the first kernel finds out about a group.
struct ShGroup {
  int unit0;        // units (a tile of an item) of the groups before it
  int tokens;       // of the prefix that its requests share, a multiple of KT
  int request;      // one that shares it (its table row is read)
  int first, members;
};

__device__ __forceinline__ int sh_row_tiles(const SharedParams& p, const ShGroup& g) {
  return (int)(((long long)g.members * p.rows + p.row_tile - 1) >> (p.row_tile == 256 ? 8 : 7));
}
__device__ __forceinline__ int sh_key_tiles(const SharedParams& p, const ShGroup& g) {
  return g.tokens / KT;
}

// Threads of the first kernel; the second where there are no more requests and groups (its
// barriers are cheaper: 4 samples of 1K tokens 30.8 us, 31.6 with 1024).
constexpr int kPlanThreads = 1024, kPlanFew = 256;
// One block: which requests share what.
__global__ void __launch_bounds__(kPlanThreads) attn_kv_shared_plan_kernel(const __grid_constant__ SharedParams p) {
  __shared__ int s_bad;
  __shared__ int s_items, s_sum[32];
  ShGroup* groups = (ShGroup*)p.group_info;
  const int T = (int)blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cap = (int64_t)p.cols << p.c.page_shift;
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) s_bad = 0, s_items = 0;
  __syncthreads();
  bool bad = false;
  for (int g = tid; g <= p.groups; g += T) {
    const int at = p.group_starts[g];
    bad |= at < 0 || at > p.batch || (g > 0 && p.group_starts[g - 1] > at);
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const bool none = s_bad != 0;  // groups that are not in order share nothing
  bad = none;
  for (int g = tid; g < p.groups; g += T) {
    const int n = p.shared_lens[g];
    const bool ok = n >= 0 && n <= cap;
    bad |= !ok;
    ShGroup x;
    x.unit0 = 0;
    x.tokens = none || !ok ? 0 : n / KT * KT;
    x.request = INT32_MAX;
    x.first = none ? 0 : p.group_starts[g];
    x.members = 0;
    groups[g] = x;
  }
  if (bad && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
  __syncthreads();
  // the group of request b, or -1 if it does not share its prefix
  auto group_of = [&](int b) {
    if (none || p.groups == 0 || b < p.group_starts[0] || b >= p.group_starts[p.groups]) return -1;
    int lo = 0, hi = p.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.group_starts[mid] <= b) lo = mid; else hi = mid;
    }
    const int n = groups[lo].tokens, len = p.seq_lens[b];
    return n > 0 && len <= cap && len >= n + p.seqlen_q ? lo : -1;
  };
  for (int b = tid; b < p.batch; b += T) {
    const int g = group_of(b);
    p.group_of[b] = g;
    if (g >= 0) {
      atomicMin(&groups[g].request, b);
      atomicAdd(&groups[g].members, 1);
    }
  }
  __syncthreads();
  // a prefix that one request has alone is that request's own
  for (int b = tid; b < p.batch; b += T) {
    int g = p.group_of[b];
    if (g >= 0 && __ldcg(&groups[g].members) < 2) p.group_of[b] = g = -1;
    p.starts[b] = g >= 0 ? groups[g].tokens : 0;
  }
  __syncthreads();
  int before = 0, items = 0;  // (the host has refused calls whose units could pass 2^31)
  for (int g0 = 0; g0 < p.groups; g0 += T) {
    const int g = g0 + tid;
    ShGroup x;
    int units = 0;
    if (g < p.groups) {
      x.first = groups[g].first;
      x.request = __ldcg(&groups[g].request);  // (atomics are done in L2)
      x.tokens = __ldcg(&groups[g].members) < 2 ? 0 : groups[g].tokens;
      x.members = none ? 0 : p.group_starts[g + 1] - x.first;
      if (x.tokens) {
        const int n = p.c.heads * sh_row_tiles(p, x);
        items += n;
        units = n * sh_key_tiles(p, x);
      }
    }
    int j = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, j, o);
      if (lane >= o) j += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = j;
    __syncthreads();
    x.unit0 = before + j - units;
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) x.unit0 += s_sum[w];
      before += s_sum[w];
    }
    if (g < p.groups) groups[g] = x;
  }
  if (items) atomicAdd(&s_items, items);
  __syncthreads();
  if (tid == 0) p.total_units[0] = before, p.total_units[1] = s_items;
}

// Starts kernel k while the one before it on the stream still runs (it waits itself).
template <typename... A>
cudaError_t launch_early(void (*k)(A...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// The list is cut into `runs` equal runs.
struct ShRuns {
  int total, each, more, runs;
  __device__ __forceinline__ ShRuns(int total_, int most) {
    total = total_;
    runs = min(most, total);
    each = runs ? total / runs : 0;
    more = total - each * runs;
  }
  __device__ __forceinline__ int start(int k) const { return each * k + min(k, more); }
  __device__ __forceinline__ int of(int u) const {
    const int big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

// The next piece of a run: tiles kt .. kt_end - 1 of one item.
struct ShPiece {
  int u, end;  // what is left of the run
  int g;
  ShGroup info;
  int head, row_tile, kt, kt_end, key_tiles;
  __device__ __forceinline__ void begin(const SharedParams& p, int u0, int u1) {
    u = u0;
    end = u1;
    const ShGroup* groups = (const ShGroup*)p.group_info;
    int lo = 0, hi = p.groups;
    while (hi - lo > 1) {  // the last group whose first unit is <= u
      const int mid = (lo + hi) >> 1;
      if (groups[mid].unit0 <= u) lo = mid; else hi = mid;
    }
    g = lo;
    info = groups[lo];
  }
  __device__ __forceinline__ bool next(const SharedParams& p) {
    if (u >= end) return false;
    const ShGroup* groups = (const ShGroup*)p.group_info;
    for (;;) {
      key_tiles = sh_key_tiles(p, info);
      const int row_tiles = sh_row_tiles(p, info);
      const int n = info.tokens ? p.c.heads * row_tiles * key_tiles : 0, at = u - info.unit0;
      if (at >= n) {  // (groups without units are passed by)
        info = groups[++g];
        continue;
      }
      const int item = at / key_tiles;
      kt = at - item * key_tiles;
      head = item / row_tiles;
      row_tile = item - head * row_tiles;
      kt_end = min(key_tiles, kt + (end - u));
      u += kt_end - kt;
      return true;
    }
  }
  // row tiles of 128 rows that hold a row
  __device__ __forceinline__ int row_slots(const SharedParams& p) const {
    return (int)min((long long)p.row_tile, (long long)info.members * p.rows - (long long)row_tile * p.row_tile) > 128 ? 2 : 1;
  }
};

// ----------------------------------------------------------------- operands
// The 8 codes of a word, less 8 each, as pairs n, n + 4 of fp16 numbers, times s:
// 1024 + code and 64 + code have the code in their low bits.
__device__ __forceinline__ uint4 scaled_codes(uint32_t w, __half2 s) {
  const __half2 o1 = __half2half2(__ushort_as_half(0xe408)), o16 = __half2half2(__ushort_as_half(0xd480));  // -1032, -72
  const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));                                                // 1 / 16
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    uint32_t lo, hi;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xEA;" : "=r"(lo) : "r"(w));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xEA;" : "=r"(hi) : "r"(w));
    const __half2 x = __hmul2(__hadd2(*reinterpret_cast<__half2*>(&lo), o1), s);
    const __half2 y = __hmul2(__hfma2(*reinterpret_cast<__half2*>(&hi), r16, o16), s);
    p[i] = *reinterpret_cast<const uint32_t*>(&x);
    p[i + 1] = *reinterpret_cast<const uint32_t*>(&y);
    w >>= 8;
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

constexpr int kExpLow = -110;  // exponents of scales from there on are told apart

struct ShBars {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t s_full[2], s_free[2], p_full[2][2], o_done[2][2];  // of a softmax group's S, and its P buffers
  uint64_t q_full, q_empty, x_full[kXRing], rows_full[kRowRing], rows_empty[kRowRing], drain[3];
};

template <int N>
__device__ __forceinline__ void row_words(const uint8_t* s, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(s) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(s) + i);
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  }
}

// Where a tile's tokens lie: the cache's rows of each 16 of them (-1: none).
struct ShRows {
  long long row[4];
};

// One side of a tile in a lane: the words of its quarter (4 G bytes, G groups of 32 dims)
// of the rows 8 i + row8, and of those rows' scales the groups c, c + 4.  K has GK
// groups, V GV.
template <int GK, int GV, int SETS>
struct ShSide {
  static constexpr int GM = GK > GV ? GK : GV, kOwn = (GM + 3) / 4;
  int G;
  uint32_t w[SETS][GM];
  uint32_t s[SETS][kOwn];
  __half2 h[SETS][kOwn];

  // (Where there are no tokens row 0 is read, and counts with scales of 0.)
  __device__ __forceinline__ void load_scales(const uint16_t* scales, const long long* rows, int row8, int c) {
    const uint16_t* const mine = scales + row8 * G + min(c, G - 1);
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      const long long at = rows[i >> 1];
      const uint16_t* src = mine + max(at, 0ll) * G + (i & 1) * 8 * G;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        s[i][j] = (GK == GV && GM % 4 == 0) || c + 4 * j < G ? __ldg(src + 4 * j) : 0u;
        if (at < 0) s[i][j] = 0u;
      }
    }
  }
  __device__ __forceinline__ void load_codes(const uint8_t* codes, const long long* rows, int row8, int c) {
    const uint8_t* const mine = codes + row8 * (16 * G) + c * 4 * G;
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      const uint8_t* src = mine + max(rows[i >> 1], 0ll) * (16 * G) + (i & 1) * 8 * (16 * G);
      if constexpr (GK == GV) {
        row_words<GM>(src, w[i]);
      } else {
#pragma unroll
        for (int j = 0; j < GM; j += 2)
          if (j < min(GK, GV) || j < G) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + j / 2);
            w[i][j] = v.x, w[i][j + 1] = v.y;
          }
      }
    }
  }
  // the largest finite scale's bits
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const uint32_t x = s[i][j] & 0x7fffu;
        if (x < 0x7f80u) m = max(m, x);
      }
    return __reduce_max_sync(0xffffffffu, m);
  }
  __device__ __forceinline__ void halves(float f) {
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
      for (int j = 0; j < kOwn; ++j) h[i][j] = __float2half2_rn(__uint_as_float(s[i][j] << 16) * f);
  }
  // V's half-words of two quarters of a group side by side, as K's words hold them
  __device__ __forceinline__ void pair_halves() {
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      uint32_t y[GV];
#pragma unroll
      for (int g = 0; g < GV; ++g) y[g] = __byte_perm(w[i][g >> 1], w[i][(GV + g) >> 1], (g & 1) ? 0x7632 : 0x5410);
#pragma unroll
      for (int g = 0; g < GV; ++g) w[i][g] = y[g];
    }
  }
  // dst: row row8 of the warp's tokens in the operand (rows of 128 bytes, swizzled).
  // (Lanes 8 p .. + 7 hold rows p and p + 4, whose chunks lie in different banks.)
  __device__ __forceinline__ void store(uint32_t dst, int row8, int c) const {
    const int quad = (threadIdx.x & 31) & ~3;
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        if (g >= min(GK, GV) && g >= G) break;
        const uint32_t sb = __shfl_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&h[i][g >> 2]), quad | (g & 3));
        const uint4 y = scaled_codes(w[i][g], *reinterpret_cast<const __half2*>(&sb));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         dst + (g >> 1) * (KT * 128) + i * 1024 + ((((g & 1) * 4 + c) ^ row8) << 4)),
                     "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                     : "memory");
      }
  }
};

// One of the four warps that turn a side's codes into its operand.  (K's and V's share this
// code, and loops that run rarely are not unrolled: what an SM's warps run in a tile has
// to fit its first instruction cache.  With two copies 256 requests over 32K tokens took
// 233 us, 192 us with one.)
template <int DQK, int DV>
__device__ __forceinline__ void sh_convert(const uint8_t* codes, const uint16_t* scales, bool is_k, uint8_t* operand,
                                           uint64_t* full, uint64_t* empty, ShBars& bars, float (*x_exp)[2],
                                           const ShRows* rows, int n, int dropped, const Abort& ab) {
  constexpr int kStages = ShShape<DQK, DV>::kKS;
  static_assert(kStages == ShShape<DQK, DV>::kVS, "one code for both sides");
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, half = warp & 1;
  const int c = lane & 3, row8 = (lane >> 3) + ((lane >> 2) & 1) * 4;
  const uint32_t dst = smem_u32(operand) + (half * 32 + row8) * 128;
  ShSide<DQK / 32, DV / 32, 4> x;
  x.G = is_k ? DQK / 32 : DV / 32;
  auto load = [&](int t) {
    const int slot = t % kRowRing;
    if (!mbar_wait_warp(&bars.rows_full[slot], (uint32_t)(t / kRowRing) & 1u, ab)) return false;
    x.load_scales(scales, &rows[slot].row[half * 2], row8, c);
    x.load_codes(codes, &rows[slot].row[half * 2], row8, c);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.rows_empty[slot]);
    return true;
  };
#pragma unroll 1
  for (int t = (warp >> 1) - 2; t < n; t += 2) {
    if (t >= 0) {
      const int e = max((int)(x.top() >> 7) - 127, kExpLow), stage = t % kStages;
      if (lane == 0) {
        x_exp[t % kXRing][half] = is_k ? pow2(e - 11) : (float)e;
        mbar_arrive(&bars.x_full[t % kXRing]);
      }
      x.halves(pow2(11 - e));
      if (!is_k) x.pair_halves();
      if (t >= kStages && !mbar_wait_warp(&empty[stage], (uint32_t)(t / kStages - 1) & 1u, ab)) return;
      x.store(dst + stage * (KT * 64 * x.G), row8, c);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0 && !(is_k && t == dropped)) mbar_arrive(&full[stage]);
    }
    if (t + 2 < n && !load(t + 2)) return;
  }
}

// Where the part of a row lies, of the rows of whole items or of cut ones.  (Where the
// softmax groups take turns, the second one's part lies beside the first's.)
template <class S>
__device__ __forceinline__ int64_t sh_part_row(const SharedParams& p, const ShPiece& pc, bool both, int slot, int r,
                                               int b, int rest, bool& whole) {
  whole = pc.kt == 0 && pc.kt_end == pc.key_tiles;
  const int part = S::kSlots == 2 && !both ? slot : 0;
  if (whole) return ((int64_t)part * p.batch + b) * p.c.heads * p.rows + (int64_t)pc.head * p.rows + rest;
  return ((int64_t)blockIdx.x * 2 + (pc.kt == 0 ? 1 : 0)) * S::kRT + (both ? slot * 128 : part * 128) + r;
}

// A softmax thread's rows where its block gave up: sums of NaN, which the join turns into
// rows of NaN.  (It must not take what the workspace held before for this call's parts.)
template <class S>
__device__ __noinline__ void sh_give_up(const SharedParams& p, int u0, int u1, int slot, int r) {
  ShPiece pc;
  pc.begin(p, u0, u1);
  while (pc.next(p)) {
    const bool both = S::kSlots == 2 && pc.row_slots(p) == 2;
    const long long row = (long long)pc.row_tile * S::kRT + (both ? slot * 128 : 0) + r;
    if (row >= (long long)pc.info.members * p.rows) continue;
    const int member = (int)p.by_rows.div((uint32_t)row), rest = (int)(row - (long long)member * p.rows);
    bool whole;
    const int64_t at = sh_part_row<S>(p, pc, both, slot, r, pc.info.first + member, rest, whole);
    *reinterpret_cast<float2*>((whole ? p.row_ml : p.cut_ml) + at * 2) = make_float2(0.0f, NAN);
  }
}

// The warp that looks up the tiles' tokens, a few tiles ahead of those that load them.
template <int DQK, int DV>
__device__ __forceinline__ void sh_look_up(const SharedParams& p, ShBars& bars, ShRows* rows, int u0, int u1,
                                           const Abort& ab) {
  constexpr int kChunks = KT / 16;  // of 16 tokens, each in one page
  const int lane = threadIdx.x & 31;
  ShPiece look;
  look.begin(p, u0, u1);
  int t = 0;
  while (look.next(p)) {
    const int32_t* table = p.table + (int64_t)look.info.request * p.table_stride;
    for (int kt = look.kt; kt < look.kt_end; ++kt, ++t) {
      const int slot = t % kRowRing, token = kt * KT + 16 * lane;
      const bool here = lane < kChunks && token < look.info.tokens;
      const int page = here ? __ldg(table + (token >> p.c.page_shift)) : -1;
      if (t >= kRowRing && !mbar_wait_warp(&bars.rows_empty[slot], (uint32_t)(t / kRowRing - 1) & 1u, ab)) return;
      const bool inside = (unsigned)page < (unsigned)p.c.num_pages;
      if (here && !inside && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
      const long long row = inside ? ((long long)page * p.c.heads + look.head) * p.c.page_size + (token & (p.c.page_size - 1)) : -1;
      if (lane < kChunks) rows[slot].row[lane] = row;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.rows_full[slot]);
      // lines of 128 bytes of the rows' codes and scales
      auto fetch = [&](auto width_of, const uint8_t* base) {
        constexpr int W = decltype(width_of)::value, kLines = (16 * W + 127) / 128;  // bytes of a row; lines of a chunk
#pragma unroll
        for (int i = 0; i < kChunks * kLines; i += 32) {
          const int chunk = (i + lane) / kLines, line = i + lane - chunk * kLines;
          const long long at = __shfl_sync(0xffffffffu, row, chunk & 31);
          if (chunk < kChunks && at >= 0)
            asm volatile("prefetch.global.L2 [%0];" ::"l"((uint64_t)__cvta_generic_to_global(base + at * W + line * 128)));
        }
      };
      fetch(std::integral_constant<int, DQK / 2>(), p.c.k_codes);
      fetch(std::integral_constant<int, DV / 2>(), p.c.v_codes);
      fetch(std::integral_constant<int, DQK / 16>(), reinterpret_cast<const uint8_t*>(p.c.k_scales));
      fetch(std::integral_constant<int, DV / 16>(), reinterpret_cast<const uint8_t*>(p.c.v_scales));
    }
  }
}

template <bool BF16, int DQK, int DV>
__global__ void __launch_bounds__(kThreads, 1) attn_kv_shared_kernel(const __grid_constant__ SharedParams p) {
  using S = ShShape<DQK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + S::kSlots * S::kQTile;
  uint8_t* sV = sK + S::kKS * S::kKTile;
  __shared__ ShBars bars;
  __shared__ __align__(8) float k_exp[kXRing][2], v_exp[kXRing][2];  // of the halves of a tile: K's unit, V's exponent
  __shared__ ShRows rows[kRowRing];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;

  Abort ab{&abort_flag, p.status, wait_limit(p.dbg)};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.kfull[i], 2);
      mbar_init(&bars.vfull[i], 2);
      mbar_init(&bars.kempty[i], S::kSlots);
      mbar_init(&bars.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_free[i], 128);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&bars.p_full[i][k], 128);
        mbar_init(&bars.o_done[i][k], 1);
      }
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bars.drain[i], 1);
    mbar_init(&bars.q_full, 128 * S::kSlots);
    mbar_init(&bars.q_empty, S::kSlots);
    for (int i = 0; i < kXRing; ++i) mbar_init(&bars.x_full[i], 4);
    for (int i = 0; i < kRowRing; ++i) {
      mbar_init(&bars.rows_full[i], 1);
      mbar_init(&bars.rows_empty[i], 4);
    }
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  // All of that comes before the first kernel's end, and the next kernel may come
  // before this one's (it needs what the first one found out, and waits for this one
  // before it ends itself).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const ShRuns runs(__ldcg(p.total_units), gridDim.x);
  const bool idle = (int)blockIdx.x >= runs.runs;
  const int u0 = idle ? 0 : runs.start(blockIdx.x), u1 = idle ? 0 : runs.start(blockIdx.x + 1);
  if (idle) {
    // (no run for this block)
  } else if (warp >= 8 && warp < 16) {
    const bool is_k = warp < 12;
    sh_convert<DQK, DV>(is_k ? p.c.k_codes : p.c.v_codes, is_k ? p.c.k_scales : p.c.v_scales, is_k, is_k ? sK : sV,
                        is_k ? bars.kfull : bars.vfull, is_k ? bars.kempty : bars.vempty, bars, is_k ? k_exp : v_exp,
                        rows, u1 - u0, dropped_load(p.dbg), ab);
  } else if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 18) sh_look_up<DQK, DV>(p, bars, rows, u0, u1, ab);
    if (warp == 17 || warp == 16 || (warp == 19 && S::kSlots == 2)) {
    // ------------------------------------------------------------ MMA issuers
    // Tile t of the run goes to both softmax groups where two row tiles share it, else to
    // one after the other.  A group's n-th tile uses its P buffer n % 2.
    constexpr uint32_t idesc_s = make_idesc(128, KT, false, false, false);
    constexpr uint32_t idesc_o = make_idesc(128, DV, false, false, true);
    uint32_t t = 0, pieces = 0;
    bool ok = true;
    ShPiece pc;
    pc.begin(p, u0, u1);
    if (warp != 17) {
      const int g = warp == 19 ? 1 : 0;
      const uint64_t kdesc = make_sdesc(smem_u32(sK), 16, 1024);
      uint32_t n = 0;  // tiles that the group had so far
      while (ok && pc.next(p)) {
        const bool both = S::kSlots == 2 && pc.row_slots(p) == 2;
        const uint64_t qa = make_sdesc(smem_u32(sQ + (both ? g : 0) * S::kQTile), 16, 1024);
        if (!mbar_wait_warp(&bars.q_full, pieces & 1u, ab)) break;
        for (int kt = pc.kt; kt < pc.kt_end; ++kt, ++t) {
          const uint32_t st = t % S::kKS;
          const bool mine = both || S::kSlots == 1 || ((kt - pc.kt) & 1) == g;
          ok = mbar_wait_warp(&bars.kfull[st], (t / S::kKS) & 1u, ab);
          // the scores before these have been read
          if (ok && mine && n) ok = mbar_wait_warp(&bars.s_free[g], (n - 1) & 1u, ab);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + g * 128;
          const uint64_t kb = kdesc + (uint64_t)(st * (S::kKTile >> 4));
          if (elect_sync()) {
            if (mine) {
#pragma unroll
              for (int c = 0; c < DQK / 64; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_ss(d, qa + (uint64_t)(c * (kSlotBytes >> 4)) + 2 * k, kb + (uint64_t)(c * (S::kKSlot >> 4)) + 2 * k,
                         idesc_s, (c | k) ? 1u : 0u);
              mma_commit(&bars.s_full[g]);
              mma_commit(&bars.kempty[st]);
            } else {
              mbar_arrive(&bars.kempty[st]);
            }
            if (kt + 1 == pc.kt_end) mma_commit(&bars.q_empty);
          }
          __syncwarp();
          n += mine;
        }
        ++pieces;
      }
    } else {
      const uint64_t vdesc = make_sdesc(smem_u32(sV), S::kKSlot, 1024);
      uint32_t used[2] = {0, 0};
      while (ok && pc.next(p)) {
        const bool both = S::kSlots == 2 && pc.row_slots(p) == 2;
        for (int kt = pc.kt; kt < pc.kt_end && ok; ++kt, ++t) {
          const int first = both || S::kSlots == 1 ? 0 : (kt - pc.kt) & 1, last = both ? 1 : first;
          const uint32_t st = t % S::kVS;
          ok = mbar_wait_warp(&bars.vfull[st], (t / S::kVS) & 1u, ab);
          for (int g = first; g <= last && ok; ++g) {
            const uint32_t n = used[g]++, buf = n & 1u;
            ok = mbar_wait_warp(&bars.p_full[g][buf], (n >> 1) & 1u, ab);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vb = vdesc + (uint64_t)(st * (S::kVTile >> 4));
            const uint32_t d = tmem + S::kTmemO + g * DV, a = tmem + g * 128 + KT + buf * 32;
            // O starts anew with the group's first tile of the piece
            const uint32_t add = kt - pc.kt >= (S::kSlots == 2 && !both ? 2 : 1) ? 1u : 0u;
            if (elect_sync()) {
              mma_ts(d, a, vb, idesc_o, add);
#pragma unroll
              for (int k = 1; k < KT / 16; ++k) mma_ts(d, a + k * 8, vb + k * 128, idesc_o, 1u);
              mma_commit(&bars.o_done[g][buf]);
              if (g == last) mma_commit(&bars.vempty[st]);
            }
            __syncwarp();
          }
        }
      }
    }
    // every MMA has ended before TMEM and shared memory are given back
    uint64_t* drain = &bars.drain[warp == 17 ? 1 : warp == 16 ? 0 : 2];
    if (elect_sync()) {
      mma_commit(drain);
      mbar_wait_quiet(drain, 0, ab.limit_ns);
    }
    __syncwarp();
    }
  } else if (warp < 4 * S::kSlots) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int slot = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t used = 0, t = 0, pieces = 0;
    bool ok = true;
    ShPiece pc;
    pc.begin(p, u0, u1);
    while (ok && pc.next(p)) {
      const bool both = S::kSlots == 2 && pc.row_slots(p) == 2;
      // ---- the query row, times a power of two, in the operand's order
      const long long grow_row = (long long)pc.row_tile * S::kRT + (both ? slot * 128 : 0) + r;  // of the group
      const bool live = grow_row < (long long)pc.info.members * p.rows;
      const int member = live ? (int)p.by_rows.div((uint32_t)grow_row) : 0;
      const int rest = live ? (int)(grow_row - (long long)member * p.rows) : 0;
      const int qi = (int)p.by_group.div(rest), qh = pc.head * p.group + rest - qi * p.group;
      const int b = pc.info.first + member;
      float xs;
      {
        // The warp copies its 32 rows as they are, whole lines at a time, to where their operand
        // goes (the second group's is not used where the groups share the rows); then each
        // thread converts its own row there.
        constexpr int kVecs = DQK / 8;
        const unsigned long long src =
            live ? (unsigned long long)((const uint16_t*)p.q + (int64_t)b * p.q_b + qi * p.q_t + qh * p.q_h) : 0ull;
        uint8_t* const tile = sQ + slot * S::kQTile;
        auto place = [&](int row, int i) {
          return reinterpret_cast<uint4*>(tile + (i >> 3) * kSlotBytes + row * 128 + (((i & 7) ^ (row & 7)) << 4));
        };
        const int lane = threadIdx.x & 31, row0 = r - lane;
#pragma unroll 4
        for (int k = 0; k < kVecs; ++k) {
          const int at = k * 32 + lane, row = at / kVecs, i = at - row * kVecs;
          const unsigned long long from = __shfl_sync(0xffffffffu, src, row);
          *place(row0 + row, i) = from ? __ldg(reinterpret_cast<const uint4*>(from) + i) : make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        uint32_t top = 0;
#pragma unroll 8
        for (int i = 0; i < kVecs; ++i) {
          const uint4 v = *place(r, i);
          const uint32_t mx = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                       __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
          top = max(top, max(mx & 0xffffu, mx >> 16));
        }
        const uint32_t tf = __float_as_uint(Pack<BF16>::to_f((uint16_t)top));
        const int ex = min(max((int)(tf >> 23) - 127 - 13, -100), 100);  // largest at 2^13 .. 2^14
        const float inv = pow2(-ex);
        xs = p.scale_log2 * pow2(ex);
#pragma unroll 4
        for (int i = 0; i < kVecs; ++i) {
          const uint4 v = *place(r, i);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = Pack<BF16>::to_f((uint16_t)(x[e >> 1] >> (16 * (e & 1)))) * inv;
          *place(r, i) = make_uint4(Pack<false>::two(f[0], f[4]), Pack<false>::two(f[1], f[5]), Pack<false>::two(f[2], f[6]),
                                    Pack<false>::two(f[3], f[7]));
        }
        fence_proxy_async();
        mbar_arrive(&bars.q_full);
      }
      // l is held times 2^(kBias - m_run), O times 2^(22 - o_run).  The references follow their
      // maxima when those pass them by more than kLag; o_run lies a whole number from m_run then,
      // so that the probability that m_run is of is exact in fp16.
      float m_run = -INFINITY, o_run = -INFINITY, l_run = 0.0f;
      int tiles = 0;  // of this group's O
      for (int kt = pc.kt; kt < pc.kt_end; ++kt, ++t) {
        if (S::kSlots == 2 && !both && ((kt - pc.kt) & 1) != slot) continue;
        const uint32_t n = used++, buf = n & 1u;
        ok = mbar_wait_warp(&bars.x_full[t % kXRing], (t / kXRing) & 1u, ab) &&
             mbar_wait_warp(&bars.s_full[slot], n & 1u, ab);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sb = tmem + lane_off + slot * 128;
        // the row's scores, read at once: then the next ones may be computed
        uint32_t s[2][32];
        tmem_ld32(sb, s[0]);
        tmem_ld32(sb + 32, s[1]);
        const float2 ku2 = *reinterpret_cast<const float2*>(k_exp[t % kXRing]);
        const float2 ve2 = *reinterpret_cast<const float2*>(v_exp[t % kXRing]);
        const float ku[2] = {ku2.x, ku2.y}, ve[2] = {ve2.x, ve2.y};
        float xt[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) xt[c] = fminf(fmaxf(xs * ku[c], 1.17549435e-38f), 3.40282347e38f);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(&bars.s_free[slot]);
        float m_half[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          auto score = [&](int i) { return __uint_as_float(s[c][i]); };
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(score(i), score(4 + i));
#pragma unroll
          for (int k = 8; k < 32; k += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmax3(m4[i], score(k + i), score(k + 4 + i));
          m_half[c] = xt[c] * fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
        }
        const float m_tile = fmaxf(m_half[0], m_half[1]);
        if (m_tile > m_run + kLag) {
          l_run *= ex2(m_run - m_tile);
          m_run = m_tile;
        }
        const float o_tile = fmaxf(m_half[0] + ve[0], m_half[1] + ve[1]);
        float alpha = 1.0f;
        if (o_tile > o_run + kLag) {
          const float o = m_run + ceilf(o_tile - m_run);
          alpha = ex2(o_run - o);
          o_run = o;
        }
        const bool none = m_run == -INFINITY;
        const float off = none ? 0.0f : kBias - m_run, from = none ? 0.0f : m_run - o_run;
        // the buffer's earlier P has been read
        if (n >= 2 && !mbar_wait_warp(&bars.o_done[slot][buf], ((n >> 1) - 1) & 1u, ab)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // (from 2^-39 down P is 0 in fp16, but must not be in the sum)
          const float lift = fmaxf(from + ve[c], -60.0f);
          const float oc = off + lift;
          const uint64_t x2 = f2_pack(xt[c], xt[c]), off2 = f2_pack(oc, oc);
          uint64_t acc2[2] = {0ull, 0ull};
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y0, y1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), x2, off2), y0, y1);
            const float e0 = ex2(y0), e1 = ex2(y1);
            acc2[i & 1] = f2_add(acc2[i & 1], f2_pack(e0, e1));
            pk[i] = Pack<false>::two(e0, e1);
          }
          tmem_st16(sb + KT + buf * 32 + c * 16, pk);
          float s0, s1;
          f2_unpack(f2_add(acc2[0], acc2[1]), s0, s1);
          sum = fmaf(s0 + s1, ex2(-lift), sum);
        }
        l_run += sum;
        // O of this row so far, if its reference moved
        if (tiles > 0) {
          if (__any_sync(0xffffffffu, alpha != 1.0f)) {
            if (!mbar_wait_warp(&bars.o_done[slot][buf ^ 1u], ((n - 1) >> 1) & 1u, ab)) {  // (the last product)
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t ob = tmem + lane_off + S::kTmemO + slot * DV;
#pragma unroll 1
            for (int c = 0; c < DV; c += 16) {
              uint32_t rr[16];
              tmem_ld16(ob + c, rr);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
              tmem_st16(ob + c, rr);
            }
          }
        }
        ++tiles;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars.p_full[slot][buf]);
      }
      if (!ok) {  // (what has been stored is there before TMEM is given back)
        tmem_st_wait();
        tc_fence_before();
        break;
      }
      // ---- the piece's part: O, maximum and sum of each row
      for (uint32_t n = used > 2 ? used - 2 : 0; n < used && ok; ++n)
        ok = mbar_wait_warp(&bars.o_done[slot][n & 1u], (n >> 1) & 1u, ab);
      // (nothing reads Q any more, the other group's tiles included)
      ok = ok && mbar_wait_warp(&bars.q_empty, pieces & 1u, ab);
      if (!ok) break;
      tc_fence_after();
      bool whole;
      const int64_t at = sh_part_row<S>(p, pc, both, slot, r, b, rest, whole);
      float* const o = (whole ? p.row_o : p.cut_o) + at * DV;
      float* const ml = (whole ? p.row_ml : p.cut_ml) + at * 2;
      if (live) *reinterpret_cast<float2*>(ml) = make_float2(m_run - kBias, l_run);
      if (tiles > 0) {
        const uint32_t ob = tmem + lane_off + S::kTmemO + slot * DV;
        const float unit = ex2(fmaxf(o_run - m_run - 11.0f, -126.0f));
        // 32 columns at a time through the warp's part of Q's memory (its MMAs have ended), so
        // that eight lanes write a row's 128 bytes
        const int lane = threadIdx.x & 31;
        float4* tile = reinterpret_cast<float4*>(sQ + slot * S::kQTile + (warp & 3) * 4096);  // [32][8], swizzled
        const unsigned long long mine = live ? (unsigned long long)o : 0ull;
#pragma unroll 1
        for (int c = 0; c < DV / 32; ++c) {
          uint32_t rr[32];
          tmem_ld32(ob + c * 32, rr);
          tmem_ld_wait();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(rr[8 * i + e]) * unit;
            tile[lane * 8 + ((2 * i) ^ (lane & 7))] = make_float4(f[0], f[2], f[4], f[6]);
            tile[lane * 8 + ((2 * i + 1) ^ (lane & 7))] = make_float4(f[1], f[3], f[5], f[7]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3), col = lane & 7;
            const unsigned long long dst = __shfl_sync(0xffffffffu, mine, row);
            if (dst) reinterpret_cast<float4*>(dst)[c * 8 + col] = tile[row * 8 + (col ^ (row & 7))];
          }
        }
      }
      tc_fence_before();
      ++pieces;
    }
    if (!ok) sh_give_up<S>(p, u0, u1, slot, r);
  }
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------- the join
// A group of d_v / 4 threads takes a row, four dims each: its own tokens and the parts
// of the prefix, in the order of the runs.  Where items are cut into many parts a whole
// block takes a row, its groups share out the parts and the first one adds up theirs.
template <bool BF16, int DV>
__global__ void __launch_bounds__(256, 6) attn_kv_shared_join_kernel(const __grid_constant__ SharedParams p, int most_runs) {
  constexpr int kLanes = DV / 4, kGroups = 256 / kLanes;
  __shared__ float4 s_acc[kGroups][kLanes];
  __shared__ float s_mx[kGroups], s_l[kGroups];
  const int64_t all = (int64_t)p.batch * p.c.heads * p.rows;
  const int d4 = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ShRuns runs(__ldcg(p.total_units), most_runs);
  const bool together = runs.runs > kJoinParts * __ldcg(p.total_units + 1);  // (not where nothing is shared)
  const int per = together ? 1 : kGroups;
  for (int64_t at0 = (int64_t)blockIdx.x * per; at0 < all; at0 += (int64_t)gridDim.x * per) {
    const int64_t at = at0 + (together ? 0 : group);
    const bool live = at < all;
    const int b = live ? (int)p.by_request.div((uint32_t)at) : 0, in = live ? (int)(at - (int64_t)b * p.c.heads * p.rows) : 0;
    const int head = (int)p.by_rows.div(in), rest = in - head * p.rows;
    const int qi = (int)p.by_group.div(rest), qh = head * p.group + rest - qi * p.group;
    const int64_t lse_at = ((int64_t)b * p.heads_q + qh) * p.seqlen_q + qi;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, sum = 0.0f, lse = -INFINITY;
    auto add = [&](const float4& y, float m, float l) {
      if (l == 0.0f) return;  // a part without tiles
      const float to = fmaxf(mx, m), f = ex2(m - to), a = mx == -INFINITY ? 0.0f : ex2(mx - to);
      mx = to;
      sum = fmaf(sum, a, l * f);
      acc.x = fmaf(acc.x, a, y.x * f), acc.y = fmaf(acc.y, a, y.y * f);
      acc.z = fmaf(acc.z, a, y.z * f), acc.w = fmaf(acc.w, a, y.w * f);
    };
    const int g = live ? p.group_of[b] : -1;
    if (live && (!together || group == 0)) {  // its own tokens
      acc = *reinterpret_cast<const float4*>(p.own_o + (((int64_t)b * p.seqlen_q + qi) * p.heads_q + qh) * DV + d4 * 4);
      lse = p.own_lse[lse_at];
      mx = lse * 1.4426950408889634f;
      sum = 1.0f;
    }
    if (g >= 0) {
      const ShGroup info = ((const ShGroup*)p.group_info)[g];
      const int key_tiles = sh_key_tiles(p, info), row_tiles = sh_row_tiles(p, info);
      const long long row = (long long)(b - info.first) * p.rows + rest;
      const int rt = (int)(row >> (p.row_tile == 256 ? 8 : 7)), r = (int)(row & (p.row_tile - 1));
      const long long left = (long long)info.members * p.rows - (long long)rt * p.row_tile;
      const int halves = p.row_tile == 256 && left <= 128 ? 2 : 1;
      const int u = info.unit0 + (head * row_tiles + rt) * key_tiles;
      const int k0 = runs.of(u), np = runs.of(u + key_tiles - 1) - k0 + 1;
      const int step = together ? kGroups : 1;
#pragma unroll 4
      for (int i = together ? group : 0; i < halves * np; i += step) {
        const int half = i >= np, k = i - half * np;
        const int64_t x = np == 1 ? half * all + at
                                  : ((int64_t)(k0 + k) * 2 + (k == 0 ? 1 : 0)) * p.row_tile + half * 128 + r;
        const float2 s = *reinterpret_cast<const float2*>((np == 1 ? p.row_ml : p.cut_ml) + x * 2);
        add(*reinterpret_cast<const float4*>((np == 1 ? p.row_o : p.cut_o) + x * DV + d4 * 4), s.x, s.y);
      }
    }
    if (together) {
      __syncthreads();
      s_acc[group][d4] = acc;
      if (d4 == 0) s_mx[group] = mx, s_l[group] = sum;
      __syncthreads();
      if (group > 0) continue;
#pragma unroll
      for (int k = 1; k < kGroups; ++k) add(s_acc[k][d4], s_mx[k], s_l[k]);
    }
    if (!live) continue;
    if (g >= 0) {
      const float inv = 1.0f / sum;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      lse = (mx + log2f(sum)) * 0.6931471805599453f;
    }
    const int64_t to = (int64_t)b * p.o_b + qi * p.o_t + qh * p.o_h + d4 * 4;
    if (p.o_f32)
      *reinterpret_cast<float4*>((float*)p.o + to) = acc;
    else
      *reinterpret_cast<uint2*>((uint16_t*)p.o + to) = make_uint2(Pack<BF16>::two(acc.x, acc.y), Pack<BF16>::two(acc.z, acc.w));
    if (d4 == 0) p.lse[lse_at] = lse;
  }
}

// ----------------------------------------------------------------- launches
namespace {

template <bool BF16, int DQK, int DV>
cudaError_t sh_launch(const SharedParams& p, int num_sms, cudaStream_t st) {
  using S = ShShape<DQK, DV>;
  auto* k = attn_kv_shared_kernel<BF16, DQK, DV>;
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_early(k, (unsigned)num_sms, kThreads, S::kSmem, st, p);
}

template <bool BF16>
cudaError_t sh_dims(const SharedParams& p, int num_sms, cudaStream_t st) {
  if (p.c.d_qk == 64 && p.c.d_v == 64) return sh_launch<BF16, 64, 64>(p, num_sms, st);
  if (p.c.d_qk == 128 && p.c.d_v == 128) return sh_launch<BF16, 128, 128>(p, num_sms, st);
  if (p.c.d_qk == 192 && p.c.d_v == 128) return sh_launch<BF16, 192, 128>(p, num_sms, st);
  if (p.c.d_qk == 256 && p.c.d_v == 256) return sh_launch<BF16, 256, 256>(p, num_sms, st);
  return cudaErrorNotSupported;
}

template <bool BF16>
cudaError_t sh_join(const SharedParams& p, int num_sms, cudaStream_t st) {
  const int64_t rows = (int64_t)p.batch * p.c.heads * p.rows;
  const unsigned blocks = (unsigned)std::min<int64_t>(rows, (int64_t)num_sms * 8);
  switch (p.c.d_v) {
    case 64: return launch_early(attn_kv_shared_join_kernel<BF16, 64>, blocks, 256, 0, st, p, num_sms);
    case 128: return launch_early(attn_kv_shared_join_kernel<BF16, 128>, blocks, 256, 0, st, p, num_sms);
    default: return launch_early(attn_kv_shared_join_kernel<BF16, 256>, blocks, 256, 0, st, p, num_sms);
  }
}

}  // namespace

void shared_tiles(int d_v, int& row_tile, int& key_tile) {
  row_tile = d_v > 128 ? 128 : 256;
  key_tile = KT;
}
size_t shared_group_bytes() { return sizeof(ShGroup); }

cudaError_t launch_kv4_shared_prefix(const SharedParams& p, bool bf16, int num_sms, cudaStream_t st) {
  const int threads = std::max(p.batch, p.groups + 1) <= kPlanFew ? kPlanFew : kPlanThreads;
  attn_kv_shared_plan_kernel<<<1, threads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return bf16 ? sh_dims<true>(p, num_sms, st) : sh_dims<false>(p, num_sms, st);
}
cudaError_t launch_kv4_shared_join(const SharedParams& p, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? sh_join<true>(p, num_sms, st) : sh_join<false>(p, num_sms, st);
}

}  // namespace attn
