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
//   warps 8..11  K codes to the fp16 operand, warps 12..15 V codes: a thread takes a
//                token's row, its codes loaded a tile ahead;
//   warp 16      issues S = Q K^T, warp 17 O += P V.
// A block's run of work is a stretch of the list (group, kv head, 256 query rows, tile
// of keys), cut into equal runs.  With more than 128 rows the two softmax groups have
// 128 rows each and share every converted tile; with fewer they take turns at the tiles
// for the same rows, each with its own O (two parts for the join).  At head dim 256 O
// fills half of TMEM: one group, tiles of 64 keys, 128 rows.
//
// Numbers: code - 8 is exact in fp16 and so is its product with a bf16 scale (4 + 8
// bits), times a power of two: K's makes the tile's largest scale 2^11 .. 2^12 and comes
// back with the scores; V's does for the largest scale of the tiles so far (with room
// for 2^3), and O follows when it grows.  q is held as in kvdecode.cu.  Probabilities
// are FP32 in the sum and rounded to fp16 for the second product, times 2^14: their
// reference moves when a score passes it by 1, so they stay below 2^15, and those 2^-38
// below the row's maximum are still told from 0.
// In a row of 8 dims the operand's order is 0 4 1 5 2 6 3 7 (a mask of a word of codes
// makes pairs n, n + 4): Q is stored the same way, O's columns are put back at the end.
#include <algorithm>
#include <atomic>

#include "kcommon.cuh"
#include "kv.h"
#include "kvtile.cuh"

namespace attn {

namespace {

constexpr int kGranule = 64;  // tokens: prefixes are taken in whole ones, the rest is the requests' own
constexpr float kBias = 14.0f;  // probabilities are held times 2^14 (2^15 where the reference lags)
constexpr int kXRing = 8;
constexpr int kThreads = 640;

template <int DQK, int DV>
struct ShShape {
  static constexpr bool kWide = DV > 128;
  static constexpr int KT = kWide ? 64 : 128;      // keys of a tile
  static constexpr int kSlots = kWide ? 1 : 2;     // softmax groups
  static constexpr int kRT = 128 * kSlots;         // query rows of an item
  static constexpr int kKSlot = KT * 128;          // 64 dims of a tile
  static constexpr int kKTile = kKSlot * (DQK / 64), kVTile = kKSlot * (DV / 64);
  static constexpr int kQTile = kSlotBytes * (DQK / 64);
  static constexpr int kKS = DQK == 64 ? 4 : 2, kVS = DQK == 64 ? 4 : DQK == 192 ? 1 : 2;  // stages
  static constexpr int kSmem = kSlots * kQTile + kKS * kKTile + kVS * kVTile + 1024;
  static constexpr int kTmemO = 256;
};

}  // namespace

// ----------------------------------------------------------------- the list of work
// What the first kernel finds out about a group.
struct ShGroup {
  long long unit0;  // units (a tile of an item) of the groups before it
  int tokens;       // of the prefix that its requests share, a multiple of kGranule
  int request;      // one that shares it (its table row is read)
  int first, members;
};

__device__ __forceinline__ int sh_row_tiles(const SharedParams& p, const ShGroup& g) {
  return (int)(((long long)g.members * p.rows + p.row_tile - 1) / p.row_tile);
}
__device__ __forceinline__ int sh_key_tiles(const SharedParams& p, const ShGroup& g) {
  return (g.tokens + p.key_tile - 1) / p.key_tile;
}

// One block: which requests share what.
__global__ void __launch_bounds__(1024) attn_kv_shared_plan_kernel(const __grid_constant__ SharedParams p) {
  __shared__ int s_bad;
  __shared__ long long s_sum[32];
  ShGroup* groups = (ShGroup*)p.group_info;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cap = (int64_t)p.cols << p.c.page_shift;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  bool bad = false;
  for (int g = tid; g <= p.groups; g += 1024) {
    const int at = p.group_starts[g];
    bad |= at < 0 || at > p.batch || (g > 0 && p.group_starts[g - 1] > at);
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const bool none = s_bad != 0;  // groups that are not in order share nothing
  bad = none;
  for (int g = tid; g < p.groups; g += 1024) {
    const int n = p.shared_lens[g];
    const bool ok = n >= 0 && n <= cap;
    bad |= !ok;
    ShGroup x;
    x.unit0 = 0;
    x.tokens = none || !ok ? 0 : n / kGranule * kGranule;
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
    return n > 0 && len <= cap && len - p.seqlen_q >= n ? lo : -1;
  };
  for (int b = tid; b < p.batch; b += 1024) {
    const int g = group_of(b);
    p.group_of[b] = g;
    if (g >= 0) {
      atomicMin(&groups[g].request, b);
      atomicAdd(&groups[g].members, 1);
    }
  }
  __syncthreads();
  // a prefix that one request has alone is that request's own
  for (int b = tid; b < p.batch; b += 1024) {
    int g = p.group_of[b];
    if (g >= 0 && __ldcg(&groups[g].members) < 2) p.group_of[b] = g = -1;
    p.starts[b] = g >= 0 ? groups[g].tokens : 0;
  }
  __syncthreads();
  long long before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 1024) {
    const int g = g0 + tid;
    ShGroup x;
    long long units = 0;
    if (g < p.groups) {
      x.first = groups[g].first;
      x.request = __ldcg(&groups[g].request);  // (atomics are done in L2)
      x.tokens = __ldcg(&groups[g].members) < 2 ? 0 : groups[g].tokens;
      x.members = none ? 0 : p.group_starts[g + 1] - x.first;
      if (x.tokens) units = (long long)p.c.heads * sh_row_tiles(p, x) * sh_key_tiles(p, x);
    }
    long long j = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, j, o);
      if (lane >= o) j += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = j;
    __syncthreads();
    x.unit0 = before + j - units;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) x.unit0 += s_sum[w];
      before += s_sum[w];
    }
    if (g < p.groups) groups[g] = x;
  }
  if (tid == 0) *p.total_units = before;
}

// The list is cut into `runs` equal runs.
struct ShRuns {
  long long total, each, more;
  int runs;
  __device__ __forceinline__ ShRuns(long long total_, int most) {
    total = total_;
    runs = (int)min((long long)most, total);
    each = runs ? total / runs : 0;
    more = total - each * runs;
  }
  __device__ __forceinline__ long long start(int k) const { return each * k + min((long long)k, more); }
  __device__ __forceinline__ int of(long long u) const {
    const long long big = more * (each + 1);
    return (int)(u < big ? u / (each + 1) : more + (u - big) / each);
  }
};

// The next piece of a run: tiles kt .. kt_end - 1 of one item.
struct ShPiece {
  long long u, end;  // what is left of the run
  int g;
  ShGroup info;
  int head, row_tile, kt, kt_end, key_tiles;
  __device__ __forceinline__ void begin(const SharedParams& p, long long u0, long long u1) {
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
      const long long n = info.tokens ? (long long)p.c.heads * row_tiles * key_tiles : 0, at = u - info.unit0;
      if (at >= n) {  // (groups without units are passed by)
        info = groups[++g];
        continue;
      }
      const int item = (int)(at / key_tiles);
      kt = (int)(at - (long long)item * key_tiles);
      head = item / row_tiles;
      row_tile = item - head * row_tiles;
      kt_end = (int)min((long long)key_tiles, kt + (end - u));
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

__device__ __forceinline__ void group_sync(int id) {  // 128 threads
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

constexpr int kExpLow = -110;  // exponents of scales from there on are told apart

struct ShBars {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t q_full, q_empty, x_full[kXRing], drain[2];
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
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  }
}

// The group of four warps that turns one side's codes into its operand.  Two threads
// share a token's row where a tile has 64 keys.
template <int DQK, int DV, bool K>
__device__ __forceinline__ void sh_convert(const SharedParams& p, uint8_t* ring, ShBars& bars, int* x_exp,
                                           uint32_t (*s_top)[4], long long u0, long long u1, const Abort& ab) {
  using S = ShShape<DQK, DV>;
  constexpr int D = K ? DQK : DV, G = D / 32, KT = S::KT, kParts = 128 / KT, kStages = K ? S::kKS : S::kVS;
  constexpr int kTileBytes = K ? S::kKTile : S::kVTile;
  constexpr int NW = D / 8 / kParts, NS = (G / 2 + kParts - 1) / kParts;  // words of codes and of scales of a thread
  static_assert(kParts == 1 || G % (4 * kParts) == 0, "halves of a row");
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  const int row = tid % KT, part = tid / KT;
  const uint8_t* codes = K ? p.c.k_codes : p.c.v_codes;
  const uint8_t* scales = reinterpret_cast<const uint8_t*>(K ? p.c.k_scales : p.c.v_scales);
  uint64_t* full = K ? bars.kfull : bars.vfull;
  uint64_t* empty = K ? bars.kempty : bars.vempty;

  // tiles are looked up two ahead (the page), loaded one ahead (the codes)
  ShPiece look;
  look.begin(p, u0, u1);
  bool more = look.next(p);
  int look_kt = look.kt;
  struct Tile {
    int page, head, offset;
    bool first;  // of its piece
  };
  auto look_up = [&]() {
    Tile t{-1, 0, 0, false};
    if (!more) return t;
    t.first = look_kt == look.kt;
    t.head = look.head;
    const int token = look_kt * KT + row;
    t.offset = token & (p.c.page_size - 1);
    if (token < look.info.tokens) {
      t.page = p.table[(int64_t)look.info.request * p.table_stride + (token >> p.c.page_shift)];
      if ((unsigned)t.page >= (unsigned)p.c.num_pages) {
        t.page = -1;
        if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
      }
    }
    if (++look_kt == look.kt_end) {
      more = look.next(p);
      look_kt = look.kt;
    }
    return t;
  };
  uint32_t w[NW], sc[NS], wn[NW], scn[NS];
  auto load = [&](const Tile& t, uint32_t (&w)[NW], uint32_t (&sc)[NS]) {
    if (t.page < 0) {  // zeros
#pragma unroll
      for (int i = 0; i < NW; ++i) w[i] = 0x88888888u;
#pragma unroll
      for (int i = 0; i < NS; ++i) sc[i] = 0u;
      return;
    }
    const int64_t at = ((int64_t)t.page * p.c.heads + t.head) * p.c.page_size + t.offset;
    if constexpr (kParts == 1) {
      row_words<NW>(codes + at * (D / 2), w);
      row_words<NS>(scales + at * (2 * G), sc);
    } else {
      // groups part * G / 2 .. of the row: K words c G + g, V half-words r G + g
      constexpr int H = G / kParts;
      row_words<NS>(scales + at * (2 * G) + part * 2 * H, sc);
      if (K) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t x[H];
          row_words<H>(codes + at * (D / 2) + (c * G + part * H) * 4, x);
#pragma unroll
          for (int g = 0; g < H; ++g) w[c * H + g] = x[g];
        }
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          uint32_t x[H / 2];
          row_words<H / 2>(codes + at * (D / 2) + (r * G + part * H) * 2, x);
#pragma unroll
          for (int g = 0; g < H / 2; ++g) w[r * (H / 2) + g] = x[g];
        }
      }
    }
  };
  const long long n = u1 - u0;
  Tile next = look_up();
  load(next, w, sc);
  bool first = next.first;
  next = look_up();
  int ref = 0;
  bool live = true;  // (after a wait that gave up the group's barriers go on, so that none of its warps is left there)
  for (long long t = 0; t < n; ++t) {
    load(next, wn, scn);
    const bool next_first = next.first;
    next = look_up();
    // ---- the tile's largest finite scale
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const uint32_t lo = sc[i] & 0x7fffu, hi = (sc[i] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) top = max(top, lo);
      if (hi < 0x7f80u) top = max(top, hi);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    uint32_t* tops = s_top[t & 1];
    if (lane == 0) tops[warp] = top;
    group_sync(K ? 1 : 2);
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const int e = max((int)(top >> 7) - 127, kExpLow);
    if (K)
      ref = e;
    else if (first)
      ref = e;
    else if (e > ref)
      ref = min(e + 3, 127);
    if (tid == 0) {
      x_exp[t % kXRing] = ref;
      mbar_arrive(&bars.x_full[t % kXRing]);
    }
    const float f = pow2(11 - ref);
    __half2 s[2 * NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      s[2 * i] = __float2half2_rn(scale_of(sc, 2 * i) * f);
      s[2 * i + 1] = __float2half2_rn(scale_of(sc, 2 * i + 1) * f);
    }
    const int stage = (int)(t % kStages);
    live = live && (t < kStages || mbar_wait_warp(&empty[stage], (uint32_t)((t / kStages) - 1) & 1u, ab));
    uint8_t* dst = ring + stage * kTileBytes + row * 128;
    constexpr int H = G / kParts;
    if (live) {
#pragma unroll
      for (int g = 0; g < H; ++g)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t x;
          if (K)
            x = w[c * H + g];
          else
            x = __byte_perm(w[(2 * c * H + g) >> 1], w[((2 * c + 1) * H + g) >> 1], (g & 1) ? 0x7632 : 0x5410);
          const int gg = part * H + g, chunk = (gg & 1) * 4 + c;
          *reinterpret_cast<uint4*>(dst + (gg >> 1) * S::kKSlot + ((chunk ^ (row & 7)) << 4)) = scaled_codes(x, s[g]);
        }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = wn[i];
#pragma unroll
    for (int i = 0; i < NS; ++i) sc[i] = scn[i];
    first = next_first;
  }
}

template <bool BF16, int DQK, int DV>
__global__ void __launch_bounds__(kThreads, 1) attn_kv_shared_kernel(const __grid_constant__ SharedParams p) {
  using S = ShShape<DQK, DV>;
  constexpr int KT = S::KT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + S::kSlots * S::kQTile;
  uint8_t* sV = sK + S::kKS * S::kKTile;
  __shared__ ShBars bars;
  __shared__ int k_exp[kXRing], v_exp[kXRing];
  __shared__ uint32_t s_top[2][2][4];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;

  const ShRuns runs(*p.total_units, gridDim.x);
  if ((int)blockIdx.x >= runs.runs) return;
  const long long u0 = runs.start(blockIdx.x), u1 = runs.start(blockIdx.x + 1);
  Abort ab{&abort_flag, p.status, kWaitLimitNs};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.kfull[i], 4);
      mbar_init(&bars.vfull[i], 4);
      mbar_init(&bars.kempty[i], 1);
      mbar_init(&bars.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 128);
      mbar_init(&bars.o_done[i], 1);
      mbar_init(&bars.drain[i], 1);
    }
    mbar_init(&bars.q_full, 128 * S::kSlots);
    mbar_init(&bars.q_empty, 1);
    for (int i = 0; i < kXRing; ++i) mbar_init(&bars.x_full[i], 2);
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp >= 8 && warp < 12) {
    sh_convert<DQK, DV, true>(p, sK, bars, k_exp, s_top[0], u0, u1, ab);
  } else if (warp >= 12 && warp < 16) {
    sh_convert<DQK, DV, false>(p, sV, bars, v_exp, s_top[1], u0, u1, ab);
  } else if (warp == 16 || warp == 17) {
    // ------------------------------------------------------------ MMA issuers
    // Tile t of the run goes to S buffers first .. last: both where two row tiles share
    // it, else one after the other.  (At head dim 256 the one group has two buffers.)
    const bool s_role = warp == 16;
    constexpr uint32_t idesc_s = make_idesc(128, KT, false, false, false);
    constexpr uint32_t idesc_o = make_idesc(128, DV, false, false, true);
    const uint64_t qdesc = make_sdesc(smem_u32(sQ), 16, 1024);
    const uint64_t kdesc = make_sdesc(smem_u32(sK), 16, 1024);
    const uint64_t vdesc = make_sdesc(smem_u32(sV), S::kKSlot, 1024);
    uint32_t used[2] = {0, 0};  // tiles that a buffer had so far
    uint32_t t = 0, pieces = 0;
    bool ok = true;
    ShPiece pc;
    pc.begin(p, u0, u1);
    while (ok && pc.next(p)) {
      const bool both = S::kSlots == 2 && pc.row_slots(p) == 2;
      if (s_role && !mbar_wait_warp(&bars.q_full, pieces & 1u, ab)) break;
      tc_fence_after();
      for (int kt = pc.kt; kt < pc.kt_end && ok; ++kt, ++t) {
        const int first = both ? 0 : (kt - pc.kt) & 1, last = both ? 1 : first;
        if (s_role) {
          const uint32_t st = t % S::kKS;
          ok = mbar_wait_warp(&bars.kfull[st], (t / S::kKS) & 1u, ab);
          for (int b = first; b <= last && ok; ++b) {
            // the buffer's earlier P has been read
            if (used[b] && !mbar_wait_warp(&bars.o_done[b], (used[b] - 1) & 1u, ab)) {
              ok = false;
              break;
            }
            ++used[b];
            tc_fence_after();
            const uint64_t qa = qdesc + (uint64_t)((both ? b : 0) * (S::kQTile >> 4));
            const uint64_t kb = kdesc + (uint64_t)(st * (S::kKTile >> 4));
            if (elect_sync()) {
#pragma unroll
              for (int c = 0; c < DQK / 64; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_ss(tmem + b * 128, qa + (uint64_t)(c * (kSlotBytes >> 4)) + 2 * k,
                         kb + (uint64_t)(c * (S::kKSlot >> 4)) + 2 * k, idesc_s, (c | k) ? 1u : 0u);
              mma_commit(&bars.s_full[b]);
              if (b == last) mma_commit(&bars.kempty[st]);
              if (b == last && kt + 1 == pc.kt_end) mma_commit(&bars.q_empty);
            }
            __syncwarp();
          }
        } else {
          const uint32_t st = t % S::kVS;
          ok = mbar_wait_warp(&bars.vfull[st], (t / S::kVS) & 1u, ab);
          for (int b = first; b <= last && ok; ++b) {
            ok = mbar_wait_warp(&bars.p_full[b], used[b] & 1u, ab);
            if (!ok) break;
            ++used[b];
            tc_fence_after();
            const uint64_t vb = vdesc + (uint64_t)(st * (S::kVTile >> 4));
            const uint32_t d = tmem + S::kTmemO + (S::kSlots == 2 ? b * DV : 0);
            // O starts anew with its first tile of the piece
            const uint32_t add = kt - pc.kt >= (S::kSlots == 2 && !both ? 2 : 1) ? 1u : 0u;
            if (elect_sync()) {
              mma_ts(d, tmem + b * 128, vb, idesc_o, add);
#pragma unroll
              for (int k = 1; k < KT / 16; ++k) mma_ts(d, tmem + b * 128 + k * 8, vb + k * 128, idesc_o, 1u);
              mma_commit(&bars.o_done[b]);
              if (b == last) mma_commit(&bars.vempty[st]);
            }
            __syncwarp();
          }
        }
      }
      ++pieces;
    }
    // every MMA has ended before TMEM and shared memory are given back
    uint64_t* drain = &bars.drain[s_role ? 0 : 1];
    if (elect_sync()) {
      mma_commit(drain);
      mbar_wait_quiet(drain, 0, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp < 4 * S::kSlots) {
    // ------------------------------------------------------------ softmax
    const int slot = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t used[2] = {0, 0}, t = 0, pieces = 0;
    bool ok = true;
    ShPiece pc;
    pc.begin(p, u0, u1);
    while (ok && pc.next(p)) {
      const bool both = S::kSlots == 2 && pc.row_slots(p) == 2;
      // ---- the query row, times a power of two, in the operand's order
      if (pieces && !mbar_wait_warp(&bars.q_empty, (pieces - 1) & 1u, ab)) break;
      const long long grow_row = (long long)pc.row_tile * S::kRT + (both ? slot * 128 : 0) + r;  // of the group
      const bool live = grow_row < (long long)pc.info.members * p.rows;
      const int member = live ? (int)p.by_rows.div((uint32_t)grow_row) : 0;
      const int rest = live ? (int)(grow_row - (long long)member * p.rows) : 0;
      const int qi = (int)p.by_group.div(rest), qh = pc.head * p.group + rest - qi * p.group;
      const int b = pc.info.first + member;
      float xs;
      {
        const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)p.q + (int64_t)b * p.q_b + qi * p.q_t + qh * p.q_h);
        uint32_t top = 0;
        if (live)
#pragma unroll 8
          for (int i = 0; i < DQK / 8; ++i) {
            const uint4 v = __ldg(src + i);
            const uint32_t mx = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
            top = max(top, max(mx & 0xffffu, mx >> 16));
          }
        const uint32_t tf = __float_as_uint(Pack<BF16>::to_f((uint16_t)top));
        const int ex = min(max((int)(tf >> 23) - 127 - 13, -100), 100);  // largest at 2^13 .. 2^14
        const float inv = pow2(-ex);
        xs = p.scale_log2 * pow2(ex);
        if (both || slot == 0) {
          uint8_t* dst = sQ + (both ? slot : 0) * S::kQTile + r * 128;
#pragma unroll 4
          for (int i = 0; i < DQK / 8; ++i) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live) v = __ldg(src + i);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = Pack<BF16>::to_f((uint16_t)(x[e >> 1] >> (16 * (e & 1)))) * inv;
            *reinterpret_cast<uint4*>(dst + (i >> 3) * kSlotBytes + (((i & 7) ^ (r & 7)) << 4)) =
                make_uint4(Pack<false>::two(f[0], f[4]), Pack<false>::two(f[1], f[5]), Pack<false>::two(f[2], f[6]),
                           Pack<false>::two(f[3], f[7]));
          }
        }
        fence_proxy_async();
        mbar_arrive(&bars.q_full);
      }
      float m_run = -INFINITY, l_run = 0.0f;
      int v_ref = 0, tiles = 0;  // of this group's O
      for (int kt = pc.kt; kt < pc.kt_end; ++kt, ++t) {
        const int buf = S::kSlots == 2 ? slot : (kt - pc.kt) & 1;
        if (S::kSlots == 2 && !both && ((kt - pc.kt) & 1) != slot) continue;
        ok = mbar_wait_warp(&bars.x_full[t % kXRing], (t / kXRing) & 1u, ab) &&
             mbar_wait_warp(&bars.s_full[buf], used[buf] & 1u, ab);
        if (!ok) break;
        ++used[buf];
        tc_fence_after();
        const float xt = fminf(xs * pow2(k_exp[t % kXRing] - 11), 3.40282347e38f);
        const int v_new = v_exp[t % kXRing];
        const uint32_t sb = tmem + lane_off + buf * 128;
        const int chunks = min(KT, pc.info.tokens - kt * KT) / 32;  // (whole granules)
        // the row's maximum
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < KT / 32; ++c) {
          if (c >= chunks) break;
          uint32_t rr[32];
          tmem_ld32(sb + c * 32, rr);
          tmem_ld_wait();
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            m4[i] = fmax3(__uint_as_float(rr[8 * i]), __uint_as_float(rr[8 * i + 1]),
                          fmax3(__uint_as_float(rr[8 * i + 2]), __uint_as_float(rr[8 * i + 3]),
                                fmax3(__uint_as_float(rr[8 * i + 4]), __uint_as_float(rr[8 * i + 5]),
                                      fmaxf(__uint_as_float(rr[8 * i + 6]), __uint_as_float(rr[8 * i + 7])))));
          mx = fmax3(mx, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        const float m_tile = mx * xt;
        const bool grow = m_tile > m_run + 1.0f;
        const float m_new = grow ? m_tile : m_run;
        float alpha = grow ? ex2(m_run - m_new) : 1.0f;
        m_run = m_new;
        const float off = m_run == -INFINITY ? 0.0f : kBias - m_run;
        const uint64_t x2 = f2_pack(xt, xt), off2 = f2_pack(off, off);
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < KT / 32; ++c) {
          uint32_t pk[16];
          if (c < chunks) {
            uint32_t rr[32];
            tmem_ld32(sb + c * 32, rr);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float y0, y1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1])), x2, off2), y0, y1);
              const float e0 = ex2(y0), e1 = ex2(y1);
              acc2[i & 3] = f2_add(acc2[i & 3], f2_pack(e0, e1));
              pk[i] = Pack<false>::two(e0, e1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0u;
          }
          tmem_st16(sb + c * 16, pk);
        }
        float s0, s1, s2, s3;
        f2_unpack(f2_add(acc2[0], acc2[1]), s0, s1);
        f2_unpack(f2_add(acc2[2], acc2[3]), s2, s3);
        l_run = l_run * alpha + ((s0 + s1) + (s2 + s3));
        // O of this row so far: the maximum grew, or V's unit did
        if (tiles > 0) {
          if (v_new > v_ref) alpha *= pow2(max(v_ref - v_new, -126));
          if (__any_sync(0xffffffffu, alpha != 1.0f)) {
            if (S::kSlots == 1 && !mbar_wait_warp(&bars.o_done[buf ^ 1], (used[buf ^ 1] - 1) & 1u, ab)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t ob = tmem + lane_off + S::kTmemO + (S::kSlots == 2 ? slot * DV : 0);
#pragma unroll
            for (int c = 0; c < DV / 32; ++c) {
              uint32_t rr[32], lo16[16], hi16[16];
              tmem_ld32(ob + c * 32, rr);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                lo16[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
                hi16[i] = __float_as_uint(__uint_as_float(rr[16 + i]) * alpha);
              }
              tmem_st16(ob + c * 32, lo16);
              tmem_st16(ob + c * 32 + 16, hi16);
            }
          }
        }
        v_ref = v_new;
        ++tiles;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars.p_full[buf]);
      }
      if (!ok) break;
      // ---- the piece's part: O, maximum and sum of each row
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int buf = S::kSlots == 2 ? slot : i;
        if (S::kSlots == 2 && i) break;
        if (used[buf] && !mbar_wait_warp(&bars.o_done[buf], (used[buf] - 1) & 1u, ab)) ok = false;
      }
      if (!ok) break;
      tc_fence_after();
      const bool whole = pc.kt == 0 && pc.kt_end == pc.key_tiles;
      // (where the groups take turns, the second one's part lies beside the first's)
      const int part = S::kSlots == 2 && !both ? slot : 0;
      float *o, *ml;
      if (whole) {
        const int64_t at = ((int64_t)part * p.batch + b) * p.c.heads * p.rows + (int64_t)pc.head * p.rows + rest;
        o = p.row_o + at * DV;
        ml = p.row_ml + at * 2;
      } else {
        const int64_t at = ((int64_t)blockIdx.x * 2 + (pc.kt == 0 ? 1 : 0)) * S::kRT + (both ? slot * 128 : part * 128) + r;
        o = p.cut_o + at * DV;
        ml = p.cut_ml + at * 2;
      }
      if (live) *reinterpret_cast<float2*>(ml) = make_float2(m_run - kBias, l_run);
      if (tiles > 0) {
        const uint32_t ob = tmem + lane_off + S::kTmemO + (S::kSlots == 2 ? slot * DV : 0);
        const float unit = pow2(v_ref - 11);
#pragma unroll
        for (int c = 0; c < DV / 32; ++c) {
          uint32_t rr[32];
          tmem_ld32(ob + c * 32, rr);
          tmem_ld_wait();
          if (live)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(rr[8 * i + e]) * unit;
              float4* dst = reinterpret_cast<float4*>(o + c * 32 + i * 8);
              dst[0] = make_float4(f[0], f[2], f[4], f[6]);
              dst[1] = make_float4(f[1], f[3], f[5], f[7]);
            }
        }
      }
      tc_fence_before();
      ++pieces;
    }
  }
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------- the join
// A thread takes four dims of a row: the parts of the prefix, in the order of the runs,
// and the request's own tokens.
template <bool BF16, int DV>
__global__ void __launch_bounds__(256) attn_kv_shared_join_kernel(const __grid_constant__ SharedParams p, int most_runs) {
  constexpr int kLanes = DV / 4, kRows = 256 / kLanes;
  const int64_t all = (int64_t)p.batch * p.c.heads * p.rows;
  const int d4 = threadIdx.x % kLanes;
  const ShRuns runs(*p.total_units, most_runs);
  for (int64_t at = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes; at < all; at += (int64_t)gridDim.x * kRows) {
    const int b = (int)(at / (p.c.heads * p.rows)), in = (int)(at - (int64_t)b * p.c.heads * p.rows);
    const int head = in / p.rows, rest = in - head * p.rows;
    const int qi = (int)p.by_group.div(rest), qh = head * p.group + rest - qi * p.group;
    const int64_t own = ((int64_t)b * p.seqlen_q + qi) * p.heads_q + qh;
    const int64_t lse_at = ((int64_t)b * p.heads_q + qh) * p.seqlen_q + qi;
    float4 acc = *reinterpret_cast<const float4*>(p.own_o + own * DV + d4 * 4);
    float lse = p.own_lse[lse_at];
    const int g = p.group_of[b];
    if (g >= 0) {
      const ShGroup info = ((const ShGroup*)p.group_info)[g];
      const int key_tiles = sh_key_tiles(p, info), row_tiles = sh_row_tiles(p, info);
      const long long row = (long long)(b - info.first) * p.rows + rest;
      const int rt = (int)(row / p.row_tile), r = (int)(row - (long long)rt * p.row_tile);
      const long long left = (long long)info.members * p.rows - (long long)rt * p.row_tile;
      const int parts = p.row_tile == 256 && left <= 128 ? 2 : 1;
      const long long u = info.unit0 + ((long long)head * row_tiles + rt) * key_tiles;
      const int k0 = runs.of(u), k1 = runs.of(u + key_tiles - 1);
      float mx = lse * 1.4426950408889634f, sum = 1.0f;
      auto add = [&](const float* o, const float* ml) {
        const float2 s = *reinterpret_cast<const float2*>(ml);
        if (s.y == 0.0f) return;  // a part without tiles
        const float4 y = *reinterpret_cast<const float4*>(o + d4 * 4);
        const float to = fmaxf(mx, s.x), f = ex2(s.x - to), a = ex2(mx - to);
        mx = to;
        sum = fmaf(sum, a, s.y * f);
        acc.x = fmaf(acc.x, a, y.x * f), acc.y = fmaf(acc.y, a, y.y * f);
        acc.z = fmaf(acc.z, a, y.z * f), acc.w = fmaf(acc.w, a, y.w * f);
      };
      for (int part = 0; part < parts; ++part) {
        if (k0 == k1) {
          const int64_t i = part * all + at;
          add(p.row_o + i * DV, p.row_ml + i * 2);
        } else {
#pragma unroll 4
          for (int k = k0; k <= k1; ++k) {
            const int64_t i = ((int64_t)k * 2 + (k == k0 ? 1 : 0)) * p.row_tile + part * 128 + r;
            add(p.cut_o + i * DV, p.cut_ml + i * 2);
          }
        }
      }
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
  k<<<num_sms, kThreads, S::kSmem, st>>>(p);
  return cudaGetLastError();
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
  const int64_t rows = (int64_t)p.batch * p.c.heads * p.rows, per = 256 / (p.c.d_v / 4);
  const unsigned blocks = (unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)num_sms * 8);
  switch (p.c.d_v) {
    case 64: attn_kv_shared_join_kernel<BF16, 64><<<blocks, 256, 0, st>>>(p, num_sms); break;
    case 128: attn_kv_shared_join_kernel<BF16, 128><<<blocks, 256, 0, st>>>(p, num_sms); break;
    default: attn_kv_shared_join_kernel<BF16, 256><<<blocks, 256, 0, st>>>(p, num_sms); break;
  }
  return cudaGetLastError();
}

}  // namespace

void shared_tiles(int d_v, int& row_tile, int& key_tile) {
  row_tile = d_v > 128 ? 128 : 256;
  key_tile = d_v > 128 ? 64 : 128;
}
size_t shared_group_bytes() { return sizeof(ShGroup); }

cudaError_t launch_kv4_shared_prefix(const SharedParams& p, bool bf16, int num_sms, cudaStream_t st) {
  attn_kv_shared_plan_kernel<<<1, 1024, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return bf16 ? sh_dims<true>(p, num_sms, st) : sh_dims<false>(p, num_sms, st);
}
cudaError_t launch_kv4_shared_join(const SharedParams& p, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? sh_join<true>(p, num_sms, st) : sh_join<false>(p, num_sms, st);
}

}  // namespace attn
