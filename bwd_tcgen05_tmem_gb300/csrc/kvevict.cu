// kvevict.cu -- eviction from the 4-bit cache: of a sequence longer than its
// budget, each kv head keeps `keep` tokens, the first ones, the last ones and of
// those between the ones with the largest weights, and its rows move together.
//
// One cluster of blocks works on one (sequence, kv head):
//   * the border: the room-th largest weight, by a radix selection over the bits of
//     the weights (as whole numbers they are ordered; 10, 8, 7 and 7 bits at a time).
//     Each block counts its slice of the candidates in shared memory, the blocks add
//     up each other's counts over the cluster's distributed shared memory;
//   * the list: every candidate above the border stays, and of those on it the first
//     ones.  Blocks count theirs, exchange the counts, and write `kept` in order;
//   * the rows: row i becomes what row kept[i] >= i was.  Rows are taken in rounds of
//     ascending i: all blocks copy a round's rows into shared memory, meet at the
//     cluster's barrier, and only then write.  What later rounds read lies behind
//     what earlier rounds write, so the next round's rows are on their way meanwhile.
// Nothing is kept in memory between the steps but the list; rows in front of the
// first evicted token do not move.
//
// What bounds it: the rows' bytes, read and written, once behind the other.  64 x 4160
// tokens of 8 kv heads of 128 / 128 cut down to 4096, one GB300: 133 us for 629 MB, 70 %
// of what a copy reaches (a block of 1024 threads an SM, a scan for every 512
// candidates and fenced barriers in the rounds took 214); 8 x 65536 to 32768 175 us for
// 640 MB; 16 x 32768 to 4096 80 us, where the selection is half of the time; one request of
// 1087 tokens 19 us: four counting passes, the list and two rounds one after the other.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kcommon.cuh"
#include "kv.h"
#include "kvtile.cuh"

namespace attn {

namespace cg = cooperative_groups;

namespace {
// Blocks of an SM: as many as their rows and counts leave room for (16 x 32768 tokens to 4096
// 80 us, with three 178; the block of 1024 threads that the head names has the SM to itself).
constexpr int kThreads = 256, kWarps = kThreads / 32, kBlocks = 4;
constexpr int kPasses = 4, kBins = 1536;  // of the selection: 10, 8, 7 and 7 bits; their counts
constexpr int kMaxCluster = 8;
// Candidates of a block whose weights stay in shared memory: 8 x 65536 tokens take 175 us,
// with none 200.  11264 leave room for three blocks an SM (252).
constexpr int kKeys = 8192;
constexpr int kAhead = 4;  // candidates that a thread loads together
constexpr int kStage = 19456;  // bytes of a round's rows of a block, at most
// Candidates of a block, of which fewer are not worth another block's barriers: one
// request of 1087 tokens takes 25 us with 2048, 21 with 512, 19 with 256, 19 with 128.
constexpr int kMinSlice = 256;

// A weight as a number whose order is the weights': NaN below all, -0 like 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

template <int N>
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    copy16(dst, src);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"((uint64_t)__cvta_generic_to_global(src)),
                 "n"(N)
                 : "memory");
}

// Inclusive sums over the block of two counts (all threads); the totals are everybody's.
__device__ __forceinline__ int2 block_scan(int2 x, int2* s_warp, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y0 = __shfl_up_sync(0xffffffffu, x.x, o), y1 = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) x.x += y0, x.y += y1;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int2 y = s_warp[w];
    if (w < warp) x.x += y.x, x.y += y.y;
    total.x += y.x, total.y += y.y;
  }
  return x;
}
}  // namespace

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.seq_lens[b], most = min(p.cols << p.c.page_shift, p.capacity);
  if (n >= 0 && n <= most) return n;
  if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
  return 0;
}
__device__ __forceinline__ int pages_of(const EvictParams& p, int n) { return (n + p.c.page_size - 1) >> p.c.page_shift; }
// Pages of a sequence that an eviction leaves without tokens: columns from .. from + count - 1.
// (One that holds a protected token is not among them, though that token goes where more
// are protected than stay: other sequences may hold the page too.)
struct PagesGone {
  int from, count;
};
__device__ __forceinline__ PagesGone pages_gone(const EvictParams& p, int b, int n) {
  if (n <= p.keep) return {0, 0};
  const int from = pages_of(p, p.first ? max(p.keep, min(p.first[b], n)) : p.keep);
  return {from, pages_of(p, n) - from};
}

// The new length of sequence b, and its pages for the free list, in front of the
// pages taken: those of all sequences in order, each one's in order of its columns.
__device__ void evict_lists(const EvictParams& p, int b, int n, int2* s_warp) {
  if (threadIdx.x == 0) p.seq_out[b] = min(n, p.keep);
  if (!p.free_head) return;
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < p.batch; i += kThreads) {
    const int g = pages_gone(p, i, evict_len(p, i)).count;
    all += g;
    if (i < b) before += g;
  }
  int2 sums;
  block_scan(make_int2(all, before), s_warp, sums);
  const int n_all = sums.x, n_before = sums.y;
  const int head = *p.free_head;
  const bool fits = head >= n_all && head <= p.n_free;
  if (threadIdx.x == 0 && b == 0) *p.free_head_out = fits ? head - n_all : head;
  if (!fits) {
    if (threadIdx.x == 0 && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    return;
  }
  const int32_t* row = p.table + (int64_t)b * p.table_stride;
  const PagesGone gone = pages_gone(p, b, n);
  for (int i = threadIdx.x; i < gone.count; i += kThreads) {
    int page = row[gone.from + i];
    if ((unsigned)page >= (unsigned)p.c.num_pages) {
      page = -1;
      if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    }
    p.free_pages[head - n_all + n_before + i] = page;
  }
}

template <int DQK, int DV>
struct EvictShape {
  static constexpr int kCodes = (DQK + DV) / 2 / 16;   // 16-byte vectors of a row's codes
  // the widest pieces of a row's scales (DQK / 16 and DV / 16 bytes) that their alignment allows
  static constexpr int kPieceK = DQK / 16 % 16 == 0 ? 16 : DQK / 16 % 8 == 0 ? 8 : 4;
  static constexpr int kPieceV = DV / 16 % 16 == 0 ? 16 : DV / 16 % 8 == 0 ? 8 : 4;
  static constexpr int kRow = kCodes * 16 + (DQK + DV) / 16 + 4;  // and its weight
  static constexpr int kMost = kStage / kRow / 32 * 32, kRows = kMost < 128 ? kMost : 128;  // of a block's round
  // where a round's rows lie, array by array: K's codes first
  static constexpr int kAtV = kRows * DQK / 2, kAtKs = kAtV + kRows * DV / 2, kAtVs = kAtKs + kRows * DQK / 16,
                       kAtW = kAtVs + kRows * DV / 16;
  static constexpr int kSelect = kBins * 4 + kKeys * 4;
  static constexpr int kSmem = 2 * kRows * kRow > kSelect ? 2 * kRows * kRow : kSelect;
};

template <int DQK, int DV>
__global__ void __launch_bounds__(kThreads, kBlocks) attn_kv_evict_kernel(const __grid_constant__ EvictParams p) {
  using S = EvictShape<DQK, DV>;
  extern __shared__ __align__(16) uint8_t smem[];  // counts and weights, then the rounds' rows
  int* hist = reinterpret_cast<int*>(smem);  // pass by pass
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + kBins * 4);
  __shared__ int2 s_warp[kWarps];
  __shared__ int s_bin, s_above, s_first[kWarps];
  __shared__ int s_count[3];  // of this block's candidates: above the border, on it; the first that goes
  __shared__ long long s_src[3][S::kRows], s_dst[3][S::kRows];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // all blocks of the cluster, and what they have written
  auto meet = [&]() {
    if (C == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / C, b = item / p.c.heads, h = item - b * p.c.heads;
  const int n = evict_len(p, b);
  if (h == 0 && rank == 0) evict_lists(p, b, n, s_warp);
  const float* w = p.w + (int64_t)b * p.w_b + (int64_t)h * p.w_h;
  float* w_out = p.w_out + (int64_t)b * p.wo_b + (int64_t)h * p.wo_h;
  int32_t* kept = p.kept + ((int64_t)b * p.c.heads + h) * p.keep;
  const int all = C * kThreads, me = rank * kThreads + tid;
  if (n <= p.keep) {  // within the budget (the whole cluster)
    for (int64_t i = me; i < p.keep; i += all) kept[i] = i < n ? (int)i : -1;
    if (w_out != w)
      for (int i = me; i < n; i += all) w_out[i] = w[i];
    return;
  }
  const int first = p.first ? min(max(p.first[b], 0), p.keep) : 0;
  const int recent = min(p.recent, p.keep - first);
  const int room = p.keep - first - recent;       // for the tokens between
  const int m = n - first - recent;               // of those (more than room)
  const int per = ((m + C - 1) / C + 31) & ~31;   // of a block
  const int c0 = min(rank * per, m), mine = min(m - c0, per);
  const bool held = per <= kKeys;
  const float* wc = w + first + c0;
  auto key = [&](int i) { return held ? keys[i] : order_of(wc[i]); };

  // ---- the border
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  if (held)
    for (int i = tid; i < mine; i += kThreads) keys[i] = order_of(wc[i]);
  __syncthreads();
  uint32_t border = 0;  // its digits so far
  int need = room;      // of the candidates that share them
  constexpr int kShift[kPasses] = {22, 14, 7, 0};
  constexpr int kDigits[kPasses] = {1024, 256, 128, 128}, kFirst[kPasses] = {0, 1024, 1280, 1408};
  if (room > 0) {
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      int* mine_h = hist + kFirst[pass];
      for (int i0 = warp * 32; i0 < mine; i0 += kAhead * kThreads) {
        uint32_t k[kAhead];  // (loaded together: those that are not held come from far)
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int i = i0 + a * kThreads + lane;
          k[a] = i < mine ? key(i) : 0u;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int i = i0 + a * kThreads + lane;
          const bool in = i < mine && (pass == 0 || (k[a] >> kShift[pass - 1]) == (border >> kShift[pass - 1]));
          const int d = in ? (int)((k[a] >> kShift[pass]) & (kDigits[pass] - 1)) : -1;
          // (equal digits throughout, as of weights that are all alike, are one addition)
          const int d0 = __shfl_sync(0xffffffffu, d, 0);
          if (__all_sync(0xffffffffu, d == d0)) {
            if (lane == 0 && d0 >= 0) atomicAdd(&mine_h[d0], 32);
          } else if (in) {
            atomicAdd(&mine_h[d], 1);
          }
        }
      }
      meet();
      // every block adds up all blocks' counts; thread t takes digits from the top on
      constexpr int kEach = 1024 / kThreads;
      static_assert(kEach == 4, "a vector of counts, or one");
      const int each = kDigits[pass] == 1024 ? kEach : 1;
      const bool digits = tid * each < kDigits[pass];
      int cnt[kEach], sum = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) cnt[j] = 0;
      if (digits)
        for (int q = 0; q < C; ++q) {
          const int* h_q = C == 1 ? mine_h : cluster.map_shared_rank(mine_h, q);
          if (each == 4) {
            const int4 x = *reinterpret_cast<const int4*>(h_q + kDigits[pass] - 4 - tid * 4);
            cnt[0] += x.w, cnt[1] += x.z, cnt[2] += x.y, cnt[3] += x.x;
          } else {
            cnt[0] += h_q[kDigits[pass] - 1 - tid];
          }
        }
#pragma unroll
      for (int j = 0; j < kEach; ++j) sum += cnt[j];
      int2 total;
      int above = block_scan(make_int2(sum, 0), s_warp, total).x - sum;
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (j < each && digits) {
          if (above < need && above + cnt[j] >= need) s_bin = kDigits[pass] - 1 - (tid * each + j), s_above = above;
          above += cnt[j];
        }
      __syncthreads();
      border |= (uint32_t)s_bin << kShift[pass];
      need -= s_above;
      __syncthreads();
    }
  } else {
    border = 0xffffffffu;  // (no weight's number)
  }
  // ---- the list: `need` of the candidates on the border stay, the first ones.  A thread
  // takes candidates in a row (an odd number of them: no two lanes' lie in one bank); of
  // those that are not held a warp does, whole lines at a time.
  const int run = held ? ((mine + kThreads - 1) / kThreads) | 1 : ((mine + kThreads - 1) / kThreads) * 32;
  const int i0 = min((held ? tid : warp) * run, mine), i1 = min(i0 + run, mine), lane0 = held ? 0 : lane, next = held ? 1 : 32;
  int2 own = make_int2(0, 0), sums;  // above the border, on it
#pragma unroll 4
  for (int i = i0 + lane0; i < i1; i += next) {
    const uint32_t k = key(i);
    own.x += k > border;
    own.y += k == border;
  }
  const int2 upto = block_scan(own, s_warp, sums);
  if (tid == 0) s_count[0] = sums.x, s_count[1] = sums.y;
  meet();
  int to = first, on_before = 0;
  for (int q = 0; q < rank; ++q) {
    const int* s = cluster.map_shared_rank(s_count, q);
    to += s[0] + min(max(need - on_before, 0), s[1]);
    on_before += s[1];
  }
  int gone = INT32_MAX;  // the first that goes, of this thread's
  const int room0 = max(need - on_before, 0), last = p.keep - recent;  // for the block's on the border; the list's end
  // (The list is full early only if another kernel changes the weights meanwhile.)
  if (!held) {
    int above0 = __shfl_sync(0xffffffffu, upto.x - own.x, 0), on0 = __shfl_sync(0xffffffffu, upto.y - own.y, 0);
    const uint32_t before = (1u << lane) - 1u;
    for (int i = i0; i < i1; i += kAhead * 32) {
      uint32_t k[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) k[a] = i + a * 32 + lane < i1 ? key(i + a * 32 + lane) : 0u;
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int j = i + a * 32 + lane;
        const bool there = j < i1;
        const uint32_t above = __ballot_sync(0xffffffffu, there && k[a] > border);
        const uint32_t on = __ballot_sync(0xffffffffu, there && k[a] == border);
        const int on_here = on0 + __popc(on & before), at = to + above0 + __popc(above & before) + min(on_here, room0);
        const bool stay = k[a] > border || (k[a] == border && on_here < room0);
        if (there && !stay) gone = min(gone, first + c0 + j);
        if (there && stay && at < last) kept[at] = first + c0 + j;
        above0 += __popc(above), on0 += __popc(on);
      }
    }
  } else {
    const int on0 = upto.y - own.y;  // of the block's, before this thread
    int at = to + upto.x - own.x + min(on0, room0), left = max(room0 - on0, 0);
    for (int i = i0; i < i1; i += kAhead) {
      uint32_t k[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) k[a] = i + a < i1 ? key(i + a) : 0u;
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (i + a >= i1) break;
        const bool on = k[a] == border, stay = k[a] > border || (on && left > 0);
        left -= on;
        if (!stay)
          gone = min(gone, first + c0 + i + a);
        else if (at < last)
          kept[at++] = first + c0 + i + a;
      }
    }
  }
  for (int i = me; i < first; i += all) kept[i] = i;
  for (int i = me; i < recent; i += all) kept[p.keep - recent + i] = n - recent + i;
  gone = (int)__reduce_min_sync(0xffffffffu, (unsigned)gone);
  if (lane == 0) s_first[warp] = gone;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kWarps; ++i) gone = min(gone, s_first[i]);
    s_count[2] = gone;
  }
  meet();  // (the list too)
  int start = INT32_MAX;  // rows in front of it stay where they are
  for (int q = 0; q < C; ++q) start = min(start, cluster.map_shared_rank(s_count, q)[2]);
  start = min(start, p.keep);

  // ---- the rows
  const bool apart = w_out != w;
  if (apart)
    for (int i = me; i < start; i += all) w_out[i] = w[i];
  const int32_t* row = p.table + (int64_t)b * p.table_stride;
  auto slot_row = [&](int t) -> long long {  // of the cache's rows; -1: a page outside it
    const int page = row[t >> p.c.page_shift];
    if ((unsigned)page >= (unsigned)p.c.num_pages) {
      if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
      return -1;
    }
    return ((long long)page * p.c.heads + h) * p.c.page_size + (t & (p.c.page_size - 1));
  };
  // (of such weights the list may lack entries: any token of the sequence stands in)
  auto kept_at = [&](int i) { return (int)min((unsigned)__ldcg(kept + i), (unsigned)(n - 1)); };
  // where a round's rows come from and go to
  auto find = [&](int base, int slot) {
    for (int i = tid; i < S::kRows && base + i < p.keep; i += kThreads) {
      const int src = kept_at(base + i);
      // (a row that comes from or goes to a page outside the cache is not written)
      const long long from = slot_row(src), dst = slot_row(base + i);
      s_src[slot][i] = from;
      s_dst[slot][i] = from < 0 ? -1 : dst;
    }
  };
  // Pieces of N bytes of the rows' W bytes of one array: a thread keeps its piece and goes
  // from row to row.  f(piece's place in the array's row 0, in the round's rows, row).
  auto pieces = [&](auto width, auto piece, const void* array, int at, int rows, auto&& f) {
    constexpr int W = decltype(width)::value, N = decltype(piece)::value, kEach = W / N, kPer = kThreads / kEach;
    const int r0 = tid / kEach, u = tid - r0 * kEach;
    if (r0 >= kPer) return;
    uint8_t* const mine = (uint8_t*)array + u * N;
#pragma unroll 2
    for (int i = r0; i < rows; i += kPer) f(mine, at + i * W + u * N, i);
  };
  using std::integral_constant;
  auto arrays = [&](int rows, auto&& f) {
    pieces(integral_constant<int, DQK / 2>(), integral_constant<int, 16>(), p.c.k_codes, 0, rows, [&](uint8_t* a, int s, int i) { f(integral_constant<int, 16>(), integral_constant<int, DQK / 2>(), a, s, i); });
    pieces(integral_constant<int, DV / 2>(), integral_constant<int, 16>(), p.c.v_codes, S::kAtV, rows, [&](uint8_t* a, int s, int i) { f(integral_constant<int, 16>(), integral_constant<int, DV / 2>(), a, s, i); });
    pieces(integral_constant<int, DQK / 16>(), integral_constant<int, S::kPieceK>(), p.c.k_scales, S::kAtKs, rows, [&](uint8_t* a, int s, int i) { f(integral_constant<int, S::kPieceK>(), integral_constant<int, DQK / 16>(), a, s, i); });
    pieces(integral_constant<int, DV / 16>(), integral_constant<int, S::kPieceV>(), p.c.v_scales, S::kAtVs, rows, [&](uint8_t* a, int s, int i) { f(integral_constant<int, S::kPieceV>(), integral_constant<int, DV / 16>(), a, s, i); });
  };
  auto load = [&](int base, int buf, int slot) {
    const int rows = min(p.keep - base, S::kRows);
    const uint32_t st = smem_u32(smem) + buf * (S::kRows * S::kRow);
    for (int i = tid; i < rows; i += kThreads) copy_bytes<4>(st + S::kAtW + i * 4, w + kept_at(base + i));
    if (p.c.num_pages == 0) return;  // (else row 0 is read where there is none)
    arrays(rows, [&](auto bytes, auto width, uint8_t* array, int at, int i) {
      copy_bytes<decltype(bytes)::value>(st + at, array + max(s_src[slot][i], 0ll) * decltype(width)::value);
    });
  };
  auto store = [&](int base, int buf, int slot) {
    const int rows = min(p.keep - base, S::kRows);
    const uint8_t* st = smem + buf * (S::kRows * S::kRow);
    arrays(rows, [&](auto bytes, auto width, uint8_t* array, int at, int i) {
      using T = std::conditional_t<decltype(bytes)::value == 16, uint4, std::conditional_t<decltype(bytes)::value == 8, uint2, uint32_t>>;
      const long long to = s_dst[slot][i];
      if (to >= 0) *reinterpret_cast<T*>(array + to * decltype(width)::value) = *reinterpret_cast<const T*>(st + at);
    });
    for (int i = tid; i < rows; i += kThreads) w_out[base + i] = *reinterpret_cast<const float*>(st + S::kAtW + i * 4);
  };
  // (A cluster's blocks all take part in every round's barrier, with rows or without.)
  // While a round's rows are written the next one's are on their way, and where those after
  // them lie has been looked up.
  const int step = C * S::kRows;
  int base = start + rank * S::kRows;
  find(base, 0);
  __syncthreads();
  if (base < p.keep) load(base, 0, 0);
  copies_end();
  find(base + step, 1);
  __syncthreads();
  for (int round = start, buf = 0, slot = 0; round < p.keep; round += step, base += step, buf ^= 1) {
    const int slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot1 == 2 ? 0 : slot1 + 1;
    if (base + step < p.keep) load(base + step, buf ^ 1, slot1);
    copies_end();
    find(base + 2 * step, slot2);
    copies_wait<1>();
    __syncthreads();
    // (The rows have arrived, and no block needs to see what another one has written: the
    // cluster's barrier without its fences is enough.)
    if (C > 1) {
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    if (base < p.keep) store(base, buf, slot);
    __syncthreads();
    slot = slot1;
  }
  copies_wait<0>();
  meet();  // (no block leaves while others may read its counts)
}

namespace {
template <int DQK, int DV>
cudaError_t evict_launch(const EvictParams& p, int num_sms, cudaStream_t st) {
  using S = EvictShape<DQK, DV>;
  auto* k = attn_kv_evict_kernel<DQK, DV>;
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
  // as large a cluster as leaves all of them on the card at once, and its blocks enough to do
  const int64_t items = (int64_t)p.batch * p.c.heads;
  const int64_t most = std::min<int64_t>((int64_t)p.cols << p.c.page_shift, p.capacity);
  int c = kMaxCluster;
  while (c > 1 && (items * c > kBlocks * num_sms || most < (int64_t)c * kMinSlice)) c /= 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}
}  // namespace

cudaError_t launch_kv4_evict(const EvictParams& p, int num_sms, cudaStream_t st) {
  if (p.c.d_qk == 64 && p.c.d_v == 64) return evict_launch<64, 64>(p, num_sms, st);
  if (p.c.d_qk == 128 && p.c.d_v == 128) return evict_launch<128, 128>(p, num_sms, st);
  if (p.c.d_qk == 192 && p.c.d_v == 128) return evict_launch<192, 128>(p, num_sms, st);
  if (p.c.d_qk == 256 && p.c.d_v == 256) return evict_launch<256, 256>(p, num_sms, st);
  return cudaErrorNotSupported;
}

}  // namespace attn
