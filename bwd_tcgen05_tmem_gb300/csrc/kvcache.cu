// kvcache.cu -- the cache that attention over 4-bit keys and values reads:
//   * attn_kv_plan_kernel: where the new tokens of a step go (pages from a free
//     list, block-table entries, slots, positions, prefix sums);
//   * attn_kv_write_kernel / attn_kv_read_kernel: rows into the cache and back.
//
// A row of d elements (one token, one kv head) is held as d codes of 4 bits and
// d / 32 bf16 scales:  s = bf16(max|x| / 7) over 32 neighbours,
// c = clamp(round(x / s), -7, 7) + 8,  value = (c - 8) s.
// The codes lie in the order in which the lanes of attn_kv_decode_kernel use
// them, so its shared-memory reads are whole vectors (G = d / 32):
//   K row: word c * G + g      holds dims 32 g + 8 c .. + 7   (c < 4)
//   V row: half-word r * G + g holds dims 32 g + 4 r .. + 3   (r < 8)
// lowest nibble first.
#include <algorithm>

#include "kcommon.cuh"
#include "kv.h"

namespace attn {

// ----------------------------------------------------------------- page plan
// Every block adds up the whole batch by itself (the lengths are a few
// kilobytes that stay in L2, and a second launch would cost more than the
// sums): each thread takes a run of neighbouring requests, the runs' sums are
// scanned, and the prefix sums of the tokens and of the new pages stay in
// shared memory, with what each request holds.  Then each block writes its
// share of the rows: the request by binary search, its page from the table or,
// where the page is new, from the free list (so no block waits for another's
// table entries).
// Latency bounds it.  Measured on a GB300 (graph replays): 64 requests of one
// new token 3.5 us (a launch); 1021 requests of up to 500 new tokens 11.4 us, most of it
// the sums that every block makes and the searches.
constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) attn_kv_plan_kernel(
    const __grid_constant__ PlanParams p) {
  extern __shared__ int sm[];
  int* cu = sm;                   // [batch + 1] tokens before a request
  int* pg = cu + p.batch + 1;     // [batch + 1] new pages before it
  int* held_by = pg + p.batch + 1;  // [batch] tokens it holds
  __shared__ int wsum[2][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.page_shift;
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  const int head = p.free_head ? *p.free_head : 0;
  bool bad = false;
  int nt = 0, np = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    // what request b holds and what it gets; one whose lengths are negative or
    // longer than its table row counts as empty
    int c = p.ctx[b], f = p.fresh[b];
    const bool ok = c >= 0 && f >= 0 && (int64_t)c + f <= (int64_t)p.cols << p.page_shift;
    if (!ok) bad = true, c = f = 0;
    cu[b] = f;
    held_by[b] = c;
    pg[b] = p.free_pages ? ((c + f + P - 1) >> p.page_shift) - ((c + P - 1) >> p.page_shift) : 0;
    nt = (int)min((unsigned)nt + (unsigned)f, (unsigned)INT32_MAX);
    np += pg[b];
  }
  // exclusive prefix of the runs; sums past 2^31 - 1 stay there
  int st = nt, sp = np;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, st, o), c = __shfl_up_sync(0xffffffffu, sp, o);
    if (lane >= o) st = (int)min((unsigned)st + (unsigned)a, (unsigned)INT32_MAX), sp += c;
  }
  if (lane == 31) wsum[0][warp] = st, wsum[1][warp] = sp;
  __syncthreads();
  int ot = 0, op = 0;
  for (int w = 0; w < warp; ++w) {
    ot = (int)min((unsigned)ot + (unsigned)wsum[0][w], (unsigned)INT32_MAX);
    op += wsum[1][w];
  }
  // (sums of the requests before this thread's, not differences: those that
  // stay at 2^31 - 1 could not be taken back)
  int rt = __shfl_up_sync(0xffffffffu, st, 1), rp = __shfl_up_sync(0xffffffffu, sp, 1);
  if (lane == 0) rt = rp = 0;
  rt = (int)min((unsigned)ot + (unsigned)rt, (unsigned)INT32_MAX);
  rp += op;
  for (int b = b0; b < b1; ++b) {
    const int f = cu[b], need = pg[b];
    cu[b] = rt;
    pg[b] = rp;
    rt = (int)min((unsigned)rt + (unsigned)f, (unsigned)INT32_MAX);
    rp += need;
  }
  if (tid == kPlanThreads - 1) {  // (without requests of its own it holds the totals too)
    cu[p.batch] = rt;
    pg[p.batch] = rp;
    if (rt > p.rows) bad = true;
    if (p.free_pages && (head < 0 || (int64_t)head + rp > p.n_free)) bad = true;
  }
  if (bad && blockIdx.x == 0 && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
  __syncthreads();
  // a page of the free list, or -1
  auto page_of = [&](int i) {
    const int64_t at = (int64_t)head + i;
    int page = head >= 0 && at < p.n_free ? p.free_pages[at] : -1;
    if ((unsigned)page >= (unsigned)p.num_pages) page = -1;
    return page;
  };
  // (unsigned: the last step of the loops below may pass 2^31 - 1)
  const uint32_t gtid = blockIdx.x * kPlanThreads + tid, gn = gridDim.x * kPlanThreads;
  for (uint32_t b = gtid; b < (uint32_t)p.batch; b += gn) {
    const int c = held_by[b];
    p.cu[b] = cu[b];
    const int f = p.fresh[b];
    const bool ok = p.ctx[b] == c && f >= 0 && (int64_t)c + f <= (int64_t)p.cols << p.page_shift;
    p.seq[b] = ok ? c + f : 0;
  }
  // the last request whose prefix sum is <= x
  auto request_of = [&](const int* sums, int x) {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  const int new_pages = pg[p.batch];
  for (uint32_t i = gtid; i < (uint32_t)new_pages; i += gn) {
    const int b = request_of(pg, (int)i), held = (held_by[b] + P - 1) >> p.page_shift;
    const int page = page_of((int)i);
    p.table[(int64_t)b * p.table_stride + held + ((int)i - pg[b])] = page;
    if (page < 0 && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
  }
  if (gtid == 0) {
    p.cu[p.batch] = cu[p.batch];
    if (p.free_head_out) *p.free_head_out = (int)min((int64_t)head + pg[p.batch], (int64_t)INT32_MAX);
  }
  const int total = min(cu[p.batch], p.rows);
#pragma unroll 2
  for (uint32_t t = gtid; t < (uint32_t)p.rows; t += gn) {
    int pos = -1, slot = -1;
    if (t < (uint32_t)total) {
      const int lo = request_of(cu, (int)t);
      const int c = held_by[lo], held = (c + P - 1) >> p.page_shift;
      pos = c + ((int)t - cu[lo]);
      const int blk = pos >> p.page_shift;  // < cols, as the lengths are
      const int page = p.free_pages && blk >= held ? page_of(pg[lo] + blk - held)
                                                   : p.table[(int64_t)lo * p.table_stride + blk];
      if ((unsigned)page < (unsigned)p.num_pages)
        slot = (page << p.page_shift) + (pos & (P - 1));
      else if (p.status)
        atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    }
    p.pos[t] = pos;
    p.slots[t] = slot;
  }
}

cudaError_t launch_kv_plan(const PlanParams& p, int num_sms, cudaStream_t st) {
  const size_t smem = (size_t)(p.batch + 1) * 12;
  int64_t blocks = (int64_t)(p.rows > p.batch ? p.rows : p.batch) / (kPlanThreads * 2) + 1;
  // as many as run at once (200 KB of shared memory on an SM)
  const int64_t most = (int64_t)num_sms * std::min<int64_t>(8, std::max<int64_t>(200000 / (int64_t)(smem + 1024), 1));
  if (blocks > most) blocks = most;
  if (smem > 40000) {  // beyond what every kernel may take
    // (the largest call's, not this one's: calls of other threads share the limit)
    const cudaError_t e = cudaFuncSetAttribute(attn_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (kPlanMaxBatch + 1) * 12);
    if (e != cudaSuccess) return e;
  }
  attn_kv_plan_kernel<<<(unsigned)blocks, kPlanThreads, smem, st>>>(p);
  return cudaGetLastError();
}

// ----------------------------------------------------------------- rows in and out
// A thread takes 8 neighbouring elements (16 bytes) of a row: a quarter of a
// scale group, one word of codes.  The vectors of a token's K row and V row
// are numbered through (H d_qk / 8, then H d_v / 8); a thread keeps one number
// and goes from token to token, so that all it computes for a token is where
// its slot lies.  Where a token has fewer than 256 vectors a block takes
// several tokens at a time; where it has more, blockIdx.y picks 256 of them.
// Groups (4 lanes) and pairs of groups (8 lanes) never straddle a warp or a
// row, because d is a multiple of 64.
// Streams, bound by HBM if a word of codes costs few enough instructions: to
// read back takes about 80 a warp and vector, to store somewhat more (its issue
// slots are 60 to 70% taken).  Measured on a GB300 (graph replays, 32768 tokens, 8
// kv heads, 128 / 128): stored in 37 us in bf16 (172 MB, 4.6 TB/s, 68% of a plain
// copy's rate), 38 us in fp16, read back in 32 (5.4 TB/s, 80%) and 33 us; 64 tokens
// stored and read back 4.7 us, two launches.  Without the ring of copies: 155 us for
// both.
struct RowLane {
  bool live, is_k;
  int token;         // of the block's first pass
  int step;          // tokens of a pass over the whole grid
  int g, c, groups;  // scale group, quarter of it, groups of a row
  int64_t in_row;    // elements from a token's row base to the vector
  int64_t stride;    // elements between tokens
  int64_t head_row;  // head * page_size: rows of the cache before the head's, within a page
};

__device__ __forceinline__ RowLane row_lane(const KvRowsParams& p) {
  RowLane r;
  const uint32_t per = p.per_token.d;
  const uint32_t many = per >= 256u ? 1u : 256u / per;  // tokens of a block
  const uint32_t t = per >= 256u ? 0u : p.per_token.div(threadIdx.x);
  uint32_t v = per >= 256u ? blockIdx.y * 256u + threadIdx.x : threadIdx.x - t * per;
  r.live = t < many && v < per;
  r.token = (int)(blockIdx.x * many + t);
  r.step = (int)(gridDim.x * many);
  const uint32_t nk = (uint32_t)p.c.heads * p.vec_k.d;
  r.is_k = v < nk;
  if (!r.is_k) v -= nk;
  const uint32_t vecs = r.is_k ? p.vec_k.d : p.vec_v.d;
  const uint32_t head = (r.is_k ? p.vec_k : p.vec_v).div(v), j = v - head * vecs;
  r.g = (int)(j >> 2);
  r.c = (int)(j & 3u);
  r.groups = (int)(vecs >> 2);
  r.in_row = (int64_t)head * (r.is_k ? p.k_h : p.v_h) + j * 8;
  r.stride = r.is_k ? p.k_t : p.v_t;
  r.head_row = (int64_t)head * p.c.page_size;
  return r;
}

// Where a lane's word and its group's scale lie in the cache.
struct CacheLane {
  uint8_t* codes;     // of row 0 of the lane's head in page 0
  uint8_t* scales;
  uint32_t page_codes, page_scales;  // bytes of a page (below 2^31: 2^16 heads, 2^8 rows, 2^7 bytes)
  uint32_t row_codes, row_scales;    // of a row
  __device__ __forceinline__ uint32_t* word(const Kv4& c, int slot) const {
    return reinterpret_cast<uint32_t*>(codes + (uint64_t)(uint32_t)(slot >> c.page_shift) * page_codes +
                                       (uint32_t)(slot & (c.page_size - 1)) * row_codes);
  }
  __device__ __forceinline__ uint16_t* scale(const Kv4& c, int slot) const {
    return reinterpret_cast<uint16_t*>(scales + (uint64_t)(uint32_t)(slot >> c.page_shift) * page_scales +
                                       (uint32_t)(slot & (c.page_size - 1)) * row_scales);
  }
};
__device__ __forceinline__ CacheLane cache_lane(const KvRowsParams& p, const RowLane& r, uint32_t odd) {
  CacheLane c;
  c.row_codes = (uint32_t)r.groups * 16u;
  c.row_scales = (uint32_t)r.groups * 2u;
  const uint32_t rows = (uint32_t)(p.c.heads * p.c.page_size);
  c.page_codes = rows * c.row_codes;
  c.page_scales = rows * c.row_scales;
  // word of the lane in a row (two half-words of one r for V)
  const int at = r.is_k ? r.c * r.groups + r.g : ((2 * r.c + (int)odd) * r.groups + (r.g & ~1)) / 2;
  c.codes = (r.is_k ? p.c.k_codes : p.c.v_codes) + r.head_row * c.row_codes + 4 * at;
  c.scales = (uint8_t*)((r.is_k ? p.c.k_scales : p.c.v_scales) + r.head_row * r.groups + r.g);
  return c;
}

// The two elements of a 16-bit pair, in FP32.
template <bool BF16>
__device__ __forceinline__ uint64_t pair_f32(uint32_t w) {
  if (BF16) return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f2_pack(f.x, f.y);
}

// The codes of 8 elements whose scale s is a normal number, without a division:
// the quotient is x * (1/s) corrected by its exact remainder (P. W. Markstein, IBM
// Journal of Research and Development 34, 1990).  A quotient that
// lies midway between two codes has few bits, so the corrected product is that
// number itself and rounds to even as the division would; any other is at
// least 2^-13 away from the middle (x has 11 bits, s (2c + 1) / 2 has 12), 2^9
// times the error of the product.  |x / s| < 7.03, so nothing needs clamping.
// Adding 1.5 * 2^23 + 8 rounds to an integer: the sum's bits are 0x4B400000 +
// code; the eight are put together by multiply-adds modulo 2^32.
template <bool BF16>
__device__ __forceinline__ uint32_t codes_of(const uint4& x, float s) {
  float rs;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
  rs = fmaf(rs, fmaf(-s, rs, 1.0f), rs);
  const uint64_t r2 = f2_pack(rs, rs), s2 = f2_pack(-s, -s), magic = f2_pack(12582920.0f, 12582920.0f);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t word = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = pair_f32<BF16>(w[i]);
    uint64_t t = f2_mul(v, r2);
    t = f2_add(f2_fma(f2_fma(t, s2, v), r2, t), magic);
    float lo, hi;
    f2_unpack(t, lo, hi);
    word += __float_as_uint(lo) << (8 * i);
    word += __float_as_uint(hi) << (8 * i + 4);
  }
  return word;
}

// The same for scales below the normal range (and for zero): by division.
template <bool BF16>
__device__ __noinline__ uint32_t tiny_codes_of(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3,
                                               float s) {
  uint32_t word = 0x88888888u;  // codes of zeros
  if (s > 0.0f) {
    word = 0u;
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = e < 2 ? w0 : e < 4 ? w1 : e < 6 ? w2 : w3;
      const float v = Pack<BF16>::to_f((uint16_t)(w >> (16 * (e & 1))));
      const float t = rintf(__fdiv_rn(v, s));
      word |= (uint32_t)((int)fminf(fmaxf(t, -7.0f), 7.0f) + 8) << (4 * e);
    }
  }
  return word;
}

// Rows come through a ring of asynchronous copies, kRing times kU tokens deep; a
// thread copies and reads its own vectors alone.  kU tokens at a time share what
// a pass of the loop costs and hide each other's exchanges (1: 76 us, 2: 67 us, 3:
// 66 us, 4: 70 us for 32768 tokens stored and read back).
template <bool BF16>
__global__ void __launch_bounds__(256, 4) attn_kv_write_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int kRing = 3, kU = 3;
  __shared__ uint4 ring[kRing][kU][256];
  const RowLane r = row_lane(p);
  const uint32_t odd = (uint32_t)(threadIdx.x >> 2) & 1u;  // odd group of a pair
  const CacheLane at = cache_lane(p, r, odd);
  const int64_t src_step = (int64_t)r.step * r.stride * 2;
  const char* src = (const char*)((const uint16_t*)(r.is_k ? p.k : p.v) + r.in_row + (int64_t)r.token * r.stride);
  // tokens of this thread that are still to copy, and to store
  int to_copy = r.live && r.token < p.tokens ? (p.tokens - r.token + r.step - 1) / r.step : 0, left = to_copy;
  const uint32_t my = smem_u32(&ring[0][0][threadIdx.x]);
  auto copy = [&](int s) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (u < to_copy)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(my + (s * kU + u) * 4096),
                     "l"((uint64_t)__cvta_generic_to_global(src)) : "memory");
      src += src_step;
    }
    to_copy -= kU;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) copy(i);
  // slots are looked up one group ahead
  const int32_t* slot_at = p.slots + r.token;
  int next_slot[kU];
  auto look_up = [&](int n) {
#pragma unroll
    for (int u = 0; u < kU; ++u) next_slot[u] = u < n ? __ldg(slot_at + (int64_t)u * r.step) : -1;
    slot_at += (int64_t)kU * r.step;
  };
  look_up(left);
  int s = 0;
  // the lanes of a warp stay together: they exchange words
  for (; __any_sync(0xffffffffu, left > 0); left -= kU) {
    copy((s + kRing - 1) % kRing);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    int slot[kU];
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      slot[u] = next_slot[u];
      x[u] = make_uint4(0x3c003c00u, 0u, 0u, 0u);  // (zeros would take the slow way below)
      if (u < left) x[u] = ring[s][u][threadIdx.x];
    }
    look_up(left - kU);
    s = (s + 1) % kRing;
    uint32_t word[kU];
    uint16_t sbits[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // max|x| of the group of 32: the bit patterns of magnitudes are ordered,
      // infinities and NaN above all finite ones
      uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                            __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = max(m & 0xffffu, m >> 16);
      // max / 7 as the division rounds it: the product corrected by its remainder
      const float amax = Pack<BF16>::to_f((uint16_t)m);
      float q = amax * (1.0f / 7.0f);
      q = fmaf(fmaf(-q, 7.0f, amax), 1.0f / 7.0f, q);
      __nv_bfloat16 sb = __float2bfloat16_rn(q);
      sbits[u] = __bfloat16_as_ushort(sb);
      word[u] = codes_of<BF16>(x[u], __bfloat162float(sb));
      if (amax < 1e-29f) {  // zeros, and numbers so small that 1 / s or a remainder is not normal
        sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
        sbits[u] = __bfloat16_as_ushort(sb);
        word[u] = tiny_codes_of<BF16>(x[u].x, x[u].y, x[u].z, x[u].w, __bfloat162float(sb));
      } else if (m >= (BF16 ? 0x7f80u : 0x7c00u)) {  // a group with an infinity or a NaN: NaN
        sbits[u] = 0x7fffu;
        word[u] = 0x88888888u;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // V rows: two neighbouring groups exchange halves, so that each lane
      // holds the half-words (r, g), (r, g + 1) of one word
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? word[u] & 0xffffu : word[u] >> 16, 4);
      if (slot[u] < 0) continue;
      if ((slot[u] >> p.c.page_shift) >= p.c.num_pages) {
        if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
        continue;
      }
      if (!r.is_k) word[u] = odd ? (other | (word[u] & 0xffff0000u)) : ((word[u] & 0xffffu) | (other << 16));
      *at.word(p.c, slot[u]) = word[u];
      if (r.c == 0) *at.scale(p.c, slot[u]) = sbits[u];
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The values of a word's 8 codes: (c - 8) s, rounded once.
template <bool BF16>
__device__ __forceinline__ uint4 values_of(uint32_t w, uint16_t sbits) {
  uint32_t o[4];
  if (BF16) {
    // a product of a code (exact) and a bf16 scale, in bf16: one rounding
    const __nv_bfloat162 s = __nv_bfloat162(__ushort_as_bfloat16(sbits), __ushort_as_bfloat16(sbits));
    const __nv_bfloat162 off = __nv_bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
    uint32_t q[4];  // codes n and n + 4
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      uint32_t y;
      asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xEA;" : "=r"(y) : "r"(w >> (4 * n)));  // 128 + code
      const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&y), off), s);
      q[n] = *reinterpret_cast<const uint32_t*>(&v);
    }
    o[0] = __byte_perm(q[0], q[1], 0x5410), o[1] = __byte_perm(q[2], q[3], 0x5410);
    o[2] = __byte_perm(q[0], q[1], 0x7632), o[3] = __byte_perm(q[2], q[3], 0x7632);
  } else {
    const float s = __uint_as_float((uint32_t)sbits << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(0x4b000000u | ((w >> (8 * i)) & 15u)) - 8388616.0f;
      const float hi = __uint_as_float(0x4b000000u | ((w >> (8 * i + 4)) & 15u)) - 8388616.0f;
      o[i] = Pack<BF16>::two(lo * s, hi * s);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// kU tokens at a time: while their values are computed, the codes of the next
// kU are on their way, and the slots of those after them.
template <bool BF16>
__global__ void __launch_bounds__(256, 4) attn_kv_read_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int kU = 4;
  const RowLane r = row_lane(p);
  const uint32_t odd = (uint32_t)(threadIdx.x >> 2) & 1u;
  const CacheLane at = cache_lane(p, r, odd);
  uint16_t* dst = (uint16_t*)(r.is_k ? p.k : p.v) + r.in_row + (int64_t)r.token * r.stride;
  const int64_t dst_step = (int64_t)r.step * r.stride;
  int slot[kU], slot1[kU], slot2[kU];  // of this group of tokens, the next, the one after
  uint32_t word[kU], word1[kU];
  uint16_t sc[kU], sc1[kU];
  auto slots = [&](int t0, int (&s)[kU]) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t t = (int64_t)t0 + (int64_t)u * r.step;
      s[u] = r.live && t < p.tokens ? __ldg(p.slots + t) : -1;
    }
  };
  auto codes = [&](int (&s)[kU], uint32_t (&w)[kU], uint16_t (&c)[kU]) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      w[u] = 0u;
      c[u] = 0;
      if (s[u] >= 0 && (s[u] >> p.c.page_shift) >= p.c.num_pages) {
        if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
        s[u] = -1;
      }
      if (s[u] >= 0) w[u] = *at.word(p.c, s[u]), c[u] = *at.scale(p.c, s[u]);
    }
  };
  const int group = r.step * kU;
  slots(r.token, slot);
  slots(r.token + group, slot1);
  codes(slot, word, sc);
  for (int t0 = r.token; __any_sync(0xffffffffu, r.live && t0 < p.tokens); t0 += group) {
    slots(t0 + 2 * group, slot2);
    codes(slot1, word1, sc1);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // a V lane of the even group holds (r, g), (r, g + 1) for r = 2c, one of
      // the odd group those for r = 2c + 1
      uint32_t w = word[u];
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w & 0xffffu : w >> 16, 4);
      if (!r.is_k) w = odd ? (other | (w & 0xffff0000u)) : ((w & 0xffffu) | (other << 16));
      if (slot[u] >= 0) *reinterpret_cast<uint4*>(dst) = values_of<BF16>(w, sc[u]);
      dst += dst_step;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) slot[u] = slot1[u], slot1[u] = slot2[u], word[u] = word1[u], sc[u] = sc1[u];
  }
}

namespace {
dim3 rows_grid(const KvRowsParams& p, int num_sms) {
  const uint32_t per = p.per_token.d;
  const int64_t many = per >= 256u ? 1 : 256u / per;
  const unsigned y = (per + 255u) / 256u;
  int64_t x = (p.tokens + many - 1) / many;
  const int64_t cap = std::max<int64_t>((int64_t)num_sms * 4 / y, 1);
  if (x > cap) x = cap;
  return dim3((unsigned)x, y);
}
}  // namespace

cudaError_t launch_kv4_write(const KvRowsParams& p, bool bf16, int num_sms, cudaStream_t st) {
  const dim3 b = rows_grid(p, num_sms);
  if (bf16)
    attn_kv_write_kernel<true><<<b, 256, 0, st>>>(p);
  else
    attn_kv_write_kernel<false><<<b, 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const KvRowsParams& p, bool bf16, int num_sms, cudaStream_t st) {
  const dim3 b = rows_grid(p, num_sms);
  if (bf16)
    attn_kv_read_kernel<true><<<b, 256, 0, st>>>(p);
  else
    attn_kv_read_kernel<false><<<b, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
