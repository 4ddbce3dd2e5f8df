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
#include "kcommon.cuh"
#include "kv.h"

namespace attn {

// ----------------------------------------------------------------- page plan
// Every block adds up the whole batch by itself (the lengths are a few
// kilobytes that stay in L2, and a second launch would cost more than the
// sums): each thread takes a run of neighbouring requests, the runs' sums are
// scanned, and the prefix sums of the tokens and of the new pages stay in
// shared memory.  Then each block writes its share of the rows: the request
// by binary search, its page from the table or, where the page is new, from
// the free list (so no block waits for another's table entries).
constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) attn_kv_plan_kernel(
    const __grid_constant__ PlanParams p) {
  extern __shared__ int sm[];
  int* cu = sm;                  // [batch + 1] tokens before a request
  int* pg = sm + p.batch + 1;    // [batch + 1] new pages before it
  __shared__ int wsum[2][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.page_shift;
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  bool bad = false;
  // what request b holds and what it gets; one whose lengths are negative or
  // longer than its table row counts as empty
  auto lengths = [&](int b, int& c, int& f) {
    c = p.ctx[b];
    f = p.fresh[b];
    const bool ok = c >= 0 && f >= 0 && (int64_t)c + f <= (int64_t)p.cols << p.page_shift;
    if (!ok) c = f = 0;
    return ok;
  };
  int nt = 0, np = 0;
  for (int b = b0; b < b1; ++b) {
    int c, f;
    bad |= !lengths(b, c, f);
    cu[b] = f;
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
  st = (int)min((unsigned)ot + (unsigned)st, (unsigned)INT32_MAX);
  sp += op;
  const int head = p.free_head ? *p.free_head : 0;
  int rt = st - nt, rp = sp - np;
  for (int b = b0; b < b1; ++b) {
    const int f = cu[b], need = pg[b];
    cu[b] = rt;
    pg[b] = rp;
    rt = (int)min((unsigned)rt + (unsigned)f, (unsigned)INT32_MAX);
    rp += need;
  }
  if (tid == kPlanThreads - 1) {
    cu[p.batch] = st;
    pg[p.batch] = sp;
    if (st > p.rows) bad = true;
    if (p.free_pages && (head < 0 || (int64_t)head + sp > p.n_free)) bad = true;
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
  const int gtid = blockIdx.x * kPlanThreads + tid, gn = gridDim.x * kPlanThreads;
  for (int b = gtid; b < p.batch; b += gn) {
    int c, f;
    lengths(b, c, f);
    p.cu[b] = cu[b];
    p.seq[b] = c + f;
    const int need = pg[b + 1] - pg[b], held = (c + P - 1) >> p.page_shift;
    for (int i = 0; i < need; ++i) {
      const int page = page_of(pg[b] + i);
      p.table[(int64_t)b * p.table_stride + held + i] = page;
      if (page < 0 && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    }
  }
  if (gtid == 0) {
    p.cu[p.batch] = cu[p.batch];
    if (p.free_head_out) *p.free_head_out = (int)min((int64_t)head + pg[p.batch], (int64_t)INT32_MAX);
  }
  const int total = min(cu[p.batch], p.rows);
  for (int t = gtid; t < p.rows; t += gn) {
    int pos = -1, slot = -1;
    if (t < total) {
      int lo = 0, hi = p.batch;  // the last request with cu <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
      }
      const int c = p.ctx[lo], held = (c + P - 1) >> p.page_shift;
      pos = c + t - cu[lo];
      const int blk = pos >> p.page_shift;  // < cols: lengths() looked
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
  int64_t blocks = (int64_t)(p.rows > p.batch ? p.rows : p.batch) / (kPlanThreads * 2) + 1;
  if (blocks > 2 * num_sms) blocks = 2 * num_sms;
  const size_t smem = (size_t)(p.batch + 1) * 8;
  if (smem > 40000) {  // beyond what every kernel may take
    const cudaError_t e = cudaFuncSetAttribute(
        attn_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  attn_kv_plan_kernel<<<(unsigned)blocks, kPlanThreads, smem, st>>>(p);
  return cudaGetLastError();
}

// ----------------------------------------------------------------- rows in and out
// A thread takes 8 neighbouring elements (16 bytes) of a row: a quarter of a
// scale group, one word of codes.  The vectors of a token's K row and V row
// are numbered through (H d_qk / 8, then H d_v / 8), so every lane works
// whatever the head dim is; groups (4 lanes) and pairs of groups (8 lanes)
// never straddle a warp or a row, because d is a multiple of 64.
struct RowAt {
  bool is_k;
  int head, j;  // kv head, vector within the row
};

__device__ __forceinline__ RowAt row_at(const KvRowsParams& p, uint32_t v) {
  RowAt r;
  const uint32_t nk = (uint32_t)p.c.heads * p.vec_k.d;
  r.is_k = v < nk;
  if (!r.is_k) v -= nk;
  r.head = (int)(r.is_k ? p.vec_k : p.vec_v).div(v);
  r.j = (int)(v - (uint32_t)r.head * (r.is_k ? p.vec_k.d : p.vec_v.d));
  return r;
}

// Row index of (slot, head) in the cache arrays.
__device__ __forceinline__ int64_t cache_row(const Kv4& c, int slot, int head) {
  const int page = slot >> c.page_shift, off = slot & (c.page_size - 1);
  return ((int64_t)page * c.heads + head) * c.page_size + off;
}

// Slot of token t: < 0 means "leave the row alone"; out of range is flagged.
__device__ __forceinline__ int slot_of(const KvRowsParams& p, uint32_t t) {
  const int s = p.slots[t];
  if (s >= 0 && (s >> p.c.page_shift) >= p.c.num_pages) {
    if (p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    return -1;
  }
  return s;
}

template <bool BF16>
__global__ void __launch_bounds__(256) attn_kv_write_kernel(const __grid_constant__ KvRowsParams p) {
  const uint32_t total = (uint32_t)p.tokens * p.per_token.d;  // < 2^31, checked at launch
  const uint32_t step = gridDim.x * 256u;
  constexpr int kU = 4;
  const int lane = threadIdx.x & 31;
  // whole warps stay in the loop: the lanes exchange words
  for (uint32_t base = blockIdx.x * 256u + (threadIdx.x & ~31u); base < total; base += step * kU) {
    uint4 x[kU];
    int64_t row[kU];
    RowAt at[kU];
    int d[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint64_t i64 = (uint64_t)base + (uint64_t)u * step + lane;
      row[u] = -1;
      d[u] = 64;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i64 < total) {
        const uint32_t i = (uint32_t)i64, t = p.per_token.div(i);
        at[u] = row_at(p, i - t * p.per_token.d);
        const int slot = slot_of(p, t);
        d[u] = at[u].is_k ? p.c.d_qk : p.c.d_v;
        if (slot >= 0) {
          const uint16_t* src =
              (const uint16_t*)(at[u].is_k ? p.k : p.v) +
              (int64_t)t * (at[u].is_k ? p.k_t : p.v_t) + (int64_t)at[u].head * (at[u].is_k ? p.k_h : p.v_h);
          x[u] = *(reinterpret_cast<const uint4*>(src) + at[u].j);
          row[u] = cache_row(p.c, slot, at[u].head);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // max|x| of the group of 32: the bit patterns of magnitudes are ordered,
      // infinities and NaN above all finite ones
      uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                            __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = max(m & 0xffffu, m >> 16);
      uint32_t word = 0x88888888u;  // codes of zeros
      uint16_t sbits = 0x7fffu;     // a group with an infinity or a NaN: NaN
      if (m < (BF16 ? 0x7f80u : 0x7c00u)) {
        const float amax = Pack<BF16>::to_f((uint16_t)m);
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
        sbits = __bfloat16_as_ushort(sb);
        float s = __bfloat162float(sb);
        if (s > 0.0f) {
          // tiny groups: scaled by a power of two, so that 1 / s stays finite
          const float f = s < 1e-30f ? 1.8446744e19f : 1.0f;  // 2^64
          s *= f;
          const float rs = __frcp_rn(s);
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          word = 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xe = f * Pack<BF16>::to_f((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
            // The quotient x / s: x * (1/s) corrected by its exact remainder.
            // A quotient that lies midway between two codes has few bits, so
            // the corrected product is that number itself and rounds to even
            // as the division would; any other is at least 2^-13 s away from
            // the middle (x has 11 bits, s (2c + 1) / 2 has 12), 2^10 times
            // the error of the product.
            float t = xe * rs;
            t = fmaf(fmaf(-t, s, xe), rs, t);
            const int c = (int)fminf(fmaxf(rintf(t), -7.0f), 7.0f) + 8;
            word |= (uint32_t)c << (4 * e);
          }
        }
      }
      const uint32_t odd = (uint32_t)(lane >> 2) & 1u;  // odd group of the pair
      // V rows: two neighbouring groups exchange halves, so that each lane
      // holds the half-words (r, g), (r, g + 1) of one word
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? word & 0xffffu : word >> 16, 4);
      if (row[u] < 0) continue;
      const int G = d[u] / 32, g = at[u].j >> 2, c = at[u].j & 3;
      if (at[u].is_k) {
        reinterpret_cast<uint32_t*>(p.c.k_codes + row[u] * (d[u] / 2))[c * G + g] = word;
      } else {
        const uint32_t pair = odd ? (other | (word & 0xffff0000u)) : ((word & 0xffffu) | (other << 16));
        const int r = 2 * c + (int)odd;
        reinterpret_cast<uint32_t*>(p.c.v_codes + row[u] * (d[u] / 2))[(r * G + (g & ~1)) / 2] = pair;
      }
      if (c == 0) (at[u].is_k ? p.c.k_scales : p.c.v_scales)[row[u] * G + g] = sbits;
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) attn_kv_read_kernel(const __grid_constant__ KvRowsParams p) {
  const uint32_t total = (uint32_t)p.tokens * p.per_token.d;
  const uint32_t step = gridDim.x * 256u;
  constexpr int kU = 4;
  const int lane = threadIdx.x & 31;
  for (uint32_t base = blockIdx.x * 256u + (threadIdx.x & ~31u); base < total; base += step * kU) {
    uint32_t word[kU];
    uint16_t sc[kU];
    uint4* dst[kU];
    bool is_k[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint64_t i64 = (uint64_t)base + (uint64_t)u * step + lane;
      dst[u] = nullptr;
      word[u] = 0u;
      sc[u] = 0;
      is_k[u] = true;
      if (i64 < total) {
        const uint32_t i = (uint32_t)i64, t = p.per_token.div(i);
        const RowAt at = row_at(p, i - t * p.per_token.d);
        const int slot = slot_of(p, t);
        is_k[u] = at.is_k;
        if (slot >= 0) {
          const int d = at.is_k ? p.c.d_qk : p.c.d_v, G = d / 32, g = at.j >> 2, c = at.j & 3;
          const int64_t row = cache_row(p.c, slot, at.head);
          const int wi = at.is_k ? c * G + g : ((2 * c + (g & 1)) * G + (g & ~1)) / 2;
          word[u] = reinterpret_cast<const uint32_t*>((at.is_k ? p.c.k_codes : p.c.v_codes) + row * (d / 2))[wi];
          sc[u] = (at.is_k ? p.c.k_scales : p.c.v_scales)[row * G + g];
          dst[u] = reinterpret_cast<uint4*>(
                       (uint16_t*)(at.is_k ? p.k : p.v) + (int64_t)t * (at.is_k ? p.k_t : p.v_t) +
                       (int64_t)at.head * (at.is_k ? p.k_h : p.v_h)) + at.j;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t odd = (uint32_t)(lane >> 2) & 1u;
      // a V lane of the even group holds (r, g), (r, g + 1) for r = 2c, one of
      // the odd group those for r = 2c + 1
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? word[u] & 0xffffu : word[u] >> 16, 4);
      if (!dst[u]) continue;
      const uint32_t w = is_k[u] ? word[u]
                         : odd   ? (other | (word[u] & 0xffff0000u))
                                 : ((word[u] & 0xffffu) | (other << 16));
      const float s = __uint_as_float((uint32_t)sc[u] << 16);
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (float)((int)((w >> (4 * e)) & 15u) - 8) * s;
      *dst[u] = make_uint4(Pack<BF16>::two(f[0], f[1]), Pack<BF16>::two(f[2], f[3]),
                           Pack<BF16>::two(f[4], f[5]), Pack<BF16>::two(f[6], f[7]));
    }
  }
}

namespace {
unsigned rows_blocks(const KvRowsParams& p, int num_sms) {
  const uint64_t total = (uint64_t)p.tokens * p.per_token.d;
  uint64_t blocks = (total + 255) / 256;
  const uint64_t cap = (uint64_t)num_sms * 8;
  if (blocks > cap) blocks = cap;
  return (unsigned)(blocks ? blocks : 1);
}
}  // namespace

cudaError_t launch_kv4_write(const KvRowsParams& p, bool bf16, int num_sms, cudaStream_t st) {
  const unsigned b = rows_blocks(p, num_sms);
  if (bf16)
    attn_kv_write_kernel<true><<<b, 256, 0, st>>>(p);
  else
    attn_kv_write_kernel<false><<<b, 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const KvRowsParams& p, bool bf16, int num_sms, cudaStream_t st) {
  const unsigned b = rows_blocks(p, num_sms);
  if (bf16)
    attn_kv_read_kernel<true><<<b, 256, 0, st>>>(p);
  else
    attn_kv_read_kernel<false><<<b, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
