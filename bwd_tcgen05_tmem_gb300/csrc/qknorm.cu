// qknorm.cu -- what stands between the projections and the attention kernels:
// the norm of each query and key head and the rotation by its position, in one
// pass, and its gradient.
//
// Row x (one token, one head, d elements), weights w, angles t_i of its
// position on the first `rot` elements (pairs (i, i + rot/2), or (2i, 2i+1)
// when interleaved):
//     r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  z = R(t) y.
// Gradient, with dy = R(t)^T dz and g = dy w:
//     dw = sum over rows of dy x r,   dx = r (g - x r^2 mean(g x)).
// r is computed again from x, which the gradient reads anyway, so the forward
// saves nothing.
//
// Both are streams: 2 (forward) or 3 (gradient) rows of 16-bit elements are
// moved for each row, with about one operation a byte, so the layout is made
// for loads.  A lane takes a "unit" of two 8-element vectors that hold both
// halves of 8 pairs (vectors u and u + rot/16 of the row), so the rotation
// needs no exchange between lanes; d / 16 lanes make a row, and a warp works on
// several heads of ONE token at a time: the token's cosines, sines and the
// weights are loaded once for all of them.  The arithmetic is in packed FP32
// pairs (fma.f32x2).  Rows come through a ring of asynchronous 16-byte copies:
// each lane copies its own vectors a few jobs ahead and waits for its own
// copies alone, so loads stay in flight while it computes, and no lane waits
// for another.
//
// Measured on a GB300 (graph replays, bf16, head dim 128, 32 + 8 heads): forward
// of 32768 tokens 116 us, 5.9 TB/s (88% of a plain copy's rate); gradient of
// 16384 tokens 96 us, 5.3 TB/s (78%: bound by instruction issue beside the
// copies, about 47 a pair of elements); 8 tokens 3.2 us, a launch; a gradient of
// 3 x 1001 tokens of 6 + 2 heads of 192 13 us, two dependent launches and the
// join of dw.  Loads into registers instead of the ring: 155 and 173 us.
#include <algorithm>
#include <type_traits>

#include "kcommon.cuh"
#include "kv.h"

namespace attn {

template <int D>
struct QkShape {
  static constexpr int kUnits = D / 16;                 // lanes of a row that work
  static constexpr int kLpr = D == 192 ? 16 : kUnits;   // lanes of a row
  static constexpr int kSlots = 32 / kLpr;              // rows a warp holds at a time
};

// The two vectors of unit u: both halves of 8 pairs, or two of the part that
// does not rotate.
__device__ __forceinline__ void unit_vectors(int u, int rot, int units, int& a, int& b) {
  const int rh = rot >> 4;
  if (u < rh) {
    a = u;
    b = u + rh;
  } else {
    a = rh + u;
    b = u + units;
  }
}

// A unit's 8 pairs (P, Q) as packed FP32 pairs over e: pair e is (a[e], b[e])
// of the two vectors or, interleaved, (a[2e], a[2e+1]) for e < 4, then b's.
struct Pairs {
  uint64_t p[4], q[4];
};

template <bool BF16>
__device__ __forceinline__ void two_floats(uint32_t w, float& lo, float& hi) {
  if (BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
}

template <bool INTER>
__device__ __forceinline__ Pairs pairs_of(const float (&a)[8], const float (&b)[8]) {
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      const float* v = i < 2 ? a : b;
      const int j = (i & 1) * 4;
      r.p[i] = f2_pack(v[j], v[j + 2]);
      r.q[i] = f2_pack(v[j + 1], v[j + 3]);
    } else {
      r.p[i] = f2_pack(a[2 * i], a[2 * i + 1]);
      r.q[i] = f2_pack(b[2 * i], b[2 * i + 1]);
    }
  }
  return r;
}

template <bool BF16, bool INTER>
__device__ __forceinline__ Pairs unpack(const uint4& va, const uint4& vb) {
  const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    two_floats<BF16>(wa[i], a[2 * i], a[2 * i + 1]);
    two_floats<BF16>(wb[i], b[2 * i], b[2 * i + 1]);
  }
  return pairs_of<INTER>(a, b);
}

template <bool BF16, bool INTER>
__device__ __forceinline__ void pack(const Pairs& x, uint4& va, uint4& vb) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p0, p1, q0, q1;
    f2_unpack(x.p[i], p0, p1);
    f2_unpack(x.q[i], q0, q1);
    if (INTER) {
      w[2 * i] = Pack<BF16>::two(p0, q0);
      w[2 * i + 1] = Pack<BF16>::two(p1, q1);
    } else {
      w[i] = Pack<BF16>::two(p0, p1);
      w[i + 4] = Pack<BF16>::two(q0, q1);
    }
  }
  va = make_uint4(w[0], w[1], w[2], w[3]);
  vb = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool BF16>
__device__ __forceinline__ void load_weights(const QkParams& p, const void* w, int vec,
                                             float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  } else if (p.w_f32) {
    const float4* s = reinterpret_cast<const float4*>((const float*)w + vec * 8);
    const float4 x = __ldg(s), y = __ldg(s + 1);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(w) + vec);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) two_floats<BF16>(u[i], f[2 * i], f[2 * i + 1]);
  }
}

// Cosines and sines of a unit's 8 pairs, packed over e (none at a negative pos).
__device__ __forceinline__ void load_angles(const QkParams& p, int pos, int u, int a, int b,
                                            uint64_t (&c)[4], uint64_t (&s)[4]) {
  if (pos < 0 || u >= (p.rot >> 4)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f2_pack(1.0f, 1.0f), s[i] = f2_pack(0.0f, 0.0f);
    return;
  }
  const int64_t row = (int64_t)pos * (p.rot >> 1);
  const int i0 = p.inter ? a * 4 : a * 8, i1 = p.inter ? b * 4 : a * 8 + 4;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(p.cos + row + i0));
  const float4 c1 = __ldg(reinterpret_cast<const float4*>(p.cos + row + i1));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(p.sin + row + i0));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(p.sin + row + i1));
  c[0] = f2_pack(c0.x, c0.y), c[1] = f2_pack(c0.z, c0.w), c[2] = f2_pack(c1.x, c1.y), c[3] = f2_pack(c1.z, c1.w);
  s[0] = f2_pack(s0.x, s0.y), s[1] = f2_pack(s0.z, s0.w), s[2] = f2_pack(s1.x, s1.y), s[3] = f2_pack(s1.z, s1.w);
}

__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }

template <int LPR>
__device__ __forceinline__ float row_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  float s = lo + hi;
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// 1 / sqrt(sum / D + eps); 0 where that is 1 / 0, so that rows of zeros give zeros
// at eps = 0 too and lanes without a row, which hold zeros, add nothing to dw.  A
// NaN stays one: a row with a NaN is NaN in all of its elements.
template <int D>
__device__ __forceinline__ float rms_inverse(float sum, float eps) {
  const float v = fmaf(sum, 1.0f / D, eps);
  float r;
  if (v < 1.17549435e-38f) {  // (rare) below the normal range: 2^12 rsqrt(2^24 v)
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 16777216.0f));
    return v == 0.0f ? 0.0f : r * 4096.0f;
  }
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A copy of 16 bytes, or of zeros.
__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool here) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"((uint64_t)__cvta_generic_to_global(src)), "r"(here ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups of this thread
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kQkThreads = 128, kQkWarps = kQkThreads / 32;
constexpr int kPad = -1, kNoAngle = -2;  // positions: padding; outside the tables

template <bool MANY>
__device__ __forceinline__ int token_position(const QkParams& p, uint32_t tok) {
  if (MANY && tok >= (uint32_t)p.batch * p.seq_div.d) return kPad;  // behind the last token
  const int pos = p.positions ? __ldg(p.positions + tok) : (int)(tok - p.seq_div.div(tok) * p.seq_div.d);
  return pos < 0 ? kPad : pos >= p.max_pos && p.rot > 0 ? kNoAngle : pos;
}

// A job is one token and one run of kSlots * U of its heads, of one side; where
// half of the kSlots rows that a warp holds at a time or more would be idle, it
// is several tokens in a row with all of their heads (48K tokens of 2 + 2 heads of
// 64, gradient: 28 us, one token a job 85 us; only calls with such a side run that
// form, which costs the others 4%).  The side's blocks share its
// jobs, a warp takes every (blocks * warps)-th.  A lane's view of the side's tensors: byte offsets from its vector a of its row
// (slot) of the first run.
struct QkLane {
  int64_t b, t, run, u;  // of a sequence, a token, a run, kSlots heads
  __device__ __forceinline__ int64_t at(uint32_t bi, uint32_t ti, uint32_t ri) const {
    return (int64_t)bi * b + (int64_t)ti * t + (int64_t)ri * run;
  }
};
template <int SLOTS, int U>
__device__ __forceinline__ QkLane qk_lane(int64_t sb, int64_t st, int64_t sh) {
  return QkLane{sb * 2, st * 2, sh * (2 * SLOTS * U), sh * (2 * SLOTS)};
}

// The ring: NV vectors a lane and row (of x, and of dz), and for each lane its
// token and that one's position.
template <int U, int NV, int STAGES>
struct QkRing {
  uint4 v[STAGES][U][NV][kQkThreads];
  uint2 job[STAGES][kQkThreads];
};

// What both directions share: which jobs a warp has, and copying the next one.
// MANY: jobs may have several tokens, so tokens and positions differ between lanes.
template <int D, int U, int NV, int STAGES, bool MANY>
struct QkWarp {
  using S = QkShape<D>;
  const QkParams& p;
  const QkSide& sd;
  QkRing<U, NV, STAGES>& ring;
  int warp, lane, slot;  // slot: the lane's head of a group of rows
  int sub, per_job;      // its token of the job, the job's tokens
  bool active;
  FastDiv runs;
  uint32_t end, step, next;
  int next_pos;
  const char *x, *dz;
  QkLane lx, lz;
  int vb;  // bytes from vector a to b

  __device__ __forceinline__ QkWarp(const QkParams& p_, QkRing<U, NV, STAGES>& r_, bool is_k, int a, int b)
      : p(p_), sd(p_.side[is_k ? 1 : 0]), ring(r_) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    slot = lane / S::kLpr;
    per_job = 1;
    sub = 0;
    if (MANY) {
      per_job = sd.per_job;
      const int heads = S::kSlots / per_job;  // (a power of two)
      sub = slot / heads;
      slot -= sub * heads;
    }
    active = lane % S::kLpr < S::kUnits;
    runs = p.runs[is_k ? 1 : 0];
    // below 2^31, checked at launch
    end = ((uint32_t)p.batch * p.seq_div.d + per_job - 1) / per_job * runs.d;
    step = (uint32_t)p.blocks[is_k ? 1 : 0] * kQkWarps;
    next = (blockIdx.x - (is_k ? (uint32_t)p.blocks[0] : 0u)) * kQkWarps + warp;
    next_pos = next < end ? token_position<MANY>(p, token(next)) : kPad;
    x = (const char*)sd.x + ((int64_t)slot * sd.x_h + a * 8) * 2;
    lx = qk_lane<S::kSlots, U>(sd.x_b, sd.x_t, sd.x_h);
    if (NV == 4) {
      dz = (const char*)sd.dz + ((int64_t)slot * sd.dz_h + a * 8) * 2;
      lz = qk_lane<S::kSlots, U>(sd.dz_b, sd.dz_t, sd.dz_h);
    }
    vb = (b - a) * 16;
  }
  __device__ __forceinline__ uint32_t token(uint32_t job) const {
    return runs.div(job) * (uint32_t)per_job + sub;
  }
  // Row groups of a run that hold a head.
  __device__ __forceinline__ int groups(uint32_t run) const {
    return min(U, (sd.heads - (int)run * (S::kSlots * U) + S::kSlots - 1) / S::kSlots);
  }
  // Whether this lane's row of group u is one.
  __device__ __forceinline__ bool here(uint32_t run, int u, int pos) const {
    return active && (int)run * (S::kSlots * U) + u * S::kSlots + slot < sd.heads && !(MANY && pos == kPad);
  }
  __device__ __forceinline__ void copy(int s) {
    if (next < end) {
      const uint32_t first = runs.div(next), run = next - first * runs.d;
      const uint32_t tok = first * (uint32_t)per_job + sub;
      if (MANY ? __any_sync(0xffffffffu, next_pos != kPad) : next_pos != kPad) {
        const uint32_t b = p.seq_div.div(tok), t = tok - b * p.seq_div.d;
        const char* px = x + lx.at(b, t, run);
        const char* pz = NV == 4 ? dz + lz.at(b, t, run) : nullptr;
        const int n = groups(run);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= n) break;
          const bool is = here(run, u, next_pos);  // (else zeros; the address is not used)
          uint4(*v)[kQkThreads] = ring.v[s][u];
          // (the gradient without the norm does not depend on x, whatever that holds)
          const bool is_x = is && (NV == 2 || p.norm);
          copy16(&v[0][threadIdx.x], is_x ? px : x, is_x);
          copy16(&v[1][threadIdx.x], is_x ? px + vb : x, is_x);
          px += lx.u;
          if (NV == 4) {
            copy16(&v[NV - 2][threadIdx.x], is ? pz : x, is);
            copy16(&v[NV - 1][threadIdx.x], is ? pz + vb : x, is);
            pz += lz.u;
          }
        }
      }
      if (MANY || lane == 0) ring.job[s][MANY ? threadIdx.x : warp] = make_uint2(tok, (uint32_t)next_pos);
      next += step;
      if (next < end) next_pos = token_position<MANY>(p, token(next));
    }
    copies_end();
  }
};

// ----------------------------------------------------------------- forward
// FULL: all elements turn, and no lane asks whether its own do (32K tokens of 32 + 8
// heads of 128: 116 us; with the question, as where half of each row turns, 120 us).
template <bool BF16, int D, int U, bool INTER, bool MANY, bool FULL>
__global__ void __launch_bounds__(kQkThreads, 6) attn_qk_fwd_kernel(
    const __grid_constant__ QkParams p) {
  using S = QkShape<D>;
  constexpr int kStages = 2;
  __shared__ QkRing<U, 2, kStages> ring;
  const int l = min((int)(threadIdx.x & 31) % S::kLpr, S::kUnits - 1);
  int va, vb;
  unit_vectors(l, p.rot, S::kUnits, va, vb);
  const bool turns = l < (p.rot >> 4);
  QkWarp<D, U, 2, kStages, MANY> w(p, ring, (int)blockIdx.x >= p.blocks[0], va, vb);
  char* out = (char*)w.sd.out + ((int64_t)w.slot * w.sd.o_h + va * 8) * 2;
  const QkLane lo = qk_lane<S::kSlots, U>(w.sd.o_b, w.sd.o_t, w.sd.o_h);
  uint32_t job = w.next;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) w.copy(i);
  for (int s = 0; job < w.end; job += w.step, s = s == kStages - 1 ? 0 : s + 1) {
    __syncwarp();
    w.copy(s == 0 ? kStages - 1 : s - 1);  // the stage used last
    copies_wait<kStages - 1>();
    __syncwarp();
    const uint2 at = ring.job[s][MANY ? threadIdx.x : w.warp];
    const uint32_t tok = at.x;
    const int pos = (int)at.y;
    if (MANY ? __all_sync(0xffffffffu, pos == kPad) : pos == kPad) continue;
    if (pos == kNoAngle && w.slot == 0 && l == 0 && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    uint64_t pc[4], ps[4], qc[4], qs[4];  // weights times cosines and sines
    {
      float fa[8], fb[8];
      load_weights<BF16>(p, w.sd.w, va, fa);
      load_weights<BF16>(p, w.sd.w, vb, fb);
      const Pairs wt = pairs_of<INTER>(fa, fb);
      load_angles(p, pos, l, va, vb, pc, ps);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qc[i] = f2_mul(wt.q[i], pc[i]);
        qs[i] = f2_neg(f2_mul(wt.q[i], ps[i]));
        pc[i] = f2_mul(wt.p[i], pc[i]);
        ps[i] = f2_mul(wt.p[i], ps[i]);
      }
    }
    const uint32_t run = job - (MANY ? w.runs.div(job) : tok) * w.runs.d;
    const uint32_t b = p.seq_div.div(tok), t = tok - b * p.seq_div.d;
    char* po = out + lo.at(b, t, run);
    const int n = w.groups(run);
#pragma unroll 1
    for (int u = 0; u < n; ++u, po += lo.u) {
      const Pairs x = unpack<BF16, INTER>(ring.v[s][u][0][threadIdx.x], ring.v[s][u][1][threadIdx.x]);
      float r = 1.0f;
      if (p.norm) {
        uint64_t ss = f2_mul(x.p[0], x.p[0]), st = f2_mul(x.q[0], x.q[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = f2_fma(x.p[i], x.p[i], ss), st = f2_fma(x.q[i], x.q[i], st);
        r = rms_inverse<D>(row_sum<S::kLpr>(f2_add(ss, st)), p.eps);
      }
      if (pos == kNoAngle) r = __int_as_float(0x7fffffff);  // NaN
      const uint64_t r2 = f2_both(r);
      Pairs z;
      if (FULL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z.p[i] = f2_mul(r2, f2_fma(x.q[i], qs[i], f2_mul(x.p[i], pc[i])));
          z.q[i] = f2_mul(r2, f2_fma(x.p[i], ps[i], f2_mul(x.q[i], qc[i])));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z.p[i] = f2_mul(x.p[i], pc[i]);
          z.q[i] = f2_mul(x.q[i], qc[i]);
          if (turns) {  // (else an infinity or a NaN times 0 would reach its neighbour)
            z.p[i] = f2_fma(x.q[i], qs[i], z.p[i]);
            z.q[i] = f2_fma(x.p[i], ps[i], z.q[i]);
          }
          z.p[i] = f2_mul(r2, z.p[i]);
          z.q[i] = f2_mul(r2, z.q[i]);
        }
      }
      if (w.here(run, u, pos)) pack<BF16, INTER>(z, *(uint4*)po, *(uint4*)(po + w.vb));
    }
  }
  copies_wait<0>();
}

// ----------------------------------------------------------------- gradient
// Blocks 0 .. blocks[0]-1 work on the queries, the others on the keys, so a
// lane's share of dw stays in registers over all rows of its block; each block
// leaves one row of partial sums, which a second kernel adds up in the order
// of the blocks (no atomics: the result does not depend on who came first).
template <bool BF16, int D, int U, bool INTER, bool MANY>
__global__ void __launch_bounds__(kQkThreads, 4) attn_qk_bwd_kernel(
    const __grid_constant__ QkParams p) {
  using S = QkShape<D>;
  constexpr int kStages = 2;
  __shared__ QkRing<U, 4, kStages> ring;
  asm volatile("griddepcontrol.launch_dependents;");
  const int l = min((int)(threadIdx.x & 31) % S::kLpr, S::kUnits - 1);
  int va, vb;
  unit_vectors(l, p.rot, S::kUnits, va, vb);
  const bool turns = l < (p.rot >> 4);
  QkWarp<D, U, 4, kStages, MANY> w(p, ring, (int)blockIdx.x >= p.blocks[0], va, vb);
  char* out = (char*)w.sd.out + ((int64_t)w.slot * w.sd.o_h + va * 8) * 2;
  const QkLane lo = qk_lane<S::kSlots, U>(w.sd.o_b, w.sd.o_t, w.sd.o_h);
  Pairs wt, dw;
  {
    float fa[8], fb[8];
    load_weights<BF16>(p, w.sd.w, va, fa);
    load_weights<BF16>(p, w.sd.w, vb, fb);
    wt = pairs_of<INTER>(fa, fb);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw.p[i] = dw.q[i] = f2_both(0.0f);
  }
  uint32_t job = w.next;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) w.copy(i);
  for (int s = 0; job < w.end; job += w.step, s = s == kStages - 1 ? 0 : s + 1) {
    __syncwarp();
    w.copy(s == 0 ? kStages - 1 : s - 1);
    copies_wait<kStages - 1>();
    __syncwarp();
    const uint2 at = ring.job[s][MANY ? threadIdx.x : w.warp];
    const uint32_t tok = at.x;
    const int pos = (int)at.y;
    if (MANY ? __all_sync(0xffffffffu, pos == kPad) : pos == kPad) continue;
    if (pos == kNoAngle && w.slot == 0 && l == 0 && p.status) atomicCAS(p.status, DEV_OK, DEV_BAD_INDEX);
    uint64_t c[4], sn[4];
    load_angles(p, pos, l, va, vb, c, sn);
    const uint32_t run = job - (MANY ? w.runs.div(job) : tok) * w.runs.d;
    const uint32_t b = p.seq_div.div(tok), t = tok - b * p.seq_div.d;
    char* po = out + lo.at(b, t, run);
    const int n = w.groups(run);
#pragma unroll 1
    for (int u = 0; u < n; ++u, po += lo.u) {
      const Pairs x = unpack<BF16, INTER>(ring.v[s][u][0][threadIdx.x], ring.v[s][u][1][threadIdx.x]);
      const Pairs z = unpack<BF16, INTER>(ring.v[s][u][2][threadIdx.x], ring.v[s][u][3][threadIdx.x]);
      Pairs dy, g;
      uint64_t ss = f2_both(0.0f), gx = f2_both(0.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dy.p[i] = f2_mul(z.p[i], c[i]);
        dy.q[i] = f2_mul(z.q[i], c[i]);
        if (turns) {
          dy.p[i] = f2_fma(z.q[i], sn[i], dy.p[i]);
          dy.q[i] = f2_fma(z.p[i], f2_neg(sn[i]), dy.q[i]);
        }
        g.p[i] = f2_mul(dy.p[i], wt.p[i]);
        g.q[i] = f2_mul(dy.q[i], wt.q[i]);
        ss = f2_fma(x.p[i], x.p[i], ss);
        ss = f2_fma(x.q[i], x.q[i], ss);
        gx = f2_fma(g.p[i], x.p[i], gx);
        gx = f2_fma(g.q[i], x.q[i], gx);
      }
      float r = 1.0f, k = 0.0f;
      if (p.norm) {
        r = rms_inverse<D>(row_sum<S::kLpr>(ss), p.eps);
        k = (r * (1.0f / D)) * (r * row_sum<S::kLpr>(gx));  // (r^2 itself may pass FP32's range)
      }
      if (pos == kNoAngle) r = __int_as_float(0x7fffffff);
      const uint64_t r2 = f2_both(r), k2 = f2_both(-k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw.p[i] = f2_fma(dy.p[i], f2_mul(x.p[i], r2), dw.p[i]);
        dw.q[i] = f2_fma(dy.q[i], f2_mul(x.q[i], r2), dw.q[i]);
        g.p[i] = f2_mul(r2, f2_fma(x.p[i], k2, g.p[i]));
        g.q[i] = f2_mul(r2, f2_fma(x.q[i], k2, g.q[i]));
      }
      if (w.here(run, u, pos)) pack<BF16, INTER>(g, *(uint4*)po, *(uint4*)(po + w.vb));
    }
  }
  copies_wait<0>();
  if (!w.sd.dw) return;
  // the block's sum of dw: over the rows a warp holds, then over its warps
  float* part = reinterpret_cast<float*>(ring.v);  // [warp][D]
  float f[16];  // as they lie in the two vectors
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p0, p1, q0, q1;
    f2_unpack(dw.p[i], p0, p1);
    f2_unpack(dw.q[i], q0, q1);
    if (INTER) {
      f[4 * i] = p0, f[4 * i + 1] = q0, f[4 * i + 2] = p1, f[4 * i + 3] = q1;
    } else {
      f[2 * i] = p0, f[2 * i + 1] = p1, f[8 + 2 * i] = q0, f[8 + 2 * i + 1] = q1;
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e)
#pragma unroll
    for (int o = S::kLpr; o < 32; o <<= 1) f[e] += __shfl_xor_sync(0xffffffffu, f[e], o);
  __syncthreads();
  if (w.lane < S::kLpr && w.active)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      part[w.warp * D + va * 8 + e] = f[e];
      part[w.warp * D + vb * 8 + e] = f[8 + e];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kQkThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kQkWarps; ++k) sum += part[k * D + c];
    p.partial[(int64_t)blockIdx.x * D + c] = sum;
  }
}

// dw: 32 columns a block, 32 runs of the partial rows each, then those.  It is
// launched while the first kernel runs, and waits for its end.
__global__ void __launch_bounds__(1024) attn_qk_dw_kernel(const __grid_constant__ QkParams p) {
  __shared__ float part[32][33];
  const QkSide& sd = p.side[blockIdx.y];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
  const int64_t first = blockIdx.y ? p.blocks[0] : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!sd.dw) return;
  float s = 0.0f;
#pragma unroll 8
  for (int i = w; i < p.blocks[blockIdx.y]; i += 32) s += p.partial[(first + i) * p.d + c];
  part[w][lane] = s;
  __syncthreads();
  s = part[lane][w];  // warp w: column w's 32 runs
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sd.dw[blockIdx.x * 32 + w] = s;
}

// ----------------------------------------------------------------- launches
namespace {

constexpr int kFwdRows = 4, kBwdRows = 2;  // groups of rows of a job
constexpr int kJobCost = 4;  // (1: 127 us, 2: 122 us, 4: 116 us for 32K tokens of 32 + 8 heads)

// Runs of `groups` times `slots` heads of each side, and its blocks: `most` in
// all, shared out by the sides' costs (a job costs kJobCost groups besides its
// own); never more than leave each warp `least` jobs.  False: too many jobs.
bool share_blocks(QkParams& p, int most, int slots, int groups, int least) {
  const int64_t all_tokens = (int64_t)p.batch * p.seqlen;
  p.seq_div = FastDiv::of((uint32_t)std::max(p.seqlen, 1));
  bool ok = true;
  int64_t runs[2], cost[2], tokens[2];
  for (int s = 0; s < 2; ++s) {
    const int64_t h = p.side[s].heads;
    int per = slots;
    while (per > 1 && per * h > slots) per /= 2;
    p.side[s].per_job = per;
    tokens[s] = (all_tokens + per - 1) / per;
    runs[s] = std::max<int64_t>((h + slots * groups - 1) / (slots * groups), 1);
    cost[s] = h ? tokens[s] * (runs[s] * kJobCost + (h + slots - 1) / slots) : 0;
    p.runs[s] = FastDiv::of((uint32_t)runs[s]);
    ok = ok && tokens[s] * runs[s] < (1ll << 31) - (1 << 20);
  }
  for (int s = 0; s < 2; ++s) {
    const int64_t all = std::max<int64_t>(cost[0] + cost[1], 1);
    int64_t n = (int64_t)((double)most * cost[s] / all + 0.5);
    n = std::min(n, (tokens[s] * runs[s] + least * kQkWarps - 1) / (least * kQkWarps));
    p.blocks[s] = p.side[s].heads > 0 ? (int)std::max<int64_t>(n, 1) : 0;
  }
  return ok;
}

int slots_of(int d) { return d == 192 ? 2 : 32 / (d / 16); }

// f with the call's order of pairs, and whether a side's jobs have several tokens
template <typename F>
void variants(const QkParams& p, F&& f) {
  const bool many = p.side[0].per_job > 1 || (p.side[1].heads && p.side[1].per_job > 1);
  using Y = std::true_type;
  using N = std::false_type;
  if (p.inter)
    many ? f(Y(), Y()) : f(Y(), N());
  else
    many ? f(N(), Y()) : f(N(), N());
}

template <bool BF16, int D>
cudaError_t fwd_launch(const QkParams& p, cudaStream_t st) {
  variants(p, [&](auto inter, auto many) {
    constexpr bool I = decltype(inter)::value, M = decltype(many)::value;
    const int blocks = p.blocks[0] + p.blocks[1];
    if (p.rot == D)
      attn_qk_fwd_kernel<BF16, D, kFwdRows, I, M, true><<<blocks, kQkThreads, 0, st>>>(p);
    else
      attn_qk_fwd_kernel<BF16, D, kFwdRows, I, M, false><<<blocks, kQkThreads, 0, st>>>(p);
  });
  return cudaGetLastError();
}

template <bool BF16, int D>
cudaError_t bwd_launch(const QkParams& p, cudaStream_t st) {
  variants(p, [&](auto inter, auto many) {
    attn_qk_bwd_kernel<BF16, D, kBwdRows, decltype(inter)::value, decltype(many)::value>
        <<<p.blocks[0] + p.blocks[1], kQkThreads, 0, st>>>(p);
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!p.side[0].dw && !p.side[1].dw)) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(D / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_qk_dw_kernel, p);
}

template <bool BF16>
cudaError_t dispatch(const QkParams& p, bool fwd, cudaStream_t st) {
  switch (p.d) {
    case 64: return fwd ? fwd_launch<BF16, 64>(p, st) : bwd_launch<BF16, 64>(p, st);
    case 128: return fwd ? fwd_launch<BF16, 128>(p, st) : bwd_launch<BF16, 128>(p, st);
    case 192: return fwd ? fwd_launch<BF16, 192>(p, st) : bwd_launch<BF16, 192>(p, st);
    case 256: return fwd ? fwd_launch<BF16, 256>(p, st) : bwd_launch<BF16, 256>(p, st);
    case 512: return fwd ? fwd_launch<BF16, 512>(p, st) : bwd_launch<BF16, 512>(p, st);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_qk_fwd(QkParams& p, bool bf16, int num_sms, cudaStream_t st) {
  if (!share_blocks(p, num_sms * 6, slots_of(p.d), kFwdRows, 1)) return cudaErrorNotSupported;
  return bf16 ? dispatch<true>(p, true, st) : dispatch<false>(p, true, st);
}

// (two jobs a warp: half the partial rows of dw where there are few tokens)
bool qk_bwd_blocks(QkParams& p, int num_sms) {
  return share_blocks(p, num_sms * 4, slots_of(p.d), kBwdRows, 2);
}

cudaError_t launch_qk_bwd(const QkParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? dispatch<true>(p, false, st) : dispatch<false>(p, false, st);
}

}  // namespace attn
