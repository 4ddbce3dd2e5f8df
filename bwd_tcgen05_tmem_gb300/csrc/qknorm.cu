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
// for loads.  A lane takes "units" of two 8-element vectors that hold both
// halves of 8 pairs (rows u and u + rot/16 of the row's vectors), so the
// rotation needs no exchange between lanes; d / 16 units make a row, LPR lanes
// share it and a warp works on 32 / LPR heads of ONE token at a time, kU of
// them in flight: the token's cosines, sines and the weights are loaded once
// and stay in registers.
#include "kcommon.cuh"
#include "kv.h"

namespace attn {

template <int D>
struct QkShape {  // lanes that share a row, units of each lane
  static constexpr int kUnits = D / 16;
  static constexpr int kLpr = D == 192 ? 4 : kUnits;
  static constexpr int kUpl = kUnits / kLpr;
  static constexpr int kSlots = 32 / kLpr;  // rows a warp holds at a time
};

// The two vectors of unit u: both halves of 8 pairs, or two neighbours of the
// part that does not rotate.
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

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = Pack<BF16>::to_f((uint16_t)(w[i] & 0xffffu));
    f[2 * i + 1] = Pack<BF16>::to_f((uint16_t)(w[i] >> 16));
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(Pack<BF16>::two(f[0], f[1]), Pack<BF16>::two(f[2], f[3]),
                    Pack<BF16>::two(f[4], f[5]), Pack<BF16>::two(f[6], f[7]));
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
    unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + vec), f);
  }
}

// Cosines and sines of a unit's 8 pairs: pair e of a half-split unit is
// (a[e], b[e]); of an interleaved one (a[2e], a[2e+1]) for e < 4, then b's.
__device__ __forceinline__ void load_angles(const QkParams& p, int pos, int u, int a, int b,
                                            float (&c)[8], float (&s)[8]) {
  if (u >= (p.rot >> 4)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.0f, s[i] = 0.0f;
    return;
  }
  const int64_t row = (int64_t)pos * (p.rot >> 1);
  const int i0 = p.inter ? a * 4 : a * 8, i1 = p.inter ? b * 4 : a * 8 + 4;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(p.cos + row + i0));
  const float4 c1 = __ldg(reinterpret_cast<const float4*>(p.cos + row + i1));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(p.sin + row + i0));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(p.sin + row + i1));
  c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
  s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
}

// Turns the unit (a, b) by its angles; sign -1 turns back.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8],
                                     const float (&s)[8], int inter, float sign) {
  if (inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = a[2 * e], x1 = a[2 * e + 1], y0 = b[2 * e], y1 = b[2 * e + 1];
      a[2 * e] = x0 * c[e] - x1 * (sign * s[e]);
      a[2 * e + 1] = x1 * c[e] + x0 * (sign * s[e]);
      b[2 * e] = y0 * c[e + 4] - y1 * (sign * s[e + 4]);
      b[2 * e + 1] = y1 * c[e + 4] + y0 * (sign * s[e + 4]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * c[e] - y * (sign * s[e]);
      b[e] = y * c[e] + x * (sign * s[e]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The position of token (b, t): -1 (padding: the rows stay as they are), or
// -2 where it lies outside the tables.
__device__ __forceinline__ int token_position(const QkParams& p, int b, int t) {
  const int pos = p.positions ? p.positions[(int64_t)b * p.seqlen + t] : t;
  if (pos < 0) return -1;
  if (pos >= p.max_pos && p.rot > 0) return -2;
  return pos;
}

__device__ __forceinline__ void flag_index(int* status) {
  if (status) atomicCAS(status, DEV_OK, DEV_BAD_INDEX);
}

// ----------------------------------------------------------------- forward
// One warp: one token, one run of kSlots * kU heads of one side.
template <bool BF16, int D, int U>
__global__ void __launch_bounds__(128) attn_qk_fwd_kernel(const __grid_constant__ QkParams p,
                                                          int runs_q, int runs) {
  using S = QkShape<D>;
  const int lane = threadIdx.x & 31, slot = lane / S::kLpr, l = lane % S::kLpr;
  const int64_t job = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t tok = job / runs;
  const int run = (int)(job - tok * runs);
  if (tok >= (int64_t)p.batch * p.seqlen) return;
  const int b = (int)(tok / p.seqlen), t = (int)(tok - (int64_t)b * p.seqlen);
  const bool is_k = run >= runs_q;
  const QkSide& sd = p.side[is_k ? 1 : 0];
  const int h0 = (is_k ? run - runs_q : run) * (S::kSlots * U) + slot;
  const int pos = token_position(p, b, t);
  if (pos == -1) return;
  if (pos == -2 && lane == 0) flag_index(p.status);

  int va[S::kUpl], vb[S::kUpl];
  uint4 xa[U][S::kUpl], xb[U][S::kUpl];
#pragma unroll
  for (int i = 0; i < S::kUpl; ++i) unit_vectors(i * S::kLpr + l, p.rot, S::kUnits, va[i], vb[i]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * S::kSlots;
    const uint4* row = reinterpret_cast<const uint4*>((const uint16_t*)sd.x + b * sd.x_b +
                                                      t * sd.x_t + (int64_t)h * sd.x_h);
#pragma unroll
    for (int i = 0; i < S::kUpl; ++i) {
      xa[u][i] = xb[u][i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < sd.heads) xa[u][i] = row[va[i]], xb[u][i] = row[vb[i]];
    }
  }
  float rms[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < S::kUpl; ++i) {
      float a[8], c[8];
      unpack8<BF16>(xa[u][i], a);
      unpack8<BF16>(xb[u][i], c);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(c[e], c[e], ss));
    }
    ss = row_sum<S::kLpr>(ss);
    rms[u] = p.norm ? rsqrtf(ss * (1.0f / D) + p.eps) : 1.0f;
    if (pos == -2) rms[u] = __int_as_float(0x7fffffff);  // NaN: no such angle
  }
#pragma unroll
  for (int i = 0; i < S::kUpl; ++i) {
    float wa[8], wb[8], cs[8], sn[8];
    load_weights<BF16>(p, sd.w, va[i], wa);
    load_weights<BF16>(p, sd.w, vb[i], wb);
    load_angles(p, pos < 0 ? 0 : pos, i * S::kLpr + l, va[i], vb[i], cs, sn);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * S::kSlots;
      float a[8], c[8];
      unpack8<BF16>(xa[u][i], a);
      unpack8<BF16>(xb[u][i], c);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] *= rms[u] * wa[e], c[e] *= rms[u] * wb[e];
      turn(a, c, cs, sn, p.inter, 1.0f);
      if (h < sd.heads) {
        uint4* out = reinterpret_cast<uint4*>((uint16_t*)sd.out + b * sd.o_b + t * sd.o_t +
                                              (int64_t)h * sd.o_h);
        out[va[i]] = pack8<BF16>(a);
        out[vb[i]] = pack8<BF16>(c);
      }
    }
  }
}

// ----------------------------------------------------------------- gradient
// Blocks 0 .. blocks[0]-1 work on the queries, the others on the keys, so a
// lane's share of dw stays in registers over all rows of its block; each block
// leaves one row of partial sums, which a second kernel adds up in the order
// of the blocks (no atomics: the result does not depend on who came first).
template <bool BF16, int D, int U>
__global__ void __launch_bounds__(256) attn_qk_bwd_kernel(const __grid_constant__ QkParams p) {
  using S = QkShape<D>;
  const int lane = threadIdx.x & 31, slot = lane / S::kLpr, l = lane % S::kLpr;
  const bool is_k = (int)blockIdx.x >= p.blocks[0];
  const QkSide& sd = p.side[is_k ? 1 : 0];
  const int blk = is_k ? (int)blockIdx.x - p.blocks[0] : (int)blockIdx.x;
  const int nblk = p.blocks[is_k ? 1 : 0];
  const int runs = (sd.heads + S::kSlots * U - 1) / (S::kSlots * U);
  const int64_t jobs = (int64_t)p.batch * p.seqlen * runs;
  int va[S::kUpl], vb[S::kUpl];
  float wa[S::kUpl][8], wb[S::kUpl][8], da[S::kUpl][8], db[S::kUpl][8];
#pragma unroll
  for (int i = 0; i < S::kUpl; ++i) {
    unit_vectors(i * S::kLpr + l, p.rot, S::kUnits, va[i], vb[i]);
    load_weights<BF16>(p, sd.w, va[i], wa[i]);
    load_weights<BF16>(p, sd.w, vb[i], wb[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) da[i][e] = db[i][e] = 0.0f;
  }
  for (int64_t job = (int64_t)blk * 8 + (threadIdx.x >> 5); job < jobs; job += (int64_t)nblk * 8) {
    const int64_t tok = job / runs;
    const int h0 = (int)(job - tok * runs) * (S::kSlots * U) + slot;
    const int b = (int)(tok / p.seqlen), t = (int)(tok - (int64_t)b * p.seqlen);
    const int pos = token_position(p, b, t);
    if (pos == -1) continue;
    if (pos == -2 && lane == 0) flag_index(p.status);
    uint4 xa[U][S::kUpl], xb[U][S::kUpl], ga[U][S::kUpl], gb[U][S::kUpl];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * S::kSlots;
      const uint4* row = reinterpret_cast<const uint4*>((const uint16_t*)sd.x + b * sd.x_b +
                                                        t * sd.x_t + (int64_t)h * sd.x_h);
      const uint4* grow = reinterpret_cast<const uint4*>((const uint16_t*)sd.dz + b * sd.dz_b +
                                                         t * sd.dz_t + (int64_t)h * sd.dz_h);
#pragma unroll
      for (int i = 0; i < S::kUpl; ++i) {
        xa[u][i] = xb[u][i] = ga[u][i] = gb[u][i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < sd.heads) {
          xa[u][i] = row[va[i]], xb[u][i] = row[vb[i]];
          ga[u][i] = grow[va[i]], gb[u][i] = grow[vb[i]];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * S::kSlots;
      float ya[S::kUpl][8], yb[S::kUpl][8];  // dy
      float ss = 0.0f, gx = 0.0f;
#pragma unroll
      for (int i = 0; i < S::kUpl; ++i) {
        float a[8], c[8], cs[8], sn[8];
        load_angles(p, pos < 0 ? 0 : pos, i * S::kLpr + l, va[i], vb[i], cs, sn);
        unpack8<BF16>(ga[u][i], ya[i]);
        unpack8<BF16>(gb[u][i], yb[i]);
        turn(ya[i], yb[i], cs, sn, p.inter, -1.0f);
        unpack8<BF16>(xa[u][i], a);
        unpack8<BF16>(xb[u][i], c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(a[e], a[e], fmaf(c[e], c[e], ss));
          gx = fmaf(ya[i][e] * wa[i][e], a[e], fmaf(yb[i][e] * wb[i][e], c[e], gx));
        }
      }
      ss = row_sum<S::kLpr>(ss);
      gx = row_sum<S::kLpr>(gx);
      float r = p.norm ? rsqrtf(ss * (1.0f / D) + p.eps) : 1.0f;
      if (pos == -2) r = __int_as_float(0x7fffffff);
      const float k = p.norm ? r * r * (gx * (1.0f / D)) : 0.0f;
#pragma unroll
      for (int i = 0; i < S::kUpl; ++i) {
        float a[8], c[8];
        unpack8<BF16>(xa[u][i], a);
        unpack8<BF16>(xb[u][i], c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          da[i][e] = fmaf(ya[i][e], a[e] * r, da[i][e]);
          db[i][e] = fmaf(yb[i][e], c[e] * r, db[i][e]);
          a[e] = r * fmaf(-a[e], k, ya[i][e] * wa[i][e]);
          c[e] = r * fmaf(-c[e], k, yb[i][e] * wb[i][e]);
        }
        if (h < sd.heads) {
          uint4* out = reinterpret_cast<uint4*>((uint16_t*)sd.out + b * sd.o_b + t * sd.o_t +
                                                (int64_t)h * sd.o_h);
          out[va[i]] = pack8<BF16>(a);
          out[vb[i]] = pack8<BF16>(c);
        }
      }
    }
  }
  if (!sd.dw) return;
  // the block's sum of dw: over the rows a warp holds, then over its 8 warps
  __shared__ float part[8][D];
#pragma unroll
  for (int i = 0; i < S::kUpl; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = S::kLpr; o < 32; o <<= 1) {
        da[i][e] += __shfl_xor_sync(0xffffffffu, da[i][e], o);
        db[i][e] += __shfl_xor_sync(0xffffffffu, db[i][e], o);
      }
      if (slot == 0) {
        part[threadIdx.x >> 5][va[i] * 8 + e] = da[i][e];
        part[threadIdx.x >> 5][vb[i] * 8 + e] = db[i][e];
      }
    }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += 256) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w][c];
    p.partial[(int64_t)blockIdx.x * D + c] = s;
  }
}

// dw: 32 columns a block, 8 runs of the partial rows each, then those.
__global__ void __launch_bounds__(256) attn_qk_dw_kernel(const __grid_constant__ QkParams p) {
  __shared__ float part[8][32];
  const QkSide& sd = p.side[blockIdx.y];
  if (!sd.dw) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  const int64_t first = blockIdx.y ? p.blocks[0] : 0;
  float s = 0.0f;
#pragma unroll 8
  for (int i = w; i < p.blocks[blockIdx.y]; i += 8) s += p.partial[(first + i) * p.d + c];
  part[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += part[k][threadIdx.x];
    sd.dw[c] = s;
  }
}

// ----------------------------------------------------------------- launches
namespace {

template <bool BF16, int D, int U>
cudaError_t fwd_launch(const QkParams& p, cudaStream_t st) {
  const int per = QkShape<D>::kSlots * U;
  const int rq = (p.side[0].heads + per - 1) / per, rk = (p.side[1].heads + per - 1) / per;
  const int64_t blocks = ((int64_t)p.batch * p.seqlen * (rq + rk) + 3) / 4;
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  attn_qk_fwd_kernel<BF16, D, U><<<(unsigned)blocks, 128, 0, st>>>(p, rq, rq + rk);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t fwd_dispatch(const QkParams& p, cudaStream_t st) {
  switch (p.d) {
    case 64: return fwd_launch<BF16, 64, 4>(p, st);
    case 128: return fwd_launch<BF16, 128, 4>(p, st);
    case 192: return fwd_launch<BF16, 192, 1>(p, st);
    case 256: return fwd_launch<BF16, 256, 4>(p, st);
    case 512: return fwd_launch<BF16, 512, 4>(p, st);
    default: return cudaErrorNotSupported;
  }
}

template <bool BF16, int D, int U>
cudaError_t bwd_launch(const QkParams& p, cudaStream_t st) {
  attn_qk_bwd_kernel<BF16, D, U><<<p.blocks[0] + p.blocks[1], 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!p.side[0].dw && !p.side[1].dw)) return e;
  attn_qk_dw_kernel<<<dim3(D / 32, 2), 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t bwd_dispatch(const QkParams& p, cudaStream_t st) {
  switch (p.d) {
    case 64: return bwd_launch<BF16, 64, 2>(p, st);
    case 128: return bwd_launch<BF16, 128, 2>(p, st);
    case 192: return bwd_launch<BF16, 192, 1>(p, st);
    case 256: return bwd_launch<BF16, 256, 2>(p, st);
    case 512: return bwd_launch<BF16, 512, 2>(p, st);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_qk_fwd(const QkParams& p, bool bf16, int num_sms, cudaStream_t st) {
  (void)num_sms;
  return bf16 ? fwd_dispatch<true>(p, st) : fwd_dispatch<false>(p, st);
}

// Two blocks an SM, shared out by the rows of each side; never more than one
// for each 8 tokens.
void qk_bwd_blocks(QkParams& p, int num_sms) {
  const int64_t tokens = (int64_t)p.batch * p.seqlen;
  const int64_t heads = p.side[0].heads + p.side[1].heads;
  for (int s = 0; s < 2; ++s) {
    int64_t n = heads ? (2 * (int64_t)num_sms * p.side[s].heads + heads / 2) / heads : 0;
    const int64_t most = (tokens * p.side[s].heads + 7) / 8;
    if (n > most) n = most;
    p.blocks[s] = p.side[s].heads > 0 ? (int)(n > 1 ? n : 1) : 0;
  }
}

cudaError_t launch_qk_bwd(const QkParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? bwd_dispatch<true>(p, st) : bwd_dispatch<false>(p, st);
}

}  // namespace attn
