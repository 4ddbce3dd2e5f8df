// kvtile.cuh -- what the kernels that compute with the 4-bit cache's codes share: the
// 16 x 8 x 16 product, K's codes as its operand, wide shared-memory loads, scales,
// asynchronous copies.
#pragma once
#include "kcommon.cuh"

namespace attn {

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = c + a b
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}

// The 8 codes of a word as pairs of fp16 numbers below the normal range: pair n
// holds codes n and n + 4.  The tensor cores take such numbers exactly, but line
// their products up by the range's lowest exponent, so that sums miss a bit for
// each zero above a code.
// K's stand high, since a score is such a sum.  Error of the LSE of few tokens of head
// dim 64, in 2^-24 of sum |q k|: codes in bits 0 and 4 (no shift for the first two
// pairs) up to 26, in bits 2 and 6 4.6, all in bit 4 1.7, normal numbers 1.5; time of
// 16 x 32K tokens of head dim 128 117, 118, 123, 120 us, 8 x 32K of 256 132, 140, 131,
// 139 us.
template <int DQK>
struct KCodes {
  static constexpr bool kLevel = DQK == 256;  // all pairs in bit 4; else the odd ones 16 fold
  static constexpr float kOdd = kLevel ? 1.0f : 0.0625f;          // what their q is multiplied with
  static constexpr float kUnit = kLevel ? 1048576.0f : 4194304.0f;  // 1 / (a code of 1 in the even ones)
  static constexpr uint32_t kEven8 = kLevel ? 0x80808080u : 0x80208020u, kOdd8 = kLevel ? 0x80808080u : 0x82008200u;  // -8
  static __device__ __forceinline__ void of(uint32_t w, uint32_t (&p)[4]) {
    if (kLevel) {
      p[0] = (w << 4) & 0x00f000f0u;
      p[1] = w & 0x00f000f0u;
      p[2] = (w >> 4) & 0x00f000f0u;
      p[3] = (w >> 8) & 0x00f000f0u;
    } else {
      p[0] = (w << 2) & 0x003c003cu;
      p[1] = (w << 2) & 0x03c003c0u;
      p[2] = (w >> 6) & 0x003c003cu;
      p[3] = (w >> 6) & 0x03c003c0u;
    }
  }
};

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

// A power of two from its exponent (-126 .. 127).
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"((uint64_t)__cvta_generic_to_global(src))
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups of this thread
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace attn
