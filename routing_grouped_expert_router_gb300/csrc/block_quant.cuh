// block_quant.cuh -- how a value becomes an e4m3 code under its block's scale,
// shared by the quantisers and by the epilogues of the grouped products.
#pragma once
#include <cstdint>
#include <cuda_fp8.h>

namespace moe {

constexpr float kCodeMax = 448.0f;  // the largest e4m3 value

// A block's scale and what dividing by it takes.  `top` is the bit pattern of
// the largest |v|: patterns of non-negative floats order as their values do,
// with infinity and NaN above all of them, so an integer maximum keeps a NaN.
struct BlockScale {
  float s;     // amax / 448, 1 for a block of zeros
  float r;     // its reciprocal, correctly rounded
  bool plain;  // s lies where the quick quotient below is exact
};
__device__ __forceinline__ BlockScale block_scale(uint32_t top) {
  BlockScale b;
  const float amax = __uint_as_float(top);
  if (amax > 7.9e-31f && amax < 1.2e30f) {
    // as the quotients below, with the constant's reciprocal
    constexpr float r = 1.0f / kCodeMax;
    const float q0 = amax * r;
    b.s = fmaf(fmaf(-q0, kCodeMax, amax), r, q0);
  } else {
    b.s = top == 0 ? 1.0f : __fdiv_rn(amax, kCodeMax);
  }
  b.r = __frcp_rn(b.s);
  b.plain = b.s > 7.9e-31f && b.s < 1.2e30f;  // 2^-100 .. 2^100
  return b;
}

// The float32 quotient v / s, rounded as IEEE division rounds it.  With r the
// correctly rounded reciprocal of s, q0 = v r is within an ulp of the quotient,
// the residual v - q0 s is exact in one fused multiply-add, and one more gives
// the correctly rounded quotient (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990).
// That holds while nothing leaves the normal range: for scales of 2^-100 to
// 2^100 a residual that does belongs to a quotient far below the least code,
// 2^-9.  Other scales (and those that are not finite) take the division.
// Two values at a time: these instructions are issued for two, and issue slots are what
// codes cost.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void halves_of(uint64_t p, float (&v)[2]) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint32_t quick_codes2(float lo, float hi, const BlockScale& b) {
  const uint64_t v = pair_of(lo, hi), r = pair_of(b.r, b.r), minus_s = pair_of(-b.s, -b.s);
  const uint64_t q0 = mul_2(v, r);
  const uint64_t q = fma_2(fma_2(q0, minus_s, v), r, q0);
  float c[2];
  halves_of(q, c);
  return codes2(c[0], c[1]);
}
// Four values -> four codes, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], const BlockScale& b) {
  if (b.plain) return quick_codes2(v[0], v[1], b) | (quick_codes2(v[2], v[3], b) << 16);
  return codes2(__fdiv_rn(v[0], b.s), __fdiv_rn(v[1], b.s)) |
         (codes2(__fdiv_rn(v[2], b.s), __fdiv_rn(v[3], b.s)) << 16);
}

// The larger magnitude's bit pattern of the two bf16 in w and of top.
__device__ __forceinline__ uint32_t top_of_pair(uint32_t top, uint32_t w) {
  const uint32_t hi = w & 0x7FFF0000u;
  const uint32_t lo = (w << 16) & 0x7FFF0000u;
  return max(top, max(hi, lo));
}

// The same for two columns of pairs at once: the larger magnitudes of w's two bf16 and of
// top's, each in its half (a NaN stays one), and the larger of the two halves as a pattern.
__device__ __forceinline__ uint32_t top_2(uint32_t top, uint32_t w) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(w & 0x7FFF7FFFu));
  return r;
}
__device__ __forceinline__ uint32_t top_of_2(uint32_t top) {
  return max(top << 16, top & 0xFFFF0000u);
}

}  // namespace moe
