// E4M3 codes with fp32 scales for blocks of 128: the rule, and what its kernels share.
#pragma once

#include "around.cuh"

namespace moe {

// A block's scale is its largest |x| / 448 (E4M3's largest value), rounded to nearest; a block
// below 2^-64 counts as 2^-64, so that quotients and their remainders stay normal numbers.
constexpr float F8_TOP = 448.0f;
constexpr float F8_FLOOR = 5.421010862427522e-20f;   // 2^-64
struct F8Scale {
  float s, inv;   // the scale and its reciprocal, both to nearest
};
__device__ __forceinline__ F8Scale f8_scale(float amax) {
  F8Scale f;
  f.s = __fdiv_rn(fmaxf(amax, F8_FLOOR), F8_TOP);
  f.inv = __frcp_rn(f.s);
  return f;
}
// x / s rounded to nearest, for two values: the product with the reciprocal, corrected once by
// its remainder (Markstein's theorem: with a correctly rounded reciprocal the result is the
// rounded quotient).  Codes then never depend on how a quotient near a tie was computed.  An
// infinity in the block (s infinite) makes all of its codes NaN.
__device__ __forceinline__ f32x2 f8_quotient(f32x2 x, f32x2 neg_s, f32x2 inv) {
  const f32x2 q = mul2(x, inv);
  return fma2(fma2(q, neg_s, x), inv, q);
}
__device__ __forceinline__ uint32_t f8_codes4(f32x2 a, f32x2 b, f32x2 neg_s, f32x2 inv) {
  const float2 x = unpair(f8_quotient(a, neg_s, inv)), y = unpair(f8_quotient(b, neg_s, inv));
  return cvt_e4m3x4(x.x, x.y, y.x, y.y);
}
// Two bf16 in a word as a pair of fp32.
__device__ __forceinline__ f32x2 bf16_pair(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
// Per half, the larger magnitude (a NaN gives way to a number: its code is NaN by itself).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));   // the signs' product comes along
  return r;
}
__device__ __forceinline__ float max_halves(uint32_t w) { return fmaxf(fabsf(bf16_lo(w)), fabsf(bf16_hi(w))); }

inline bool f8_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline long long up128(long long x) { return (x + 127) / 128 * 128; }

}  // namespace moe
