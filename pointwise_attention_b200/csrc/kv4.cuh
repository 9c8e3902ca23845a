// kv4.cuh -- 4-bit cache values: scale, code and the pairs that readers use.
#pragma once
#include <cstdint>

#include "tile_math.cuh"

namespace hstu {

// Scale of a group whose largest |x| has the bit pattern m: the smallest
// number of five significant bits >= max / 7, the maximum taken as at least
// 2^-100 (so that 1 / s is finite).  A group that holds an infinity or a NaN
// gets a NaN scale and reads as NaN.
__device__ __forceinline__ float kv4_scale(uint32_t m) {
  if (m >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float top = fmaxf(__uint_as_float(m), 7.8886090522101181e-31f);
  const uint32_t s = __float_as_uint(__fdiv_rn(top, 7.0f));
  return __uint_as_float((s + 0x7FFFFu) & ~0x7FFFFu);
}

// rint(x / s) + 8 for q = x * (1 / s) in fp32.  q carries a relative error of
// 2^-23; exact quotients of an 8-bit by a 5-bit significand are either ties
// or 2^-10 and more away from one, so rounding q to a multiple of 2^-11 first
// (adding and taking away 1.5 * 2^12) restores ties, and the second rounding
// sends them to even as the exact quotient's would.
__device__ __forceinline__ uint32_t kv4_code(float q) {
  const float t = __fadd_rn(__fadd_rn(q, 6144.0f), -6144.0f);
  // 1.5 * 2^23 + 8: the low bits of the sum are the whole number plus 8
  return __float_as_uint(__fadd_rn(t, 12582920.0f)) & 15u;
}

// bf16 pair (value 2I, value 2I + 1) of a word of eight: 128 + (n + 8) is the
// code in a bf16 significand, minus 136 leaves n exactly, and n s is exact.
template <int I>
__device__ __forceinline__ uint32_t kv4_pair(uint32_t word, uint32_t s2) {
  const uint32_t b = ((word >> (4 * I)) & 0x000F000Fu) | 0x43004300u;
  return hmul2(hadd2(b, 0xC308C308u), s2);   // 0xC308 = -136
}

// The pair (value 2I, value 2I + 1) again, in one operation after the
// extraction: the code c = n + 8 in bits 3..6 of a bf16 significand is 16 + c
// = 24 + n, and (24 + n) s - 24 s is n s exactly, 24 s having seven
// significant bits at most.  m24s = -24 s2 (kv4_m24): infinite for scales
// above 2^123, so values of such groups are not finite here.
template <int I>
__device__ __forceinline__ uint32_t kv4_pair_fma(uint32_t word, uint32_t s2, uint32_t m24s) {
  const uint32_t w = I == 0 ? word << 3 : word >> (I == 0 ? 0 : 4 * I - 3);
  uint32_t c;   // (w & mask) | 16.0 in one operation
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(c) : "r"(w), "r"(0x00780078u), "r"(0x41804180u));
  return hfma2(c, s2, m24s);
}
__device__ __forceinline__ uint32_t kv4_m24(uint32_t s2) { return hmul2(s2, 0xC1C0C1C0u); }

}  // namespace hstu
