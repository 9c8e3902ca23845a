// kv4.cuh -- 4-bit cache values: scale, code and the pairs that readers use.
#pragma once
#include <cstdint>

#include "ops.cuh"
#include "tile_math.cuh"

namespace hstu {

// Scale of a group whose largest |x| is the bf16 number with the bits m: the
// smallest number of five significant bits >= max / 7, the maximum taken as at
// least 2^-100 (so that 1 / s is finite).  A group that holds an infinity or a
// NaN gets a NaN scale and reads as NaN.
// The quotient is max times the fp32 number nearest to 1 / 7, off by less than
// 2^-22 of itself.  Where max = 7 k for a k of five bits it has to come out at
// or below k, and elsewhere it is 2^-9 or more away from such a k (7 k has
// eight bits, as max has), so 64 units in the last place (2^-17) are taken off
// before rounding upwards.
__device__ __forceinline__ float kv4_scale(uint32_t m) {
  if (m >= 0x7F80u) return __uint_as_float(0x7FC00000u);
  const float top = fmaxf(__uint_as_float(m << 16), 7.8886090522101181e-31f);
  const uint32_t s = __float_as_uint(top * 0.14285714924335479736f);
  return __uint_as_float((s - 64u + 0x7FFFFu) & ~0x7FFFFu);
}

// 1 / s to one unit in the last place.
__device__ __forceinline__ float kv4_inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// The codes n + 8 of a bf16 pair w, in bits 0..3 and 16..19 (the other bits
// hold anything): n = rint(x / s) for q = x (1 / s) in fp32, which is off by
// less than 2^-22 of itself.  Exact quotients of an 8-bit by a 5-bit
// significand are either ties or 2^-10 and more away from one, so rounding q to
// a multiple of 2^-11 first (adding and taking away 1.5 * 2^12) restores ties,
// and the second rounding sends them to even as the exact quotient's would.
// The last constant is 1.5 * 2^23 + 8: the low bits of the sum are n + 8.
__device__ __forceinline__ uint32_t kv4_codes(uint32_t w, uint64_t inv2) {
  uint64_t q = fmul2(pack_f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), inv2);
  q = fadd2(q, pack_f32x2(6144.0f, 6144.0f));
  q = fadd2(q, pack_f32x2(-6144.0f, -6144.0f));
  q = fadd2(q, pack_f32x2(12582920.0f, 12582920.0f));
  const float2 f = unpack_f32x2(q);
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x5410);
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
