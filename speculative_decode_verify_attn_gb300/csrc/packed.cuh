// 4-bit groups: 16 values in 8 bytes of e2m1 codes (the even value in a byte's low 4 bits) and one e4m3 scale.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace vfy {

// Bytes of one (chunk, KV head) record of K or V.
template <int HD>
constexpr int kPackedBytes = 36 * HD;

// A byte's two codes as fp16 values.
__device__ __forceinline__ uint32_t e2m1_pair_f16(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 c, x0, x1, x2;\n\tmov.b32 {c, x0, x1, x2}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}
__device__ __forceinline__ float f16_value(uint32_t bits) {
  float f;
  asm("{\n\t.reg .f16 h;\n\tmov.b16 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "h"(static_cast<uint16_t>(bits)));
  return f;
}
__device__ __forceinline__ float2 e2m1_pair(uint32_t byte) {
  const uint32_t h = e2m1_pair_f16(byte);
  return make_float2(f16_value(h & 0xffffu), f16_value(h >> 16));
}
// Two e4m3 bytes as fp16 values (the low byte in the low half).
__device__ __forceinline__ uint32_t e4m3_pair_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) { return f16_value(e4m3_pair_f16(byte) & 0xffffu); }

// g s e in bf16, rounded once. A product's 30 bits are rounded to odd first (to zero, the last bit set where that dropped
// anything): a rounding to fewer bits behind it gives the exact product's. Below 2^-90 remainders would underflow: g 2^100 in
// place of g, and back. `se` = s e has 6 bits and is 0 or at least 2^-10 in size.
__device__ __forceinline__ float product_to_odd(float se, float g) {
  constexpr float kSmall = 8e-28f, kUp = 1.2676506002282294e30f, kDown = 7.888609052210118e-31f;   // 2^-90, 2^100, 2^-100
  const bool small = g < kSmall;
  if (small) g *= kUp;
  float p = __fmul_rz(se, g);
  bool inexact = fmaf(se, g, -p) != 0.f;
  if (small) {
    const float up = p;
    p = __fmul_rz(up, kDown);
    inexact = inexact || p * kUp != up;
  }
  return __uint_as_float(__float_as_uint(p) | (inexact ? 1u : 0u));
}
// For all e with one s: is e times the rounded s g, rounded again, as near? e is a power of two, or 3 of them: s g and its
// triple decide, each off by at most 1.5 units, where they are not next to a tie of bf16, nor near either end of fp32.
// (One group in 4700 is; with every product rounded to odd, reading back 8 x 1024 tokens took 0.9 us more.)
__device__ __forceinline__ bool plain_product(float s, float sg) {
  auto off_tie = [](float x) { return ((__float_as_uint(x) - 0x7ffdu) & 0xffffu) > 6u; };
  return s == 0.f || (sg > 1e-30f && sg < 4e37f && off_tie(sg) && off_tie(1.5f * sg));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The two codes of byte Y of a word times a scale (a pair of them, one for each half).
template <int Y>
__device__ __forceinline__ uint32_t unpack_byte(uint32_t codes, uint32_t scale2) {
  uint32_t r;
  if constexpr (Y == 0)
    asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, x0;\n\t}" : "=r"(r) : "r"(codes));
  else if constexpr (Y == 1)
    asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, x1;\n\t}" : "=r"(r) : "r"(codes));
  else if constexpr (Y == 2)
    asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, x2;\n\t}" : "=r"(r) : "r"(codes));
  else
    asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, x3;\n\t}" : "=r"(r) : "r"(codes));
  return mul_f16x2(r, scale2);
}
// Eight codes (a 32-bit word) times a scale: eight fp16 values, two a register.
__device__ __forceinline__ void unpack_word(uint32_t codes, uint32_t scale2, uint32_t* out) {
  out[0] = unpack_byte<0>(codes, scale2);
  out[1] = unpack_byte<1>(codes, scale2);
  out[2] = unpack_byte<2>(codes, scale2);
  out[3] = unpack_byte<3>(codes, scale2);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The e4m3 byte nearest to x >= 0 (ties to even, at most 448; NaN gives 448).
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(fminf(x, 448.f)));
  return r & 0xffu;
}
// The codes nearest to eight values (the first in the low 4 bits): ties to the even code, at most 6 in size.
__device__ __forceinline__ uint32_t e2m1_of(const float2& a, const float2& b, const float2& c, const float2& d) {
  uint32_t r;
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 x1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 x3, %8, %7;\n\t"
      "mov.b32 %0, {x0, x1, x2, x3};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// A power of two by halves: x * a * b = x 2^e for |e| <= 252, and nothing that the product can hold is lost between.
struct PowerOfTwo {
  float a, b;
  __device__ __forceinline__ explicit PowerOfTwo(int e) {
    e = min(max(e, -252), 252);
    const int h = e >> 1;
    a = __int_as_float((127 + h) << 23);
    b = __int_as_float((127 + e - h) << 23);
  }
  __device__ __forceinline__ float times(float x) const { return x * a * b; }
};
// The queries of a tile, the largest of them with bf16 bits `top` (its size), are scaled by 2^-exponent to at most 2^15.
__device__ __forceinline__ int query_exponent(unsigned top) { return static_cast<int>(top >> 7) - 127 - 14; }
// What a product of scaled queries and s e is multiplied with to be a score in log2 units: a normal number, because 0 times a
// masked key's -inf is NaN, and so is infinity times 0.
__device__ __forceinline__ float score_scale(float scale_log2, int scale_exp, int query_exp) {
  return fminf(fmaxf(PowerOfTwo(scale_exp + query_exp).times(scale_log2), 1.2e-38f), 3e38f);
}

// A row's reference (log2) is at most this in size, or the call reports the row: neighbouring fp32 scores are 8 apart from here
// on, and a weight could land 16 above the place that its reference gives it, past fp16.
constexpr float kMostScore = 67108864.f;   // 2^26

// Exponent e for which a partial's O, sum and reference are handed on as O 2^-e, sum 2^-e and reference + e. Sums of weights
// times values stay below 2^57 times g (2^15 a weight, 2^31 keys, values of 2688), which fp32 holds up to g = 1e20: until
// there e is 0. Past it the sum becomes 2^-7 .. 2^-6, so that O, and what the combine adds up of 64 partials, is no larger
// than the largest value.
__device__ __forceinline__ int partial_exponent(float sum, float g) {
  return g > 1e20f && sum > 0.f ? (static_cast<int>(__float_as_uint(sum) >> 23) - 127) + 7 : 0;
}

// 16 values x to the codes of x / g and their scale. Quotients are rounded as IEEE divisions: the scale's quotient can lie on
// a tie of e4m3 only if it is exact, and so can a value's on a tie of e2m1. `x`: pairs.
//
// A quotient comes from the rounded reciprocal, one remainder and one correction (Markstein's division), two at a time
// (with divisions the append of 8 x 1024 tokens took a quarter longer). That is exact where nothing overflows and no
// remainder underflows: g within 2^-100 .. 2^100, s is 2^-9 .. 448 and below 448 |x / g| is at most a little over 6 s, and a
// value whose remainder underflows is far below a code. Anything else, infinities among it, is divided.
__device__ __forceinline__ float2 quotients(float2 v, float2 minus_by, float2 r) {
  const float2 q = mul_f32x2(v, r);
  return fma_f32x2(fma_f32x2(q, minus_by, v), r, q);
}
// `inv`: 1 / g rounded, 0 where g is out of that range.
__device__ __forceinline__ uint2 pack_group(float2 (&x)[8], float g, float inv, uint32_t* scale) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(fmaxf(top, fabsf(x[e].x)), fabsf(x[e].y));
  if (inv != 0.f && top < 1e38f && top * inv < 1e38f) {
    // (the quotients' largest is the largest's: rounding keeps order)
    const float2 most = quotients(make_float2(top, 0.f), make_float2(-g, -g), make_float2(inv, inv));
    constexpr float kSixth = 1.f / 6.f;
    *scale = e4m3_of(quotients(most, make_float2(-6.f, -6.f), make_float2(kSixth, kSixth)).x);
    const float s = e4m3_value(*scale);
    if (!(s > 0.f)) return make_uint2(0u, 0u);
    const float rs = __frcp_rn(s);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = quotients(quotients(x[e], make_float2(-g, -g), make_float2(inv, inv)), make_float2(-s, -s), make_float2(rs, rs));
  } else {
    *scale = e4m3_of(__fdiv_rn(__fdiv_rn(top, g), 6.f));
    const float s = e4m3_value(*scale);
    if (!(s > 0.f)) return make_uint2(0u, 0u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e].x = __fdiv_rn(__fdiv_rn(x[e].x, g), s);
      x[e].y = __fdiv_rn(__fdiv_rn(x[e].y, g), s);
    }
  }
  return make_uint2(e2m1_of(x[0], x[1], x[2], x[3]), e2m1_of(x[4], x[5], x[6], x[7]));
}

}  // namespace vfy
