// The greedy rule's order of logits, shared by the acceptance kernels: a 64-bit key per entry whose
// high 32 bits are the fp32 value mapped to an unsigned integer that sorts like the value (every NaN
// maps to the top, -0 to +0) and whose low 32 bits are the complement of the index (so equal values
// prefer the lower index). 0 is below every key.
#pragma once

#include <cstdint>

namespace vfy {

__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;  // NaN: above everything
  if (u == 0x80000000u) u = 0u;                              // -0 ties +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ unsigned long long pack(float x, int idx) {
  return (static_cast<unsigned long long>(order_key(x)) << 32) |
         static_cast<unsigned long long>(0xffffffffu - static_cast<uint32_t>(idx));
}

__device__ __forceinline__ int unpack_index(unsigned long long key) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key & 0xffffffffull));
}

// max that returns NaN when either operand is NaN (fmaxf returns the other operand)
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ unsigned long long umax64(unsigned long long a, unsigned long long b) {
  return a > b ? a : b;
}

// The best key of the n4 float4 words s4[0 ..], whose first entry has index `first`, over the words
// of this thread (thread t of THREADS takes words t, t + THREADS, ...; UNROLL loads in flight).
template <int THREADS, int UNROLL>
__device__ __forceinline__ unsigned long long scan_words(const float4* s4, int n4, int first) {
  unsigned long long best = 0ull;
  for (int i0 = threadIdx.x; i0 < n4; i0 += THREADS * UNROLL) {
    float4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (i0 + u * THREADS < n4) v[u] = __ldcs(s4 + i0 + u * THREADS);
      else v[u] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    // The round's best key without packing every entry: the largest value by a NaN-propagating
    // max (NaN iff the round holds one), then the lowest index holding that value (a float
    // compare: -0 == +0, the two keys' tie) or, with a NaN, the lowest NaN's index. Padding
    // entries hold -inf at indices past the segment, so they never win a tie.
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      m = max_nan(m, max_nan(max_nan(v[u].x, v[u].y), max_nan(v[u].z, v[u].w)));
    int at = 0x7fffffff;
    if (m == m) {
#pragma unroll
      for (int u = UNROLL - 1; u >= 0; --u) {
        const int base = first + 4 * (i0 + u * THREADS);
        at = v[u].w == m ? base + 3 : at;
        at = v[u].z == m ? base + 2 : at;
        at = v[u].y == m ? base + 1 : at;
        at = v[u].x == m ? base : at;
      }
    } else {
      m = __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int u = UNROLL - 1; u >= 0; --u) {
        const int base = first + 4 * (i0 + u * THREADS);
        at = v[u].w != v[u].w ? base + 3 : at;
        at = v[u].z != v[u].z ? base + 2 : at;
        at = v[u].y != v[u].y ? base + 1 : at;
        at = v[u].x != v[u].x ? base : at;
      }
    }
    if (at != 0x7fffffff) best = umax64(best, pack(m, at));
  }
  return best;
}

}  // namespace vfy
