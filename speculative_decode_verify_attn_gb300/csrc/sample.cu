// Acceptance of sampled drafts. With p_r = softmax(x_r / T) of the target's row r and q_j the drafter's distribution:
//     draft j (token d) stays iff u_j q_j(d) < p_j(d);   n = the first that does not, or D
//     next token = argmax_v w_v / E_v,   w = max(p_n - q_n, 0) for n < D, p_D for n = D
// With E exponentially distributed the argmax of w_v / E_v is a draw in proportion to w (the smallest of independent
// exponential times E_v / w_v). It needs no running sum over the vocabulary, whose order would decide draws near the
// borders of 100,000 tokens: here only two tokens whose times agree to 2^-21 can change places.
//
// Two kernels. The first reads every row once: each CTA takes a segment of one row and leaves its maximum and its sum of
// exponentials against that maximum (greedy rows: the key of the argmax, argmax.cuh); at most four CTAs an SM, which run at
// once, at most 32 a row. The second has up to two CTAs an SM for the sequences; each of them merges the row statistics (a
// part a lane), finds n, and races its segment of row n; the last one to finish (a ticket) writes the outputs. What does not
// wait for the first kernel (drafts, their probabilities, the first noise) is read before it is over.
//
// One sequence of 17 rows of 131072 fp32 logits takes 8.6 us, of which 1.5 are bytes: two kernels' chains of look-ups.
// 16 sequences of 164 rows of 100003 bf16 logits take 18.5 us (46 MB, 2.5 TB/s; 15.5 from L2): the first kernel
// ends at 3 instructions an entry, the second at 45 for one row a sequence; with the argmax and the race over p in its loop, and
// no loads ahead, 20.2 us.
#include <cuda_bf16.h>

#include "argmax.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;             // of the first kernel
constexpr int kWarps = kThreads / 32;
constexpr int kDrawThreads = 512;         // of the second
constexpr int kDrawWarps = kDrawThreads / 32;

// log2(e) / T in two pieces (the rest of a division is exact in one fma; fp64, 1/64 of fp32's rate here, cost 2 us a CTA).
// A tiny T is held at 2^-100: any two different logits are then further apart than fp32 can weigh. T = 0 (or one that is no
// temperature, which is reported) is greedy: 0.
struct Heat {
  float hi, lo;
};
__device__ __forceinline__ bool is_temperature(float t) { return t >= 0.f && t < INFINITY; }
__device__ __forceinline__ Heat heat_of(float t) {
  Heat h = {0.f, 0.f};
  if (is_temperature(t) && t > 0.f) {
    constexpr double kLog2e = 1.4426950408889634;
    constexpr float kHi = static_cast<float>(kLog2e), kLo = static_cast<float>(kLog2e - static_cast<double>(kHi));
    t = fmaxf(t, 7.9e-31f);
    h.hi = kHi / t;
    h.lo = (fmaf(-h.hi, t, kHi) + kLo) / t;
  }
  return h;
}

template <bool BF16>
__device__ __forceinline__ float entry(const void* row, int v) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[v]) << 16)
              : static_cast<const float*>(row)[v];
}
template <bool BF16>
__device__ __forceinline__ const void* row_at(const SampleParams& p, int row) {
  return static_cast<const char*>(p.logits) + static_cast<long long>(row) * p.stride * (BF16 ? 2 : 4);
}

// f(x, index) of every entry of a 16-byte word.
template <bool BF16, typename F>
__device__ __forceinline__ void each(const uint4& w, F f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f(__uint_as_float(u[i] << 16), 2 * i);
      f(__uint_as_float(u[i] & 0xffff0000u), 2 * i + 1);
    } else {
      f(__uint_as_float(u[i]), i);
    }
  }
}

// The largest entry of a word and `top`: without its NaN, or NaN if there is one.
template <bool BF16>
__device__ __forceinline__ float word_max(const uint4& w, float top) {
  if constexpr (BF16) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return fmaxf(fmaxf(top, __uint_as_float(a << 16)), __uint_as_float(a & 0xffff0000u));
  } else {
    return fmaxf(fmaxf(fmaxf(fmaxf(top, __uint_as_float(w.x)), __uint_as_float(w.y)), __uint_as_float(w.z)), __uint_as_float(w.w));
  }
}
template <bool BF16>
__device__ __forceinline__ float word_max_nan(const uint4& w, float top) {
  if constexpr (BF16) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return max_nan(max_nan(top, __uint_as_float(a << 16)), __uint_as_float(a & 0xffff0000u));
  } else {
    return max_nan(max_nan(max_nan(top, __uint_as_float(w.x)), __uint_as_float(w.y)),
                   max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
}
// The sum of 2^(x c - mc) over a word's entries, in two parts.
template <bool BF16>
__device__ __forceinline__ float2 word_sum(const uint4& w, float2 c, float2 minus_mc, float2 sum) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < (BF16 ? 4 : 2); ++i) {
    const float2 x = BF16 ? make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u))
                          : make_float2(__uint_as_float(u[2 * i % 4]), __uint_as_float(u[2 * i % 4 + 1]));
    const float2 t = fma_f32x2(x, c, minus_mc);
    sum = add_f32x2(sum, make_float2(ex2_approx(t.x), ex2_approx(t.y)));
  }
  return sum;
}

// 2^((a - top) c) where a <= top: the weight of a part whose maximum is a.
__device__ __forceinline__ float rescale(float a, float top, float c) {
  return a == top ? 1.f : ex2_approx((a - top) * c);
}

// Maximum and sum of exponentials of some entries of a row.
struct Stat {
  float m, z;
  // Over the lanes of a converged warp; all of them get it.
  __device__ __forceinline__ void merge_lanes(float c) {
    const float top = warp_max(m);
    z *= rescale(m, top, c);
    m = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  // Entries of at most `top`, the largest of them; any(f) calls f(x) for each.
  template <typename Any>
  __device__ __forceinline__ void add(float top, float c, Any any) {
    if (top > m) {
      z *= rescale(m, top, c);
      m = top;
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int e = 0;
    if (m == INFINITY) {                  // +inf entries share the row
      any([&](float x) { s[e++ & 3] += x == INFINITY ? 1.f : 0.f; });
    } else if (m != -INFINITY) {
      any([&](float x) { s[e++ & 3] += ex2_approx((x - m) * c); });
    }
    z += (s[0] + s[1]) + (s[2] + s[3]);
  }
};

// The largest of 32 keys, in all lanes.
__device__ __forceinline__ unsigned long long warp_umax64(unsigned long long key) {
  const uint32_t hi = static_cast<uint32_t>(key >> 32), top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(key) : 0u);
  return static_cast<unsigned long long>(top) << 32 | lo;
}

// ------------------------------ row statistics ----------------------------------------------
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) sample_stats_kernel(const SampleParams p) {
  constexpr int kVec = BF16 ? 8 : 4;      // entries of a 16-byte word
  constexpr int kUnroll = 4;
  __shared__ Stat s_stat[kWarps];
  __shared__ unsigned long long s_key[kWarps];
  pdl_wait();
  // The second kernel starts reading the callers' inputs before it waits for this one: they are complete from here on.
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.y;
  int total;
  float temperature;
  if (p.num_seqs <= 32) {                 // the row's sequence and its temperature in one round trip
    const int end = lane < p.num_seqs ? p.cu_rows[lane + 1] : INT_MAX;
    const float mine = lane < p.num_seqs ? p.temperature[lane] : 0.f;
    total = __shfl_sync(0xffffffffu, end, p.num_seqs - 1);
    const int b = min(__popc(__ballot_sync(0xffffffffu, end <= row)), p.num_seqs - 1);
    temperature = __shfl_sync(0xffffffffu, mine, b);
    if (row >= total) return;
  } else {
    total = p.cu_rows[p.num_seqs];
    if (row >= total) return;
    temperature = p.temperature[sequence_of(p.cu_rows, p.num_seqs, row, lane)];
  }
  const float c = heat_of(temperature).hi;
  const int v0 = blockIdx.x * p.seg, v1 = min(p.vocab, v0 + p.seg);
  const void* src = row_at<BF16>(p, row);
  // entries before the first whole 16-byte word, whole words, entries behind the last
  const uintptr_t at = reinterpret_cast<uintptr_t>(src) + static_cast<uintptr_t>(v0) * (BF16 ? 2 : 4);
  const int n = max(0, v1 - v0);
  const int head = min(n, static_cast<int>((16 - (at & 15)) & 15) / (BF16 ? 2 : 4));
  const int words = (n - head) / kVec;
  const int tail = v0 + head + words * kVec;
  const uint4* body = reinterpret_cast<const uint4*>(at + head * (BF16 ? 2 : 4));
  Stat st = {-INFINITY, 0.f};
  unsigned long long key = 0ull;
  // 2^((x - m) c) as 2^(x c - mc), mc the rounded product: one instruction, and what the rounding of mc did to all of a
  // round's entries taken back from their sum. Where mc is not small the differences are taken first.
  float mc = 0.f, back = 1.f;
  bool small = false;
  constexpr uint32_t kNone = BF16 ? 0xff80ff80u : 0xff800000u;   // -inf
  auto load = [&](int i0, uint4 (&w)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      w[u] = i < words ? __ldg(body + i) : make_uint4(kNone, kNone, kNone, kNone);
    }
  };
  float best = -INFINITY;                 // greedy rows: the largest entry so far (or NaN), and its round
  int best_round = -1;
  uint4 next[kUnroll];
  load(threadIdx.x, next);
  for (int i0 = threadIdx.x; i0 < words; i0 += kThreads * kUnroll) {
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) w[u] = next[u];
    load(i0 + kThreads * kUnroll, next);  // (the next round's, while this one is summed)
    float top = -INFINITY;
    if (c > 0.f) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) top = word_max<BF16>(w[u], top);
      if (top > st.m) {
        st.z *= rescale(st.m, top, c);
        st.m = top;
        mc = top * c;
        back = fmaf(fmaf(top, c, -mc), -0.6931472f, 1.f);
        small = fabsf(mc) < 4096.f;       // (not so for an infinite top)
      }
      float sum = NAN;
      if (small) {
        float2 part[2] = {};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          part[u & 1] = word_sum<BF16>(w[u], make_float2(c, c), make_float2(-mc, -mc), part[u & 1]);
        const float2 both = add_f32x2(part[0], part[1]);
        sum = both.x + both.y;
      }
      if (sum == sum)
        st.z = fmaf(sum, back, st.z);
      else                                // a NaN among them, +inf, or large products
        st.add(top, c, [&](auto f) {
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) each<BF16>(w[u], [&](float x, int) { f(fmaxf(x, -INFINITY)); });
        });
    } else {
      // Greedy: the first round with the largest value; a NaN is above all.
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) top = word_max_nan<BF16>(w[u], top);
      if (best_round < 0 || (best == best && !(top <= best))) {
        best = top;
        best_round = i0;
      }
    }
  }
  if (best_round >= 0) {                  // the first such entry in it
    load(best_round, next);
    int first = INT_MAX;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = best_round + u * kThreads;
      if (i < words)
        each<BF16>(next[u], [&](float x, int e) {
          if (x == best || (x != x && best != best)) first = min(first, v0 + head + i * kVec + e);
        });
    }
    key = pack(best, first);
  }
  // (fewer than kVec entries on each side)
  if (threadIdx.x < 2 * kVec) {
    const int v = threadIdx.x < kVec ? v0 + static_cast<int>(threadIdx.x) : tail + static_cast<int>(threadIdx.x) - kVec;
    if (threadIdx.x < kVec ? v < v0 + head : v < v1) {
      const float x = entry<BF16>(src, v);
      if (c > 0.f)
        st.add(fmaxf(x, -INFINITY), c, [&](auto f) { f(fmaxf(x, -INFINITY)); });
      else
        key = umax64(key, pack(x, v));
    }
  }
  if (c > 0.f)
    st.merge_lanes(c);
  else
    key = warp_umax64(key);
  if (lane == 0) {
    s_stat[warp] = st;
    s_key[warp] = key;
  }
  __syncthreads();
  if (warp == 0) {
    st.m = -INFINITY;
    st.z = 0.f;
    key = 0ull;
    if (lane < kWarps) {
      st = s_stat[lane];
      key = s_key[lane];
    }
    st.merge_lanes(c);
    key = warp_umax64(key);
    if (lane == 0)
      p.stats[static_cast<size_t>(row) * p.parts + blockIdx.x] =
          make_float4(st.m, st.z, __uint_as_float(static_cast<uint32_t>(key >> 32)), __uint_as_float(static_cast<uint32_t>(key)));
  }
}

// ------------------------------ acceptance and draw ------------------------------------------
// A whole row's statistics from its parts, one a lane (all lanes get them).
__device__ __forceinline__ Stat row_stat(const float4& f, float c, unsigned long long* key) {
  Stat st = {f.x, f.y};
  st.merge_lanes(c);
  *key = warp_umax64((static_cast<unsigned long long>(__float_as_uint(f.z)) << 32) | __float_as_uint(f.w));
  return st;
}

// exp((x - m) / T) to 2^-22, x <= m: the difference with its rounding error, the exponent's whole part taken off exactly.
__device__ __forceinline__ float weight(float x, float m, const Heat& c) {
  if (m == -INFINITY) return 0.f;         // a row without tokens
  if (x == m) return 1.f;
  const float d = x - m;
  const float back = d - x;
  const float off = (x - (d - back)) - (m + back);
  const float t = d * c.hi;
  if (!(t > -125.f)) return 0.f;          // -inf among them
  const float j = rintf(t);
  const float f = fmaf(d, c.hi, -j) + fmaf(d, c.lo, off * c.hi);
  return ex2_approx(f) * __int_as_float((static_cast<int>(j) + 127) << 23);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__global__ void __launch_bounds__(kDrawThreads) sample_draw_kernel(const SampleParams p) {
  constexpr int kUnroll = 4;
  __shared__ int s_first;
  __shared__ Stat s_stat;
  __shared__ unsigned long long s_greedy;
  __shared__ unsigned long long s_keys[kDrawWarps];
  __shared__ bool s_last;
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  // Inputs of the callers' (complete since the first kernel let this one start): the first drafts of a warp, and the noise of
  // a thread's first tokens.
  const int r0 = p.cu_rows[b], r1 = p.cu_rows[b + 1], total = p.cu_rows[p.num_seqs];
  const float temperature = p.temperature[b];
  const float* noise = p.noise + static_cast<size_t>(b) * p.vocab;
  const int v0 = blockIdx.x * p.draw_seg, v1 = min(p.vocab, v0 + p.draw_seg);
  float es[kUnroll];
  auto load_noise = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int v = i0 + k * kDrawThreads;
      es[k] = v < v1 ? noise[v] : 0.f;
    }
  };
  load_noise(v0 + threadIdx.x);
  const int depth = r1 - r0 - 1;
  const int d0 = r0 - b;                  // drafts of the sequence (every sequence before it has a row)
  // (a sequence without rows behind it shifts the places of its drafts: they may end behind the total - num_seqs there are.
  // The caller has as many as max_rows allow, whatever the total says: none, and no arrays for them, up to num_seqs rows.)
  const int rows = min(total, p.max_rows);
  const bool bad = d0 < 0 || depth < 0 || r1 > rows || (depth > 0 && d0 + depth > rows - p.num_seqs);
  int token = -1;
  float u = 0.f, q = 1.f, x = -INFINITY;
  auto load_draft = [&](int j) {
    token = p.drafts[d0 + j];
    u = p.uniform[d0 + j];
    const bool known = token >= 0 && token < p.vocab;
    q = known && p.probs != nullptr ? p.probs[static_cast<size_t>(d0 + j) * p.vocab + token] : 1.f;
    x = known ? entry<BF16>(row_at<BF16>(p, r0 + j), token) : -INFINITY;
  };
  if (!bad && warp < depth) load_draft(warp);
  float xs[kUnroll];
  auto load_logits = [&](int n, int i0) {
    const void* src = row_at<BF16>(p, r0 + n);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int v = i0 + k * kDrawThreads;
      xs[k] = v < v1 ? fmaxf(entry<BF16>(src, v), -INFINITY) : -INFINITY;
    }
  };
  if (!bad && depth == 0) load_logits(0, v0 + threadIdx.x);   // nothing to accept: this is the row to draw from
  if (threadIdx.x == 0) s_first = depth;
  pdl_wait();
  if (bad || (blockIdx.x == 0 && !is_temperature(temperature))) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    if (bad) return;
  }
  __syncthreads();
  const Heat c = heat_of(temperature);
  // A warp takes every sixteenth row (the one behind the drafts among them) and stops at its first refusal: the statistics
  // that it then holds are the row's to draw from, if no other warp stops before.
  auto load_parts = [&](int j) {
    return j <= depth && lane < p.parts ? p.stats[static_cast<size_t>(r0 + j) * p.parts + lane]
                                        : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  };
  Stat st = {-INFINITY, 0.f};
  unsigned long long greedy = 0ull;
  int j = warp;
  float4 part = load_parts(j);
  for (; j <= depth; j += kDrawWarps) {
    const float4 next = load_parts(j + kDrawWarps);
    if (j != warp && j < depth) load_draft(j);
    st = row_stat(part, c.hi, &greedy);
    part = next;
    if (j == depth) break;
    const bool known = token >= 0 && token < p.vocab;
    if (!known && lane == 0 && blockIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    float prob;
    if (c.hi > 0.f)
      prob = st.z > 0.f ? weight(fmaxf(x, -INFINITY), st.m, c) / st.z : 0.f;
    else
      prob = token == unpack_index(greedy) ? 1.f : 0.f;
    // u q < prob exactly: where the rounded product equals prob, fp64 holds the whole one.
    const float uq = u * q;
    const bool stays =
        known && (uq < prob || (uq == prob && static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(prob)));
    if (!stays) {
      if (lane == 0) atomicMin(&s_first, j);
      break;
    }
  }
  __syncthreads();
  const int n = s_first;
  if (j == n && lane == 0) {
    s_stat = st;
    s_greedy = greedy;
  }
  __syncthreads();
  st = s_stat;
  greedy = s_greedy;

  int bonus = 0;
  if (c.hi > 0.f) {
    const int draft = n < depth ? p.drafts[d0 + n] : -1;
    const float* qs = draft >= 0 && draft < p.vocab && p.probs != nullptr ? p.probs + static_cast<size_t>(d0 + n) * p.vocab : nullptr;
    const float inv_z = st.z > 0.f ? 1.f / st.z : 0.f;
    // max(p - taken, 0) / E, 0 where E is no exponential
    auto race = [&](float x, float e, float taken) {
      const float w = fmaxf(weight(x, st.m, c) * inv_z - taken, 0.f);
      // (a factor to 2^-23 in place of a division, where it is no denormal)
      if (e > 1e-36f && e < 1e36f) return w * rcp_approx(e);
      return e > 0.f && e < INFINITY ? w / e : 0.f;
    };
    // The largest, with its first index, of a thread, a warp, the CTA (thread 0).
    auto cta_max = [&](unsigned long long key) {
      key = warp_umax64(key);
      if (lane == 0) s_keys[warp] = key;
      __syncthreads();
      return warp == 0 ? warp_umax64(lane < kDrawWarps ? s_keys[lane] : 0ull) : 0ull;
    };
    float best = 0.f;
    int index = -1;
    // (a round's entries are asked for before the one before is weighed)
    float ps[kUnroll];
    auto load_taken = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int v = i0 + k * kDrawThreads;
        ps[k] = qs != nullptr && v < v1 ? qs[v] : (v == draft ? 1.f : 0.f);
      }
    };
    if (depth != 0) load_logits(n, v0 + threadIdx.x);
    load_taken(v0 + threadIdx.x);
    for (int i0 = v0 + threadIdx.x; i0 < v1; i0 += kDrawThreads * kUnroll) {
      float x[kUnroll], e[kUnroll], taken[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) x[k] = xs[k], e[k] = es[k], taken[k] = ps[k];
      const int next = i0 + kDrawThreads * kUnroll;
      if (next < v1) {
        load_noise(next);
        load_logits(n, next);
        load_taken(next);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const float t = race(x[k], e[k], taken[k]);
        if (t > best) best = t, index = i0 + k * kDrawThreads;
      }
    }
    unsigned long long key = cta_max(index >= 0 ? pack(best, index) : 0ull);
    if (threadIdx.x == 0) {
      if (key != 0ull) atomicMax(p.keys + b, key);
      // (the add releases the key; the finishing CTA acquires)
      unsigned int ticket;
      asm volatile("fence.acq_rel.gpu;\n\tatom.add.relaxed.gpu.global.u32 %0, [%1], 1;"
                   : "=r"(ticket)
                   : "l"(p.counters + b)
                   : "memory");
      s_last = ticket == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    key = __ldcg(p.keys + b);
    // Nothing left to draw, which is rare (the drafter's q nowhere below p, noise that is none): this CTA alone draws from p,
    // and where that leaves nothing either takes the largest logit, or token 0.
    for (int mode = n < depth ? 0 : 1; mode < 2 && key == 0ull; ++mode) {
      for (int v = threadIdx.x; v < p.vocab; v += kDrawThreads) {
        const float x = fmaxf(entry<BF16>(row_at<BF16>(p, r0 + n), v), -INFINITY);
        const float t = mode == 0 ? race(x, noise[v], 0.f) : x;
        if (t > (mode == 0 ? 0.f : -INFINITY)) key = umax64(key, pack(t, v));
      }
      __syncthreads();
      key = cta_max(key);
      if (threadIdx.x == 0) s_greedy = key;
      __syncthreads();
      key = s_greedy;
    }
    bonus = key != 0ull ? unpack_index(key) : 0;
    __syncthreads();
    // Leave the workspace as this call found it.
    if (threadIdx.x == 0) {
      p.keys[b] = 0ull;
      p.counters[b] = 0u;
    }
  } else {
    if (blockIdx.x != 0) return;
    bonus = unpack_index(greedy);
  }
  for (int j = threadIdx.x; j <= depth; j += kDrawThreads)
    p.committed[r0 + j] = j < n ? p.drafts[d0 + j] : (j == n ? bonus : -1);
  if (threadIdx.x == 0) {
    p.accepted_len[b] = n;
    p.bonus[b] = bonus;
  }
}

template <bool BF16>
cudaError_t launch_typed(const SampleParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(sample_stats_kernel<BF16>, dim3(p.parts, p.max_rows), dim3(kThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(sample_draw_kernel<BF16>, dim3(p.draw_parts, p.num_seqs), dim3(kDrawThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_accept_sampled(const SampleParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_typed<true>(p, stream) : launch_typed<false>(p, stream);
}

}  // namespace vfy
