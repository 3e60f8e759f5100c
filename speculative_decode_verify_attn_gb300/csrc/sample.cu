// Acceptance of sampled drafts. With p_r = softmax(x_r / T) of the target's row r and q_j the drafter's distribution:
//     draft j (token d) stays iff u_j q_j(d) < p_j(d);   n = the first that does not, or D
//     next token = argmax_v w_v / E_v,   w = max(p_n - q_n, 0) for n < D, p_D for n = D
// With E exponentially distributed the argmax of w_v / E_v is a draw in proportion to w (the smallest of independent
// exponential times E_v / w_v). It needs no running sum over the vocabulary, whose order would decide draws near the
// borders of 100,000 tokens: here only two tokens whose times agree to 2^-21 can change places.
//
// Two kernels. The first reads every row once: each CTA takes a segment of one row and leaves its maximum and its sum of
// exponentials against that maximum (greedy rows: the key of the argmax, argmax.cuh). The second has one row of CTAs for
// each sequence; each of them merges the row statistics, finds n, and races its segment of row n; the last one to finish
// (a ticket) writes the outputs.
#include <cuda_bf16.h>

#include "argmax.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// log2(e) / T in two pieces. A tiny T is held at 2^-100: any two different logits are then further apart than fp32 can
// weigh. T = 0 (or one that is no temperature, which is reported) is greedy: 0.
struct Heat {
  float hi, lo;
};
__device__ __forceinline__ bool is_temperature(float t) { return t >= 0.f && t < INFINITY; }
__device__ __forceinline__ Heat heat_of(float t) {
  Heat h = {0.f, 0.f};
  if (is_temperature(t) && t > 0.f) {
    const double c = 1.4426950408889634 / static_cast<double>(fmaxf(t, 7.9e-31f));
    h.hi = static_cast<float>(c);
    h.lo = static_cast<float>(c - static_cast<double>(h.hi));
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

// 2^((a - top) c) where a <= top: the weight of a part whose maximum is a.
__device__ __forceinline__ float rescale(float a, float top, float c) {
  return a == top ? 1.f : ex2_approx((a - top) * c);
}

// Maximum and sum of exponentials of some entries of a row.
struct Stat {
  float m, z;
  __device__ __forceinline__ void merge(const Stat& o, float c) {
    const float top = fmaxf(m, o.m);
    z = z * rescale(m, top, c) + o.z * rescale(o.m, top, c);
    m = top;
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float c) {
    float top = x[0];
#pragma unroll
    for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
    if (top > m) {
      z *= rescale(m, top, c);
      m = top;
    }
    if (m == INFINITY) {                  // +inf entries share the row
#pragma unroll
      for (int e = 0; e < N; ++e) z += x[e] == INFINITY ? 1.f : 0.f;
    } else if (m != -INFINITY) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < N; ++e) s[e & 3] += ex2_approx((x[e] - m) * c);
      z += (s[0] + s[1]) + (s[2] + s[3]);
    }
  }
};

// ------------------------------ row statistics ----------------------------------------------
template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_stats_kernel(const SampleParams p) {
  constexpr int kVec = BF16 ? 8 : 4;      // entries of a 16-byte word
  constexpr int kUnroll = 4;
  __shared__ Stat s_stat[kWarps];
  __shared__ unsigned long long s_key[kWarps];
  pdl_wait();
  // The second kernel starts reading the callers' inputs before it waits for this one: they are complete from here on.
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.y;
  const int total = p.cu_rows[p.num_seqs];
  if (row >= total) return;
  const int b = sequence_of(p.cu_rows, p.num_seqs, row, lane);
  const float c = heat_of(p.temperature[b]).hi;
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
  for (int i0 = threadIdx.x; i0 < words; i0 += kThreads * kUnroll) {
    float x[kUnroll * kVec];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      const uint32_t none = BF16 ? 0xff80ff80u : 0xff800000u;
      const uint4 w = i < words ? __ldg(body + i) : make_uint4(none, none, none, none);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (BF16) {
          x[u * 8 + 2 * e] = __uint_as_float(ws[e] << 16);
          x[u * 8 + 2 * e + 1] = __uint_as_float(ws[e] & 0xffff0000u);
        } else {
          x[u * 4 + e] = __uint_as_float(ws[e]);
        }
      }
    }
    if (c > 0.f) {
#pragma unroll
      for (int e = 0; e < kUnroll * kVec; ++e) x[e] = fmaxf(x[e], -INFINITY);   // NaN -> -inf
      st.add(x, c);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (i0 + u * kThreads < words)
            key = umax64(key, pack(x[u * kVec + e], v0 + head + (i0 + u * kThreads) * kVec + e));
    }
  }
  // (fewer than kVec entries on each side)
  if (threadIdx.x < 2 * kVec) {
    const int v = threadIdx.x < kVec ? v0 + static_cast<int>(threadIdx.x) : tail + static_cast<int>(threadIdx.x) - kVec;
    if (threadIdx.x < kVec ? v < v0 + head : v < v1) {
      const float x[1] = {entry<BF16>(src, v)};
      if (c > 0.f) {
        const float y[1] = {fmaxf(x[0], -INFINITY)};
        st.add(y, c);
      } else {
        key = umax64(key, pack(x[0], v));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat other = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.z, o)};
    st.merge(other, c);
    key = umax64(key, __shfl_xor_sync(0xffffffffu, key, o));
  }
  if (lane == 0) {
    s_stat[warp] = st;
    s_key[warp] = key;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) {
      st.merge(s_stat[w], c);
      key = umax64(key, s_key[w]);
    }
    p.stats[static_cast<size_t>(row) * p.parts + blockIdx.x] =
        make_float4(st.m, st.z, __uint_as_float(static_cast<uint32_t>(key >> 32)), __uint_as_float(static_cast<uint32_t>(key)));
  }
}

// ------------------------------ acceptance and draw ------------------------------------------
// A whole row's statistics, merged by a converged warp (all lanes get them).
__device__ __forceinline__ Stat row_stat(const SampleParams& p, int row, float c, int lane, unsigned long long* key) {
  Stat st = {-INFINITY, 0.f};
  unsigned long long k = 0ull;
  for (int i = lane; i < p.parts; i += 32) {
    const float4 f = p.stats[static_cast<size_t>(row) * p.parts + i];
    const Stat part = {f.x, f.y};
    st.merge(part, c);
    k = umax64(k, (static_cast<unsigned long long>(__float_as_uint(f.z)) << 32) | __float_as_uint(f.w));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat other = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.z, o)};
    st.merge(other, c);
    k = umax64(k, __shfl_xor_sync(0xffffffffu, k, o));
  }
  *key = k;
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

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_draw_kernel(const SampleParams p) {
  constexpr int kUnroll = 4;
  __shared__ int s_first;
  __shared__ unsigned long long s_keys[3][kWarps];
  __shared__ bool s_last;
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  // Inputs of the callers' (complete since the first kernel let this one start), of a warp's first row.
  const int r0 = p.cu_rows[b], r1 = p.cu_rows[b + 1], total = p.cu_rows[p.num_seqs];
  const float temperature = p.temperature[b];
  const int depth = r1 - r0 - 1;
  const int d0 = r0 - b;                  // drafts of the sequence (every sequence before it has a row)
  const bool bad = d0 < 0 || depth < 0 || r1 > min(total, p.max_rows);
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
  if (threadIdx.x == 0) s_first = depth;
  pdl_wait();
  if (bad || (blockIdx.x == 0 && !is_temperature(temperature))) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    if (bad) return;
  }
  __syncthreads();
  const Heat c = heat_of(temperature);
  for (int j = warp; j < depth; j += kWarps) {
    if (j != warp) load_draft(j);
    unsigned long long key;
    const Stat st = row_stat(p, r0 + j, c.hi, lane, &key);
    const bool known = token >= 0 && token < p.vocab;
    if (!known && lane == 0 && blockIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    float prob;
    if (c.hi > 0.f)
      prob = st.z > 0.f ? weight(fmaxf(x, -INFINITY), st.m, c) / st.z : 0.f;
    else
      prob = token == unpack_index(key) ? 1.f : 0.f;
    const bool stays = known && static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(prob);
    if (!stays && lane == 0) atomicMin(&s_first, j);
  }
  __syncthreads();
  const int n = s_first, row = r0 + n;
  unsigned long long greedy;
  const Stat st = row_stat(p, row, c.hi, lane, &greedy);

  int bonus = 0;
  if (c.hi > 0.f) {
    const int refused = n < depth ? p.drafts[d0 + n] : -1;
    const float* qs = n < depth && p.probs != nullptr && refused >= 0 && refused < p.vocab
                          ? p.probs + static_cast<size_t>(d0 + n) * p.vocab
                          : nullptr;
    const void* src = row_at<BF16>(p, row);
    const float* noise = p.noise + static_cast<size_t>(b) * p.vocab;
    const int v0 = blockIdx.x * p.draw_seg, v1 = min(p.vocab, v0 + p.draw_seg);
    const float inv_z = st.z > 0.f ? 1.f / st.z : 0.f;
    // The best of w, of p and of the logits, each with its first index.
    float best[3] = {0.f, 0.f, -INFINITY};
    int index[3] = {-1, -1, -1};
    for (int i0 = v0 + threadIdx.x; i0 < v1; i0 += kThreads * kUnroll) {
      float xs[kUnroll], es[kUnroll], ps[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int v = i0 + k * kThreads;
        const bool in = v < v1;
        xs[k] = in ? fmaxf(entry<BF16>(src, v), -INFINITY) : -INFINITY;
        es[k] = in ? noise[v] : 0.f;
        ps[k] = in && qs != nullptr ? qs[v] : (v == refused ? 1.f : 0.f);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int v = i0 + k * kThreads;
        const float prob = weight(xs[k], st.m, c) * inv_z;
        const bool drawn = es[k] > 0.f && es[k] < INFINITY;
        const float race = drawn ? prob / es[k] : 0.f;
        const float left = drawn ? fmaxf(prob - ps[k], 0.f) / es[k] : 0.f;
        if (left > best[0]) best[0] = left, index[0] = v;
        if (race > best[1]) best[1] = race, index[1] = v;
        if (xs[k] > best[2]) best[2] = xs[k], index[2] = v;
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      unsigned long long key = index[k] >= 0 ? pack(best[k], index[k]) : 0ull;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) key = umax64(key, __shfl_xor_sync(0xffffffffu, key, o));
      if (lane == 0) s_keys[k][warp] = key;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int k = 0; k < 3; ++k) {
        unsigned long long key = s_keys[k][0];
        for (int w = 1; w < kWarps; ++w) key = umax64(key, s_keys[k][w]);
        if (key != 0ull) atomicMax(p.keys + 3 * b + k, key);
      }
      // (the add releases this CTA's keys; the finishing CTA acquires)
      unsigned int ticket;
      asm volatile("atom.add.release.gpu.global.u32 %0, [%1], 1;" : "=r"(ticket) : "l"(p.counters + b) : "memory");
      s_last = ticket == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    bonus = 0;                            // nothing to draw and no logit above -inf: token 0
    for (int k = 2; k >= 0; --k) {
      const unsigned long long key = __ldcg(p.keys + 3 * b + k);
      if (key != 0ull) bonus = unpack_index(key);
    }
    __syncthreads();
    // Leave the workspace as this call found it.
    if (threadIdx.x < 3) p.keys[3 * b + threadIdx.x] = 0ull;
    if (threadIdx.x == 3) p.counters[b] = 0u;
  } else {
    if (blockIdx.x != 0) return;
    bonus = unpack_index(greedy);
  }
  for (int j = threadIdx.x; j <= depth; j += kThreads)
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
  return launch_pdl(sample_draw_kernel<BF16>, dim3(p.draw_parts, p.num_seqs), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_accept_sampled(const SampleParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_typed<true>(p, stream) : launch_typed<false>(p, stream);
}

}  // namespace vfy
