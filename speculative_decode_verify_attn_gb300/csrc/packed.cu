// 4-bit chunks: the block's K/V rows written in 4 bits (append) and chunks read back as bf16 (unpack).
// A record holds one (chunk, KV head) of K or V in 36 d bytes: codes [d / 32][64 tokens][16 bytes], then e4m3 scales
// [64 tokens][d / 16]; a value is g * s * e, e a 4-bit float e2m1. Codes are laid out by 32 channels, so that neighbouring
// tokens' 16-byte words are neighbours: a warp that reads one word for each of 32 tokens reads 512 bytes in a row.
//
// The append gives one thread one group of 16 channels: its scale and its 8 bytes of codes. s * e has 6 significant bits, so
// that the read value is exact in bf16 where g is a power of two.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;

// Jobs of a token: K then V, KV heads, groups of a head; a CTA takes as many whole tokens as it has threads for, and goes
// from tokens to tokens, the next ones' values on their way while these are packed: three CTAs an SM (8 x 1024 tokens of 4 KV
// heads of 128 take 10.5 us in a loop, and 94 into a pinned store, which is the host link; a CTA for every few tokens 4 us
// more). Threads of a token are neighbours, and d / 16 is a multiple of 4: the two groups of a 16-byte code word are a lane and
// the next, and four lanes have four neighbouring scales.
__host__ __device__ __forceinline__ int jobs_of(int hkv, int head_dim) { return 2 * hkv * (head_dim / 16); }
__host__ __device__ __forceinline__ int cta_tokens(int jobs) { return jobs < kThreads ? kThreads / jobs : 1; }
__host__ __device__ __forceinline__ int job_rounds(int jobs) { return (jobs + kThreads - 1) / kThreads; }

// One thread's job: its values, and where their codes go.
struct AppendJob {
  bool live;
  int job, row, slot;
  long long chunk;
  uint4 lo, hi;
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 3) append_packed_kernel(const PackedAppendParams p) {
  constexpr int kGroups = HD / 16;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int jobs = jobs_of(p.hkv, HD), tokens = cta_tokens(jobs), rounds = job_rounds(jobs), per_side = p.hkv * kGroups;
  const int sub = tokens > 1 ? static_cast<int>(threadIdx.x) / jobs : 0, job0 = static_cast<int>(threadIdx.x) - sub * jobs;
  // Up to 32 sequences are looked up by a lane each, in one round trip.
  const bool few = p.num_seqs <= 32;
  int lo = 0, hi = INT_MAX, len = 0, from = 0;
  if (few && lane < p.num_seqs) {
    lo = p.cu_q[lane];
    hi = p.cu_q[lane + 1];
    len = p.seq_len[lane];
    from = p.cu_chunks[lane];
  }
  const int total = min(few ? __shfl_sync(0xffffffffu, hi, p.num_seqs - 1) : p.cu_q[p.num_seqs], p.token_cap);

  // Item `at`: `rounds` items for every `tokens` tokens.
  auto load = [&](long long at) {
    AppendJob a = {};
    const long long group = rounds > 1 ? at / rounds : at;
    a.job = job0 + static_cast<int>(at - group * rounds) * kThreads;
    const int t = static_cast<int>(min(group * tokens + sub, static_cast<long long>(total)));
    int q0, q1, L, first_chunk, b = 0;                      // its sequence, the last that starts at or before it
    if (few) {
#pragma unroll
      for (int step = 16; step > 0; step >>= 1) {
        const int start = __shfl_sync(0xffffffffu, lo, (b + step) & 31);
        if (b + step < p.num_seqs && start <= t) b += step;
      }
      q0 = __shfl_sync(0xffffffffu, lo, b);
      q1 = __shfl_sync(0xffffffffu, hi, b);
      L = __shfl_sync(0xffffffffu, len, b);
      first_chunk = __shfl_sync(0xffffffffu, from, b);
    } else {
      int last = p.num_seqs - 1;
      while (b < last) {
        const int mid = (b + last + 1) >> 1;
        if (p.cu_q[mid] <= t) b = mid; else last = mid - 1;
      }
      q0 = p.cu_q[b];
      q1 = p.cu_q[b + 1];
      L = p.seq_len[b];
      first_chunk = p.cu_chunks[b];
    }
    if (sub >= tokens || t >= total || a.job >= jobs) return a;
    const int nq = q1 - q0, i = t - q0;
    const long long pos = static_cast<long long>(L) - nq + i;
    bool bad = q0 < 0 || nq < 1 || nq > p.max_q || L < nq || i < 0 || i >= nq || q0 > p.token_cap - nq;
    if (!bad) {
      a.chunk = static_cast<long long>(first_chunk) + pos / kChunk;
      bad = a.chunk < 0 || a.chunk >= p.num_host_chunks;
    }
    if (bad) {
      if (a.job == 0) atomicOr(p.err, kErrDeviceInput);
      return a;
    }
    a.live = true;
    a.row = static_cast<int>(pos % kChunk);
    const bool is_v = a.job >= per_side;
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.v_new : p.k_new) + static_cast<size_t>(t) * p.hkv * HD +
                                                      (is_v ? a.job - per_side : a.job) * 16);
    a.lo = src[0];
    a.hi = src[1];
    a.slot = p.slot_of_chunk[a.chunk];
    return a;
  };
  auto pack = [&](const AppendJob& a) {
    const bool is_v = a.job >= per_side;
    const int in_side = is_v ? a.job - per_side : a.job, h = in_side / kGroups, g = in_side % kGroups;
    uint2 codes = make_uint2(0u, 0u);
    uint32_t scale = 0u;
    if (a.live) {
      const uint32_t w[8] = {a.lo.x, a.lo.y, a.lo.z, a.lo.w, a.hi.x, a.hi.y, a.hi.z, a.hi.w};
      float2 x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
      codes = pack_group(x, is_v ? p.v_scale : p.k_scale, is_v ? p.v_inv : p.k_inv, &scale);
    }
    // A pair of lanes holds a 16-byte word of codes; the even one writes it.
    const uint32_t ox = __shfl_xor_sync(0xffffffffu, codes.x, 1), oy = __shfl_xor_sync(0xffffffffu, codes.y, 1);
    // Four lanes hold four neighbouring scale bytes; the first writes them.
    uint32_t scales = scale << (8 * (g & 3));
    scales |= __shfl_xor_sync(0xffffffffu, scales, 1);
    scales |= __shfl_xor_sync(0xffffffffu, scales, 2);
    if (!a.live) return;
    const size_t word = (static_cast<size_t>(g / 2) * kChunk + a.row) * 16;
    const size_t scale_at = static_cast<size_t>(kChunk) * (HD / 2) + static_cast<size_t>(a.row) * kGroups + (g & ~3);
    uint8_t* store = (is_v ? p.host_v : p.host_k) + (static_cast<size_t>(a.chunk) * p.hkv + h) * kPackedBytes<HD>;
    uint8_t* pool = a.slot >= 0 && a.slot < p.num_slots
                        ? (is_v ? p.v_pool : p.k_pool) + (static_cast<size_t>(a.slot) * p.hkv + h) * kPackedBytes<HD>
                        : nullptr;
    if ((g & 1) == 0) {
      const uint4 v = make_uint4(codes.x, codes.y, ox, oy);
      *reinterpret_cast<uint4*>(store + word) = v;
      if (pool != nullptr) *reinterpret_cast<uint4*>(pool + word) = v;
    }
    if ((g & 3) == 0) {
      *reinterpret_cast<uint32_t*>(store + scale_at) = scales;
      if (pool != nullptr) *reinterpret_cast<uint32_t*>(pool + scale_at) = scales;
    }
  };
  const long long items = (static_cast<long long>(total) + tokens - 1) / tokens * rounds;
  if (static_cast<long long>(blockIdx.x) >= items) return;
  AppendJob next = load(blockIdx.x);
  for (long long at = blockIdx.x; at < items; at += gridDim.x) {
    const AppendJob a = next;
    next = load(at + gridDim.x);
    pack(a);
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const UnpackParams p) {
  pdl_launch_dependents();
  pdl_wait();
  // One CTA row (blockIdx.x) per (entry, KV head); K and V by blockIdx.y.
  const unsigned entry = blockIdx.x / static_cast<unsigned>(p.hkv);
  const int h = static_cast<int>(blockIdx.x - entry * p.hkv);
  const int slot = p.slots[entry];
  if (slot < 0 || slot >= p.num_slots) {
    if (threadIdx.x == 0 && h == 0 && blockIdx.y == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const bool is_v = blockIdx.y != 0;
  const uint8_t* rec = (is_v ? p.v_pool : p.k_pool) + (static_cast<size_t>(slot) * p.hkv + h) * kPackedBytes<HD>;
  uint16_t* out = (is_v ? p.v_out : p.k_out) + static_cast<size_t>(blockIdx.x) * kChunk * HD;
  const float gs = is_v ? p.v_scale : p.k_scale;
  // Eight channels a thread and step: 4 bytes of codes in, 16 bytes out, side by side in a warp.
  constexpr int kEights = HD / 8, kMine = kChunk * kEights / kThreads;
  uint32_t codes[kMine], scale[kMine];
#pragma unroll
  for (int y = 0; y < kMine; ++y) {        // (all loads before the first store)
    const int x = threadIdx.x + y * kThreads, row = x / kEights, u = x % kEights;
    codes[y] = *reinterpret_cast<const uint32_t*>(rec + (u / 4 * kChunk + row) * 16 + u % 4 * 4);
    scale[y] = rec[kChunk * (HD / 2) + x / 2];
  }
#pragma unroll
  for (int y = 0; y < kMine; ++y) {
    const float s = e4m3_value(scale[y]), sg = s * gs;
    uint16_t* to = out + static_cast<size_t>(threadIdx.x + y * kThreads) * 8;
    if (plain_product(s, sg)) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = e2m1_pair((codes[y] >> (8 * e)) & 0xffu);
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(v.x * sg, v.y * sg);
        o[e] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float2 v = e2m1_pair((codes[y] >> (8 * e)) & 0xffu);
        *reinterpret_cast<__nv_bfloat162*>(to + 2 * e) =
            __floats2bfloat162_rn(product_to_odd(v.x * s, gs), product_to_odd(v.y * s, gs));
      }
    }
  }
}

}  // namespace

cudaError_t launch_append_packed(const PackedAppendParams& p, cudaStream_t stream) {
  const int jobs = jobs_of(p.hkv, p.head_dim), tokens = cta_tokens(jobs);
  const long long items = (static_cast<long long>(p.token_cap) + tokens - 1) / tokens * job_rounds(jobs);
  const dim3 grid(static_cast<unsigned>(items < 3LL * p.num_sms ? items : 3LL * p.num_sms));   // as many as run at once
  if (p.head_dim == 128) return launch_pdl(append_packed_kernel<128>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(append_packed_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_unpack(const UnpackParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.n) * p.hkv, 2);
  if (p.head_dim == 128) return launch_pdl(unpack_kernel<128>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(unpack_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace vfy
