// 4-bit chunks: the block's K/V rows written in 4 bits (append) and chunks read back as bf16 (unpack).
// A record holds one (chunk, KV head) of K or V in 36 d bytes: codes [d / 32][64 tokens][16 bytes], then e4m3 scales
// [64 tokens][d / 16]; a value is g * s * e, e a 4-bit float e2m1. Codes are laid out by 32 channels, so that neighbouring
// tokens' 16-byte words are neighbours: a warp that reads one word for each of 32 tokens reads 512 bytes in a row.
//
// Both kernels give one thread one group of 16 channels: its scale and its 8 bytes of codes. s * e has 6 significant bits,
// so that the read value is exact in bf16 where g is a power of two.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;

// Group job of token t: K then V, KV heads, groups of a head. Threads of a token are neighbours, and d / 16 is even: the
// two groups of a 16-byte code word are a lane and the next.
template <int HD>
__global__ void __launch_bounds__(kThreads) append_packed_kernel(const PackedAppendParams p) {
  constexpr int kGroups = HD / 16;
  pdl_launch_dependents();
  pdl_wait();
  const unsigned per_token = 2u * p.hkv * kGroups;
  const unsigned long long at = static_cast<unsigned long long>(blockIdx.x) * kThreads + threadIdx.x;
  const unsigned long long tok = at / per_token;
  const unsigned job = static_cast<unsigned>(at - tok * per_token);
  const int total = p.cu_q[p.num_seqs];
  bool live = tok < static_cast<unsigned long long>(p.token_cap) && static_cast<int>(tok) < total;
  const int t = live ? static_cast<int>(tok) : 0;
  int lo = 0, hi = p.num_seqs - 1;                        // the last sequence that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_q[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0, L = p.seq_len[b];
  const int i = t - q0;
  bool bad = q0 < 0 || nq < 1 || nq > p.max_q || L < nq || i < 0 || i >= nq || q0 > p.token_cap - nq;
  const long long pos = static_cast<long long>(L) - nq + i;
  long long chunk = 0;
  if (live && !bad) {
    chunk = static_cast<long long>(p.cu_chunks[b]) + pos / kChunk;
    bad = chunk < 0 || chunk >= p.num_host_chunks;
  }
  if (live && bad && job == 0) atomicOr(p.err, kErrDeviceInput);
  live = live && !bad;

  const unsigned per_head = kGroups, per_side = p.hkv * kGroups;
  const bool is_v = job >= per_side;
  const unsigned in_side = is_v ? job - per_side : job;
  const int h = static_cast<int>(in_side / per_head), g = static_cast<int>(in_side % per_head);
  uint2 codes = make_uint2(0u, 0u);
  uint32_t scale = 0u;
  if (live) {
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.v_new : p.k_new) +
                                                      (static_cast<size_t>(t) * p.hkv + h) * HD + g * 16);
    const uint4 lo4 = src[0], hi4 = src[1];
    const uint32_t w[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
    float x[16];
    const float gs = is_v ? p.v_scale : p.k_scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = __fdiv_rn(__uint_as_float(w[e] << 16), gs);
      x[2 * e + 1] = __fdiv_rn(__uint_as_float(w[e] & 0xffff0000u), gs);
    }
    codes = pack_group(x, &scale);
  }
  // A pair of lanes holds a 16-byte word of codes; the even one writes it. (Lanes of one token: d / 16 is even.)
  const uint32_t ox = __shfl_xor_sync(0xffffffffu, codes.x, 1), oy = __shfl_xor_sync(0xffffffffu, codes.y, 1);
  // Four lanes hold four neighbouring scale bytes; the first writes them. (d / 16 is a multiple of 4.)
  uint32_t scales = scale << (8 * (g & 3));
  scales |= __shfl_xor_sync(0xffffffffu, scales, 1);
  scales |= __shfl_xor_sync(0xffffffffu, scales, 2);
  if (!live) return;
  const int row = static_cast<int>(pos % kChunk);
  const size_t word = (static_cast<size_t>(g / 2) * kChunk + row) * 16;
  const size_t scale_at = static_cast<size_t>(kChunk) * (HD / 2) + static_cast<size_t>(row) * kGroups + (g & ~3);
  const int slot = p.slot_of_chunk[chunk];
  uint8_t* store = (is_v ? p.host_v : p.host_k) + (static_cast<size_t>(chunk) * p.hkv + h) * kPackedBytes<HD>;
  uint8_t* pool = slot >= 0 && slot < p.num_slots
                      ? (is_v ? p.v_pool : p.k_pool) + (static_cast<size_t>(slot) * p.hkv + h) * kPackedBytes<HD>
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
}

template <int HD>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const UnpackParams p) {
  constexpr int kGroups = HD / 16;
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
#pragma unroll
  for (int x = threadIdx.x; x < kChunk * kGroups; x += kThreads) {
    const int row = x / kGroups, g = x % kGroups;
    const uint2 codes =
        *reinterpret_cast<const uint2*>(rec + (static_cast<size_t>(g / 2) * kChunk + row) * 16 + (g & 1) * 8);
    const float s = e4m3_value(rec[kChunk * (HD / 2) + x]) * gs;
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t byte = ((e < 4 ? codes.x : codes.y) >> (8 * (e & 3))) & 0xffu;
      const float2 v = e2m1_pair(byte);
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(v.x * s, v.y * s);
      o[e] = *reinterpret_cast<const uint32_t*>(&h2);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + static_cast<size_t>(x) * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_append_packed(const PackedAppendParams& p, cudaStream_t stream) {
  const unsigned long long jobs = static_cast<unsigned long long>(p.token_cap) * 2 * p.hkv * (p.head_dim / 16);
  const dim3 grid(static_cast<unsigned>((jobs + kThreads - 1) / kThreads));
  if (p.head_dim == 128) return launch_pdl(append_packed_kernel<128>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(append_packed_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_unpack(const UnpackParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.n) * p.hkv, 2);
  if (p.head_dim == 128) return launch_pdl(unpack_kernel<128>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(unpack_kernel<64>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace vfy
