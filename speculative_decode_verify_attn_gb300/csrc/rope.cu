// Per-head normalisation and position rotation of a block's queries and keys, with keys and values written straight to
// rows, to the chunk store and pool, or to the position ring.
//     x^ = x * w / sqrt(mean(x^2) + eps);   (a, b) -> (a cos t - b sin t, a sin t + b cos t),   t = position * inv_freq
// in fp32, rounded once to bf16.
//
// One CTA per block token. Its first rot_dim / 2 threads work out the token's cosines and sines once, in shared memory:
// the turns position * inv_freq / 2 pi reduced to [-1/2, 1/2] in fp64 (at position 262144 an fp32 product is off by 1/64
// radian), then fp32. A warp takes one head row at a time: 32 lanes of d / 32 neighbouring channels, the mean by
// shuffles, the partner of a pair by one shuffle per channel.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
enum { kRows = 0, kFull = 1, kRing = 2 };

// HD / 32 bf16 values of one lane as fp32.
template <int PER>
struct Vals {
  float x[PER];
};

template <int PER>
__device__ __forceinline__ Vals<PER> unpack_bf16(const uint32_t (&u)[PER / 2]) {
  Vals<PER> v;
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    v.x[2 * i] = __uint_as_float(u[i] << 16);
    v.x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return v;
}

template <int PER>
__device__ __forceinline__ void load_words(const uint16_t* at, uint32_t (&u)[PER / 2]) {
  if constexpr (PER == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    u[0] = w.x;
    u[1] = w.y;
  } else {
    u[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

template <int PER>
__device__ __forceinline__ void store_words(uint16_t* at, const uint32_t (&u)[PER / 2]) {
  if constexpr (PER == 4)
    *reinterpret_cast<uint2*>(at) = make_uint2(u[0], u[1]);
  else
    *reinterpret_cast<uint32_t*>(at) = u[0];
}

template <int HD, int DST>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int PER = HD / 32;
  __shared__ float s_cos[HD / 2], s_sin[HD / 2];
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (t >= p.cu_q[p.num_seqs]) return;
  const int b = sequence_of(p.cu_q, p.num_seqs, t, lane);
  const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0, L = p.seq_len[b];
  const int i = t - q0;
  if (q0 < 0 || nq < 1 || nq > p.max_q || L < nq || i < 0 || i >= nq || q0 > p.token_cap - nq) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const long long pos = static_cast<long long>(L) - nq + i;
  const int half = p.rot / 2;
  if (threadIdx.x < half) {
    const long long at = p.depth != nullptr ? static_cast<long long>(L) - nq + p.depth[t] : pos;
    const double turns = static_cast<double>(at) * static_cast<double>(p.inv_freq[threadIdx.x]) * 0.15915494309189535;
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    s_cos[threadIdx.x] = c * p.factor;
    s_sin[threadIdx.x] = s * p.factor;
  }
  __syncthreads();

  // Where the token's K and V go.
  uint16_t* kd[2] = {nullptr, nullptr};   // [copy], row of KV head 0
  uint16_t* vd[2] = {nullptr, nullptr};
  size_t head_step = HD;                  // values between the rows of two KV heads
  if constexpr (DST == kRows) {
    if (p.k_dst != nullptr) kd[0] = p.k_dst + static_cast<size_t>(t) * p.hkv * HD;
  } else if constexpr (DST == kRing) {
    const int R = p.ring_len;
    const int phi = ((p.ring_off[b] % R) + R) % R;
    const size_t at = (static_cast<size_t>(b) * p.hkv * R + static_cast<size_t>((pos + phi) % R)) * HD;
    kd[0] = p.k_dst + at;
    vd[0] = p.v_dst + at;
    head_step = static_cast<size_t>(R) * HD;
  } else {
    const long long chunk = static_cast<long long>(p.cu_chunks[b]) + pos / kChunk;
    const size_t row = static_cast<size_t>(pos % kChunk) * HD;
    head_step = static_cast<size_t>(kChunk) * HD;
    if (chunk < 0 || chunk >= p.num_host_chunks) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    } else {
      const size_t at = static_cast<size_t>(chunk) * p.hkv * head_step + row;
      kd[0] = p.host_k + at;
      vd[0] = p.host_v + at;
      const int slot = p.slot_of_chunk[chunk];
      if (slot >= 0 && slot < p.num_slots) {
        const size_t in_pool = static_cast<size_t>(slot) * p.hkv * head_step + row;
        kd[1] = p.k_dst + in_pool;
        vd[1] = p.v_dst + in_pool;
      }
    }
  }

  // This lane's channels are PER * lane + x; their partners sit half channels away (halves) or beside them.
  const int first = lane * PER;
  const bool turned = first < p.rot;
  const int reach = half / PER;           // lanes between partners (halves)
  const int partner = p.interleaved ? lane : (first < half ? lane + reach : lane - reach);
  const int f0 = p.interleaved ? first / 2 : (first < half ? first : first - half);
  const int nq_heads = p.q != nullptr ? p.hq : 0;
  const int nk_heads = p.k != nullptr ? p.hkv : 0;
  const int nv_heads = DST != kRows ? p.hkv : 0;
  for (int job = warp; job < nq_heads + nk_heads + nv_heads; job += kWarps) {
    uint32_t u[PER / 2];
    if (job >= nq_heads + nk_heads) {     // V passes as it is
      const int h = job - nq_heads - nk_heads;
      load_words<PER>(p.v + static_cast<size_t>(t) * p.v_stride + h * HD + first, u);
      if (vd[0] != nullptr) store_words<PER>(vd[0] + h * head_step + first, u);
      if (vd[1] != nullptr) store_words<PER>(vd[1] + h * head_step + first, u);
      continue;
    }
    const bool is_q = job < nq_heads;
    const int h = is_q ? job : job - nq_heads;
    load_words<PER>((is_q ? p.q + static_cast<size_t>(t) * p.q_stride : p.k + static_cast<size_t>(t) * p.k_stride) +
                        h * HD + first,
                    u);
    Vals<PER> v = unpack_bf16<PER>(u);
    const uint16_t* norm = is_q ? p.q_norm : p.k_norm;
    if (norm != nullptr) {
      float sq = 0.f;
#pragma unroll
      for (int x = 0; x < PER; ++x) sq = fmaf(v.x[x], v.x[x], sq);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      const float inv = 1.f / sqrtf(sq * (1.f / HD) + p.eps);
      uint32_t wu[PER / 2];
      load_words<PER>(norm + first, wu);
      const Vals<PER> w = unpack_bf16<PER>(wu);
#pragma unroll
      for (int x = 0; x < PER; ++x) v.x[x] = v.x[x] * inv * w.x[x];
    }
    if (p.rot > 0) {
      Vals<PER> r = v;
      if (p.interleaved) {
        if (turned) {
#pragma unroll
          for (int x = 0; x < PER; x += 2) {
            const float c = s_cos[f0 + x / 2], s = s_sin[f0 + x / 2];
            r.x[x] = v.x[x] * c - v.x[x + 1] * s;
            r.x[x + 1] = v.x[x] * s + v.x[x + 1] * c;
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          const float other = __shfl_sync(0xffffffffu, v.x[x], partner & 31);
          if (turned) {
            const float c = s_cos[f0 + x], s = s_sin[f0 + x];
            r.x[x] = first < half ? v.x[x] * c - other * s : v.x[x] * c + other * s;
          }
        }
      }
      v = r;
    }
#pragma unroll
    for (int x = 0; x < PER / 2; ++x) {
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(v.x[2 * x], v.x[2 * x + 1]);
      u[x] = *reinterpret_cast<const uint32_t*>(&h2);
    }
    if (is_q) {
      store_words<PER>(p.q_out + (static_cast<size_t>(t) * p.hq + h) * HD + first, u);
    } else {
      if (kd[0] != nullptr) store_words<PER>(kd[0] + h * head_step + first, u);
      if (kd[1] != nullptr) store_words<PER>(kd[1] + h * head_step + first, u);
    }
  }
}

template <int HD>
cudaError_t launch_hd(const RopeParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.token_cap));
  if (p.ring_off != nullptr) return launch_pdl(rope_kernel<HD, kRing>, grid, dim3(kThreads), 0, stream, p);
  if (p.cu_chunks != nullptr) return launch_pdl(rope_kernel<HD, kFull>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(rope_kernel<HD, kRows>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_hd<128>(p, stream) : launch_hd<64>(p, stream);
}

}  // namespace vfy
