// Per-head normalisation and position rotation of a block's queries and keys, with keys and values written straight to
// rows, to the chunk store and pool, or to the position ring.
//     x^ = x * w / sqrt(mean(x^2) + eps);   (a, b) -> (a cos t - b sin t, a sin t + b cos t),   t = position * inv_freq
// in fp32, rounded once to bf16.
//
// A CTA of four warps takes one token (few tokens: latency), or a token a warp (8 x 1024 tokens 25 us against 52). The warps of
// a token work out its cosines and sines once, in shared memory. A row of d channels is d / 8 lanes of two groups of four
// channels: the two groups that rotate with one another, so that a pair lies in one lane. Queries, keys and values have a
// loop each, without choices by row, and two rows a lane ahead of the one it works on. The look-up of up to 32 sequences is
// one round trip to memory.
// 17 tokens of 16 + 2 x 4 heads of 128 take 2.9 us (latency), 264 of a batch of trees 3.2, 8 x 1024 24.7 (117 MB, 4.7 TB/s:
// leaving out the angles or the norms changes nothing; CTAs of eight warps 25.7, of two 24.6 but 17 tokens 4.2).
//
// Angles: the turns position * inv_freq / 2 pi modulo 1 (at position 262144 an fp32 product is off by 1/64 radian), with
// inv_freq / 2 pi as the sum of three fp32 values (to 2^-53) and the products exact in pairs (product and fma remainder):
// within 2^-25 turns up to position 2^22 (the last addition), 2^-22 up to 2^31, for frequencies up to 1 in size: 1 / 2 pi has
// 53 bits, so that larger ones add some |inv_freq| position 2^-55. (fp64 has 1/64 of the fp32 rate here.)
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
enum { kRows = 0, kFull = 1, kRing = 2 };

// position * freq / 2 pi, modulo 1
__device__ __forceinline__ float turns_of(long long position, float freq) {
  constexpr double kInv2Pi = 0.15915494309189535;
  constexpr float k0 = static_cast<float>(kInv2Pi), k1 = static_cast<float>(kInv2Pi - static_cast<double>(k0));
  constexpr float k2 = static_cast<float>(kInv2Pi - static_cast<double>(k0) - static_cast<double>(k1));
  // freq / 2 pi = c0 + c1 + c2: a product; its remainder and the next product; their sum's error and what is left
  const float c0 = freq * k0, r = fmaf(freq, k0, -c0);
  const float m = freq * k1, c1 = r + m, back = c1 - r;
  const float c2 = ((r - (c1 - back)) + (m - back)) + fmaf(freq, k2, fmaf(freq, k1, -m));
  const float a1 = static_cast<float>(static_cast<int>(position >> 16)) * 65536.f;   // both exact
  const float a0 = static_cast<float>(static_cast<int>(position & 0xffff));
  const float p1 = a1 * c0, p0 = a0 * c0, p2 = a1 * c1;
  const float e1 = fmaf(a1, c0, -p1), e0 = fmaf(a0, c0, -p0), e2 = fmaf(a1, c1, -p2);
  // (the sum of the first two fractions with its error: what is rounded is the last addition)
  const float f1 = p1 - rintf(p1), f0 = p0 - rintf(p0);
  const float sum = f1 + f0, of0 = sum - f1, error = (f1 - (sum - of0)) + (f0 - of0);
  const float small = ((e1 - rintf(e1)) + (e0 - rintf(e0))) + ((p2 - rintf(p2)) + e2) + (fmaf(a1, c2, a0 * c1) + error);
  return (sum - rintf(sum)) + small;
}

// Where a token's K and V go: the row of KV head 0, of up to two copies. (`origin` of its sequence: cu_chunks, or the ring's
// offset.)
struct Target {
  uint16_t *k[2], *v[2];
};

template <int DST>
__device__ __forceinline__ Target target_of(const RopeParams& p, int HD, int t, int b, int origin, long long pos) {
  Target to = {{nullptr, nullptr}, {nullptr, nullptr}};
  if constexpr (DST == kRows) {
    if (p.k_dst != nullptr) to.k[0] = p.k_dst + static_cast<size_t>(t) * p.hkv * HD;
  } else if constexpr (DST == kRing) {
    const int R = p.ring_len;
    const int phi = (origin % R + R) % R;
    const size_t at = (static_cast<size_t>(b) * p.hkv * R + static_cast<size_t>((pos + phi) % R)) * HD;
    to.k[0] = p.k_dst + at;
    to.v[0] = p.v_dst + at;
  } else {
    const long long chunk = static_cast<long long>(origin) + pos / kChunk;
    const size_t row = static_cast<size_t>(pos % kChunk) * HD, record = static_cast<size_t>(p.hkv) * kChunk * HD;
    if (chunk < 0 || chunk >= p.num_host_chunks) {
      atomicOr(p.err, kErrDeviceInput);
    } else {
      const size_t at = static_cast<size_t>(chunk) * record + row;
      to.k[0] = p.host_k + at;
      to.v[0] = p.host_v + at;
      const int slot = p.slot_of_chunk[chunk];
      if (slot >= 0 && slot < p.num_slots) {
        const size_t in_pool = static_cast<size_t>(slot) * record + row;
        to.k[1] = p.k_dst + in_pool;
        to.v[1] = p.v_dst + in_pool;
      }
    }
  }
  return to;
}

// Two groups of four channels. In pairs (2 i, 2 i + 1): the first of each and the second of each, so that either way a
// channel of `a` rotates with the same of `b`.
struct Words {
  uint2 a, b;
};
__device__ __forceinline__ Words apart(const Words& w) {
  return {make_uint2(__byte_perm(w.a.x, w.a.y, 0x5410), __byte_perm(w.b.x, w.b.y, 0x5410)),
          make_uint2(__byte_perm(w.a.x, w.a.y, 0x7632), __byte_perm(w.b.x, w.b.y, 0x7632))};
}
__device__ __forceinline__ Words together(const Words& w) {
  return {make_uint2(__byte_perm(w.a.x, w.b.x, 0x5410), __byte_perm(w.a.x, w.b.x, 0x7632)),
          make_uint2(__byte_perm(w.a.y, w.b.y, 0x5410), __byte_perm(w.a.y, w.b.y, 0x7632))};
}
__device__ __forceinline__ float2 floats(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rows of one kind (queries, keys or values) of a token: a warp takes `kPer` neighbours at a time, `warps` warps in turn.
template <int HD, int AHEAD>
struct Loader {
  static constexpr int kPer = 32 / (HD / 8);
  const uint16_t* from;                   // this lane's first group in row `sub`
  int dc, sub, rows, first, warps;        // second group - first; the warp's first job
  Words ahead[AHEAD];
  __device__ __forceinline__ Words load(int job) const {
    Words w = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
    if (job * kPer + sub < rows) {
      const uint16_t* at = from + static_cast<size_t>(job) * (kPer * HD);
      w.a = *reinterpret_cast<const uint2*>(at);
      w.b = *reinterpret_cast<const uint2*>(at + dc);
    }
    return w;
  }
  __device__ __forceinline__ void start(const uint16_t* f, int d, int s, int r, int j, int w) {
    from = f;
    dc = d;
    sub = s;
    rows = r;
    first = j;
    warps = w;
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) ahead[x] = load(first + x * warps);
  }
  // f(words, row, whether the row is one) by all lanes of the warp
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    for (int j0 = first; j0 * kPer < rows; j0 += AHEAD * warps) {
#pragma unroll
      for (int x = 0; x < AHEAD; ++x) {
        const int j = j0 + x * warps;
        if (j * kPer >= rows) break;
        const Words w = ahead[x];
        ahead[x] = load(j + AHEAD * warps);
        f(w, j * kPer + sub, j * kPer + sub < rows);
      }
    }
  }
};

template <int HD, int DST>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeParams p) {
  constexpr int kLanes = HD / 8, kPer = 32 / kLanes;    // lanes of a row, rows of a warp at a time
  __shared__ float4 s_cos[kWarps][HD / 8], s_sin[kWarps][HD / 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = kWarps / p.tokens_per_cta;          // of a token
  const int k = warp / warps, wi = warp - k * warps;
  const int t = blockIdx.x * p.tokens_per_cta + k;
  pdl_launch_dependents();
  pdl_wait();

  // The token's sequence: up to 32 are looked up by a lane each.
  const int32_t* origins = DST == kFull ? p.cu_chunks : DST == kRing ? p.ring_off : nullptr;
  int total, b, q0 = 0, q1 = 0, L = 0, origin = 0;
  if (p.num_seqs <= 32) {
    int lo = 0, hi = INT_MAX, len = 0, from = 0;
    if (lane < p.num_seqs) {
      lo = p.cu_q[lane];
      hi = p.cu_q[lane + 1];
      len = p.seq_len[lane];
      if (DST != kRows) from = origins[lane];
    }
    total = __shfl_sync(0xffffffffu, hi, p.num_seqs - 1);
    b = min(__popc(__ballot_sync(0xffffffffu, hi <= t)), p.num_seqs - 1);
    q0 = __shfl_sync(0xffffffffu, lo, b);
    q1 = __shfl_sync(0xffffffffu, hi, b);
    L = __shfl_sync(0xffffffffu, len, b);
    if (DST != kRows) origin = __shfl_sync(0xffffffffu, from, b);
  } else {
    total = p.cu_q[p.num_seqs];
    b = sequence_of(p.cu_q, p.num_seqs, t, lane);
    q0 = p.cu_q[b];
    q1 = p.cu_q[b + 1];
    L = p.seq_len[b];
    if (DST != kRows) origin = origins[b];
  }
  const int nq = q1 - q0, i = t - q0;
  bool live = t < total;
  if (live && (q0 < 0 || nq < 1 || nq > p.max_q || L < nq || i < 0 || i >= nq || q0 > p.token_cap - nq)) {
    if (wi == 0 && lane == 0) atomicOr(p.err, kErrDeviceInput);
    live = false;
  }
  const long long start = static_cast<long long>(L) - nq, pos = start + i;

  // This lane's channels: two groups of four that rotate with one another (halves), or are neighbours.
  const int li = lane % kLanes, sub = lane / kLanes, half = p.rot / 2;
  const bool turned = li < half / 4;
  int c0 = 8 * li, c1 = c0 + 4;
  if (!p.interleaved) {
    c0 = turned ? 4 * li : p.rot + 8 * (li - half / 4);
    c1 = turned ? half + 4 * li : c0 + 4;
  }
  const int dc = c1 - c0, at = sub * HD + c0;
  const int nq_heads = live && p.q != nullptr ? p.hq : 0, nk_heads = live && p.k != nullptr ? p.hkv : 0;
  const int nv_heads = live && DST != kRows ? p.hkv : 0;
  // (keys first, then values and queries: a warp's first jobs of each)
  const int k_jobs = (nk_heads + kPer - 1) / kPer, v_jobs = (nv_heads + kPer - 1) / kPer;
  Loader<HD, 2> keys, values, queries;
  keys.start(p.k + t * p.k_stride + at, dc, sub, nk_heads, wi, warps);
  values.start(p.v + t * p.v_stride + at, dc, sub, nv_heads, (wi + k_jobs) & (warps - 1), warps);
  queries.start(p.q + t * p.q_stride + at, dc, sub, nq_heads, (wi + k_jobs + v_jobs) & (warps - 1), warps);

  if (live) {
    const long long turn_pos = p.depth != nullptr ? start + p.depth[t] : pos;
    for (int x = wi * 32 + lane; x < half; x += warps * 32) {
      float s, c;
      sincospif(2.f * turns_of(turn_pos, p.inv_freq[x]), &s, &c);
      reinterpret_cast<float*>(s_cos[k])[x] = c * p.factor;
      reinterpret_cast<float*>(s_sin[k])[x] = s * p.factor;
    }
  }
  Target to = {};
  if (live) to = target_of<DST>(p, HD, t, b, origin, pos);
  const size_t head_step = static_cast<size_t>(DST == kRows ? 1 : DST == kRing ? p.ring_len : kChunk) * HD;
  auto store = [&](uint16_t* row, const Words& w) {
    *reinterpret_cast<uint2*>(row + c0) = w.a;
    *reinterpret_cast<uint2*>(row + c1) = w.b;
  };
  if constexpr (DST != kRows)
    values.each([&](const Words& w, int r, bool in) {
#pragma unroll
      for (int copy = 0; copy < (DST == kFull ? 2 : 1); ++copy)
        if (in && to.v[copy] != nullptr) store(to.v[copy] + r * head_step, w);
    });
  __syncthreads();
  float2 cs[2] = {}, sn[2] = {};
  if (live && turned) {
    const float4 c = s_cos[k][li], s = s_sin[k][li];
    cs[0] = make_float2(c.x, c.y);
    cs[1] = make_float2(c.z, c.w);
    sn[0] = make_float2(s.x, s.y);
    sn[1] = make_float2(s.z, s.w);
  }
  const float2 ns[2] = {make_float2(-sn[0].x, -sn[0].y), make_float2(-sn[1].x, -sn[1].y)};
  auto rows = [&](auto& loader, const uint16_t* norm, auto put) {
    float2 g[4];
    if (norm != nullptr) {
      Words w = {*reinterpret_cast<const uint2*>(norm + c0), *reinterpret_cast<const uint2*>(norm + c1)};
      if (p.interleaved) w = apart(w);
      g[0] = floats(w.a.x);
      g[1] = floats(w.a.y);
      g[2] = floats(w.b.x);
      g[3] = floats(w.b.y);
    }
    loader.each([&](Words w, int r, bool in) {
      if (p.interleaved) w = apart(w);
      float2 v[4] = {floats(w.a.x), floats(w.a.y), floats(w.b.x), floats(w.b.y)};
      if (norm != nullptr) {
        float2 sq = mul_f32x2(v[0], v[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) sq = fma_f32x2(v[e], v[e], sq);
        float sum = sq.x + sq.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, 1.f / HD, p.eps));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul_f32x2(v[e], mul_f32x2(make_float2(inv, inv), g[e]));
      }
      if (turned) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 x = fma_f32x2(v[e + 2], ns[e], mul_f32x2(v[e], cs[e]));
          v[e + 2] = fma_f32x2(v[e], sn[e], mul_f32x2(v[e + 2], cs[e]));
          v[e] = x;
        }
      }
      w = {make_uint2(pack_bf16(v[0]), pack_bf16(v[1])), make_uint2(pack_bf16(v[2]), pack_bf16(v[3]))};
      if (p.interleaved) w = together(w);
      if (in) put(w, r);
    });
  };
  rows(keys, p.k_norm, [&](const Words& w, int r) {
#pragma unroll
    for (int copy = 0; copy < (DST == kFull ? 2 : 1); ++copy)
      if (to.k[copy] != nullptr) store(to.k[copy] + r * head_step, w);
  });
  uint16_t* out = p.q_out + static_cast<size_t>(t) * p.hq * HD;
  rows(queries, p.q_norm, [&](const Words& w, int r) { store(out + r * HD, w); });
}

template <int HD>
cudaError_t launch_hd(const RopeParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.token_cap + p.tokens_per_cta - 1) / p.tokens_per_cta));
  if (p.ring_off != nullptr) return launch_pdl(rope_kernel<HD, kRing>, grid, dim3(kThreads), 0, stream, p);
  if (p.cu_chunks != nullptr) return launch_pdl(rope_kernel<HD, kFull>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(rope_kernel<HD, kRows>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

int rope_cta_tokens() { return kWarps; }

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_hd<128>(p, stream) : launch_hd<64>(p, stream);
}

}  // namespace vfy
