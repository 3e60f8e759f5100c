// Attention of a block over a pool of 4-bit chunks.
#include <cuda_bf16.h>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int HD>
struct Shape {
  static constexpr int kKStride = HD + 1;
  static constexpr int kSmemFloats = kChunk * kKStride + kChunk * HD + kMaxRows * HD + 2 * kMaxRows;
};

// One CTA per (split, KV head, sequence and row tile): its chunks one by one, read as fp32 into shared memory; a warp per
// row, a lane per key, then a lane per channel.
template <int HD>
__global__ void __launch_bounds__(kThreads) attend_packed_kernel(const PackedAttnParams p) {
  constexpr int kStride = Shape<HD>::kKStride;
  constexpr int PER = HD / 32;
  extern __shared__ float smem[];
  float* sk = smem;
  float* sv = sk + kChunk * kStride;
  float* so = sv + kChunk * HD;
  float* sm = so + kMaxRows * HD;
  float* sl = sm + kMaxRows;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x, h = blockIdx.y;
  const int b = blockIdx.z / p.row_tiles, rt = blockIdx.z - b * p.row_tiles;
  const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0, L = p.seq_len[b];
  if (nq < 0 || nq > p.max_q || L < nq || q0 < 0 || q0 > p.token_cap - nq) {
    if (threadIdx.x == 0 && s == 0 && h == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const int row0 = rt * kMaxRows;
  const int rows = min(kMaxRows, nq * p.group - row0);
  if (rows <= 0) return;
  const int r0 = p.cu_res[b], nres = max(0, p.cu_res[b + 1] - r0);
  const int c0 = static_cast<int>(static_cast<long long>(s) * nres / p.num_splits);
  const int c1 = static_cast<int>(static_cast<long long>(s + 1) * nres / p.num_splits);
  for (int x = threadIdx.x; x < rows * HD; x += kThreads) so[x] = 0.f;
  for (int x = threadIdx.x; x < rows; x += kThreads) sm[x] = -INFINITY, sl[x] = 0.f;
  for (int e = c0; e < c1; ++e) {
    const int cid = p.res_ids[r0 + e], slot = p.res_slots[r0 + e];
    if (cid < 0 || cid >= (1 << 25) || slot < 0 || slot >= p.num_slots) {
      if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
      continue;
    }
    const int base = cid * kChunk;
    __syncthreads();
    const size_t at = (static_cast<size_t>(slot) * p.hkv + h) * kPackedBytes<HD>;
    for (int x = threadIdx.x; x < 2 * kChunk * (HD / 2); x += kThreads) {
      const bool is_v = x >= kChunk * (HD / 2);
      const int y = is_v ? x - kChunk * (HD / 2) : x;
      const int row = y / (HD / 2), cb = y % (HD / 2);       // token, code byte of its row
      const uint8_t* rec = (is_v ? p.v_pool : p.k_pool) + at;
      float2 v = make_float2(0.f, 0.f);
      if (base + row < L) {
        const float sc = e4m3_value(rec[kChunk * (HD / 2) + row * (HD / 16) + cb / 8]);
        v = e2m1_pair(rec[((cb / 16) * kChunk + row) * 16 + cb % 16]);
        v.x *= sc;
        v.y *= sc;
      }
      float* dst = is_v ? sv + row * HD + 2 * cb : sk + row * kStride + 2 * cb;
      dst[0] = v.x;
      dst[1] = v.y;
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kWarps) {
      const int i = (row0 + r) / p.group, g = (row0 + r) % p.group;
      const int pos = L - nq + i;
      const uint16_t* qr = p.q + (static_cast<size_t>(q0 + i) * p.hq + static_cast<size_t>(h) * p.group + g) * HD;
      float s0 = 0.f, s1 = 0.f;
      for (int c = 0; c < HD; ++c) {
        const float qv = __uint_as_float(static_cast<uint32_t>(__ldg(qr + c)) << 16);
        s0 = fmaf(qv, sk[lane * kStride + c], s0);
        s1 = fmaf(qv, sk[(lane + 32) * kStride + c], s1);
      }
      s0 = base + lane <= pos ? s0 * p.scale_log2 : -INFINITY;
      s1 = base + lane + 32 <= pos ? s1 * p.scale_log2 : -INFINITY;
      float m = fmaxf(s0, s1);
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float m_old = sm[r], m_new = fmaxf(m_old, m);
      if (m_new == -INFINITY) continue;
      const float alpha = ex2_approx(m_old - m_new);
      const float p0 = ex2_approx(s0 - m_new), p1 = ex2_approx(s1 - m_new);
      float l = p0 + p1;
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      float acc[PER];
      for (int x = 0; x < PER; ++x) acc[x] = so[r * HD + lane + 32 * x] * alpha;
      for (int k = 0; k < kChunk; ++k) {
        const float pk = __shfl_sync(0xffffffffu, k < 32 ? p0 : p1, k & 31);
        for (int x = 0; x < PER; ++x) acc[x] = fmaf(pk, sv[k * HD + lane + 32 * x], acc[x]);
      }
      for (int x = 0; x < PER; ++x) so[r * HD + lane + 32 * x] = acc[x];
      __syncwarp();
      if (lane == 0) sm[r] = m_new, sl[r] = sl[r] * alpha + l;
      __syncwarp();
    }
  }
  __syncthreads();
  const size_t pidx = ((static_cast<size_t>(b) * p.row_tiles + rt) * p.hkv + h) * p.num_splits + s;
  for (int x = threadIdx.x; x < rows * HD; x += kThreads) p.part_o[pidx * kMaxRows * HD + x] = so[x] * p.v_scale;
  for (int x = threadIdx.x; x < rows; x += kThreads)
    reinterpret_cast<float2*>(p.part_ml)[pidx * kMaxRows + x] = make_float2(sm[x], sl[x]);
}

template <int HD>
cudaError_t launch_hd(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  static size_t done[64] = {};
  constexpr size_t kSmem = Shape<HD>::kSmemFloats * 4;
  const cudaError_t e = ensure_smem_limit(attend_packed_kernel<HD>, kSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.num_splits, p.hkv, num_seqs * p.row_tiles);
  return launch_pdl(attend_packed_kernel<HD>, grid, dim3(kThreads), kSmem, stream, p);
}

}  // namespace

cudaError_t launch_attend_packed(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_hd<128>(p, num_seqs, stream) : launch_hd<64>(p, num_seqs, stream);
}

}  // namespace vfy
