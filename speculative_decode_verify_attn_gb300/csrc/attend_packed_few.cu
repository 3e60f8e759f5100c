// Attention of at most 16 block rows (queries x q-heads of one KV head) over a pool of 4-bit chunks: plain decoding, short
// blocks. So few rows leave the tensor cores idle whatever feeds them, and what a tile costs is the way from its codes to
// an MMA's operands: here there is none but registers. A warp takes chunks of its own and meets no other before the end.
//
//     S^T [16 keys][8 rows] = K Q^T,    O^T [16 channels][8 rows] += V^T P^T        (m16n8k16, fp16 in, fp32 out)
//
// Which channels a k-step multiplies is free as long as K and Q agree, and which channel a row of O^T is, so the fragments
// are what a lane's wide loads give it (g = lane / 4, c = lane % 4):
//   K   key g of eight: lane c has channels c d/4 .. (c+1) d/4 - 1, whose codes are neighbours: a load of d/8 bytes gives the
//       lane's A operands of all d/16 k-steps
//   V   keys 2c, 2c+1, 2c+8, 2c+9 of sixteen: lane g has channels g d/8 .. ; two keys' codes are interleaved by nibbles, so
//       that one conversion gives a register of both keys
//   P   S^T's accumulators, rounded to fp16 and transposed in eights (movmatrix)
// Tensor-core operands are exact, queries scaled by a power of two and weights placed as in attend_packed.cu. A warp has
// references of its own; its lanes keep those, the sums and O of rows 2c and 2c + 1.
//
// Each warp keeps a ring of three (six) stages of 32 keys in shared memory, which its lanes fill by asynchronous copies of 16
// bytes: 16 warps an SM have up to 220 KB on their way.
//
// 16 q-heads over 4 KV heads of 128, one row: 8K tokens in 8.5 us, 64K in 17.1, 256K in 36.5 (151 MB: 22.6 at the copy rate).
// Between short and long contexts it streams 5.9 TB/s at 53% of the issue slots; look-up, first copies, the merge of the warps
// and of the splits are 10 us. With up to eight rows a thread takes 125 registers: 16 warps; with 16 rows twice, 8 warps.
#include <cuda_bf16.h>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr float kTop = 7.f, kLimit = 15.f;   // log2: where a row's maximum is placed, where its reference moves
constexpr float kNone = 3.4028235e38f;       // minus the reference of a row that has none: any finite score is above that

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int HD, int NT>     // NT: tiles of eight rows
struct Few {
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = NT == 1 ? 16 : 8;                // one CTA an SM, with the registers that its warps take
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = NT == 1 ? 3 : 6;
  // A stage holds 32 keys of K and of V: codes [d / 32][32 tokens][16 bytes], then scales [32][d / 16]. The words of 32
  // channels lie 528 bytes apart: V's loads then take every bank once.
  static constexpr int kWords = HD / 32, kWordStride = 32 * 16 + 16;
  static constexpr int kScaleBytes = 32 * (HD / 16);
  static constexpr int kSide = kWords * kWordStride + kScaleBytes;
  static constexpr int kStageBytes = 2 * kSide;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kMerge = kWarps * kRows * HD * 4;         // the warps' O at the end, over the ring
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
};

__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "l"(policy) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint16_t v;
  asm volatile("{\n\t.reg .b8 x;\n\tld.shared.u8 %0, [%1];\n\t}" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
// N 32-bit words
template <int N>
__device__ __forceinline__ void lds(uint32_t at, uint32_t (&v)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(at));
}

template <int HD, int NT>
__global__ void __launch_bounds__(Few<HD, NT>::kThreads, 1) attend_packed_few_kernel(const PackedAttnParams p) {
  constexpr int kRows = Few<HD, NT>::kRows;
  constexpr int kSteps = HD / 16;          // k-steps of S, tiles of 16 channels of O^T
  using F = Few<HD, NT>;
  constexpr int kWarps = F::kWarps, kThreads = F::kThreads;
  extern __shared__ __align__(128) float s_o[];   // the rings; at the end [warp][row][channel]
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ uint64_t s_never;
  __shared__ int s_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  if (threadIdx.x == 0) {
    mbar_init(&s_never, 1);
    s_abort = 0;
  }
  __syncthreads();
  pdl_launch_dependents();
  if (!p.stable_metadata) pdl_wait();
  const int s = blockIdx.x, h = blockIdx.y;
  const SequenceMeta meta = longest_first(p.cu_q, p.cu_res, p.seq_len, p.num_seqs, blockIdx.z, lane);
  const int b = meta.b, q0 = meta.c0, nq = meta.c1 - q0, L = meta.len, r0 = meta.r0, nres = max(0, meta.r1 - r0);
  if (p.stable_metadata) pdl_wait();
  if (nq < 0 || nq > p.max_q || L < nq || static_cast<unsigned>(q0) > static_cast<unsigned>(p.token_cap - nq)) {
    if (threadIdx.x == 0 && s == 0 && h == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const int rows = nq * p.group;           // at most kRows (the context's capacity)
  if (rows == 0) return;
  // (the timeout path's test: this kernel has no other wait that could run out)
  if (p.timeout_test_ns != 0 && !mbar_wait_limit(&s_never, 0, p.timeout_test_ns, &s_abort, p.err)) return;
  const unsigned ns = static_cast<unsigned>(p.num_splits);
  // halves of chunks: 32 keys
  const int u0 = static_cast<int>(static_cast<unsigned long long>(s) * (2u * nres) / ns);
  const int u1 = static_cast<int>(static_cast<unsigned long long>(s + 1) * (2u * nres) / ns);
  const int p0 = L - nq;

  // This warp's halves are u0 + warp, + kWarps, ...: keys 32 (u % 2) .. of list entry u / 2.
  const int halves = u0 + warp < u1 ? (u1 - u0 - warp + kWarps - 1) / kWarps : 0;
  const uint32_t ring = smem_u32(s_o) + warp * F::kStages * F::kStageBytes;
  const uint64_t pol = l2_policy_evict_first();
  int first_l = -1, slot_l = 0;            // lane l: of the warp's half 32 k + l: position of its first key (-1: none)
  int first_before = -1;                   // of the 32 before those
  auto look_up = [&](int i) {
    first_before = first_l;
    const int u = u0 + warp + kWarps * (i + lane);
    const int id = u < u1 ? __ldg(p.res_ids + r0 + u / 2) : -1;
    slot_l = u < u1 ? __ldg(p.res_slots + r0 + u / 2) : -1;
    const bool ok = id >= 0 && id < (1 << 25) && slot_l >= 0 && slot_l < p.num_slots;
    if (u < u1 && !ok) atomicOr(p.err, kErrDeviceInput);
    first_l = ok ? id * kChunk + (u & 1) * 32 : -1;
  };
  auto issue = [&](int i, int st) {
    if ((i & 31) == 0) look_up(i);
    const int first = __shfl_sync(0xffffffffu, first_l, i & 31), sl = __shfl_sync(0xffffffffu, slot_l, i & 31);
    if (first >= 0) {
      const size_t rec = (static_cast<size_t>(sl) * p.hkv + h) * kPackedBytes<HD>;
      const int key0 = first & 32;
      const uint8_t* k_from = p.k_pool + rec + (key0 + lane) * 16;
      const uint8_t* v_from = p.v_pool + rec + (key0 + lane) * 16;
      const uint32_t to = ring + st * F::kStageBytes + lane * 16;
#pragma unroll
      for (int w = 0; w < F::kWords; ++w) {
        copy16(to + w * F::kWordStride, k_from + w * kChunk * 16, pol);
        copy16(to + F::kSide + w * F::kWordStride, v_from + w * kChunk * 16, pol);
      }
      constexpr int kLanes = F::kScaleBytes / 16;          // scales: K's by the first lanes, V's by the next
      if (lane < 2 * kLanes) {
        const bool is_v = lane >= kLanes;
        const int part = (lane - (is_v ? kLanes : 0)) * 16;
        copy16(ring + st * F::kStageBytes + (is_v ? F::kSide : 0) + F::kWords * F::kWordStride + part,
               (is_v ? p.v_pool : p.k_pool) + rec + kChunk * (HD / 2) + key0 * (HD / 16) + part, pol);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (a group for every stage, also behind the last half: the waits count groups)
  for (int i = 0; i < F::kStages; ++i) {
    if (i < halves)
      issue(i, i);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // Q as the B operands of the k-steps: row 8 t + g, channels c d/4 + 4 k .. + 3
  uint32_t qf[NT][kSteps][2];
  float q_scale;
  {
    unsigned top = 0u;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + g;
      const unsigned qi = static_cast<unsigned>(r) / static_cast<unsigned>(p.group), hg = r - qi * p.group;
      const uint2* src = reinterpret_cast<const uint2*>(
          p.q + (static_cast<size_t>(q0 + qi) * p.hq + static_cast<size_t>(h) * p.group + hg) * HD + c * (HD / 4));
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const uint2 w = r < rows ? __ldg(src + k) : make_uint2(0u, 0u);
        qf[t][k][0] = w.x;
        qf[t][k][1] = w.y;
        top = max(top, max(max(w.x & 0x7fffu, w.x >> 16 & 0x7fffu), max(w.y & 0x7fffu, w.y >> 16 & 0x7fffu)));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const int qe = query_exponent(top);
    const PowerOfTwo down(-qe);
    q_scale = score_scale(p.scale_log2, p.scale_exp, qe);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[t][k][i] = pack_f16(down.times(__uint_as_float(qf[t][k][i] << 16)), down.times(__uint_as_float(qf[t][k][i] & 0xffff0000u)));
  }

  float o[NT][kSteps][4];
  float neg_ref[NT][2], l[NT][2];          // rows 8 t + 2 c + i
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int m = 0; m < kSteps; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][m][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      neg_ref[t][i] = 8 * t + 2 * c + i < rows ? kNone : 0.f;   // (rows past the block, Q = 0, keep weight 1)
      l[t][i] = 0.f;
    }
  }

  // A lane's places in a stage.
  const uint32_t k_at = ring + (HD == 128 ? c * F::kWordStride : (c >> 1) * F::kWordStride + (c & 1) * 8) + g * 16;
  const uint32_t ks_at = ring + F::kWords * F::kWordStride + g * (HD / 16) + (HD == 128 ? 2 * c : c);
  const uint32_t v_at = ring + F::kSide + (HD == 128 ? (g >> 1) * F::kWordStride + (g & 1) * 8
                                                     : (g >> 2) * F::kWordStride + (g & 3) * 4) + 2 * c * 16;
  const uint32_t vs_at = ring + F::kSide + F::kWords * F::kWordStride + 2 * c * (HD / 16) + (HD == 128 ? g : g >> 1);
  // The 32 keys of the stage at `at`, the first of them at position `first`.
  auto work = [&](uint32_t at, int first) {
    const bool whole = first + 31 <= p0;
    float sc[NT][2][4];                    // [16 keys][key g: rows 2c, 2c + 1; key g + 8]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[t][u][i] = 0.f;
    uint32_t s2[4][2];                     // [key g + 8 i][first and second half of the lane's channels]
    uint32_t kc[4][HD / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // lane c has channels c d/4 ..: with d = 128 one word of 32, with 64 half of one
      lds(k_at + at + i * 8 * 16, kc[i]);
      const uint32_t two = e4m3_pair_f16(HD == 128 ? lds16(ks_at + at + i * 8 * (HD / 16)) : lds8(ks_at + at + i * 8 * (HD / 16)));
      s2[i][0] = __byte_perm(two, two, 0x1010);
      s2[i][1] = HD == 128 ? __byte_perm(two, two, 0x3232) : s2[i][0];
    }
#pragma unroll
    for (int w = 0; w < HD / 32; ++w) {                    // eight channels: two k-steps
      uint32_t kf[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack_word(kc[i][w], s2[i][w / (HD / 64)], kf[i]);
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u) {                      // (two sums side by side: an MMA's latency is 24 cycles)
          const uint32_t a[4] = {kf[2 * u][2 * y], kf[2 * u + 1][2 * y], kf[2 * u][2 * y + 1], kf[2 * u + 1][2 * y + 1]};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(sc[t][u], a, qf[t][2 * w + y][0], qf[t][2 * w + y][1]);
        }
    }
    // exponents s scale - ref; masked keys -inf
    if (!whole) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = first + 16 * u + g + 8 * (i >> 1), r = 8 * t + 2 * c + (i & 1);
            if (pos >= L || pos > p0 + static_cast<int>(static_cast<unsigned>(r) / static_cast<unsigned>(p.group)))
              sc[t][u][i] = -INFINITY;
          }
    }
    auto over = [&](float limit) {
      bool any = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m = fmaxf(fmaxf(sc[t][0][i], sc[t][0][i + 2]), fmaxf(sc[t][1][i], sc[t][1][i + 2]));
          any = any || fmaf(m, q_scale, neg_ref[t][i]) > limit;
        }
      return any;
    };
    if (__any_sync(0xffffffffu, over(kLimit))) {
      // a weight would pass 2^15, or a row has no reference yet
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(fmaxf(sc[t][0][i], sc[t][0][i + 2]), fmaxf(sc[t][1][i], sc[t][1][i + 2]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16)) * q_scale;
          if (m + neg_ref[t][i] > kLimit) {
            const float a = neg_ref[t][i] == kNone ? 0.f : ex2_approx(kTop - m - neg_ref[t][i]);
            neg_ref[t][i] = kTop - m;
            if (!(fabsf(m) < kMostScore)) atomicOr(p.err, kErrDeviceInput);
            l[t][i] *= a;
#pragma unroll
            for (int y = 0; y < kSteps; ++y) {
              o[t][y][i] *= a;
              o[t][y][i + 2] *= a;
            }
          }
        }
    }
    uint32_t pf[NT][2][2];                 // P as B operands: [16 keys][keys 0-7, 8-15]
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float2 sum = make_float2(0.f, 0.f);  // (added up first: one addition to a long sum for 32 keys)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = ex2_approx(fmaf(sc[t][u][2 * i], q_scale, neg_ref[t][0]));
          const float bb = ex2_approx(fmaf(sc[t][u][2 * i + 1], q_scale, neg_ref[t][1]));
          sum.x += a;
          sum.y += bb;
          pf[t][u][i] = transpose8(pack_f16(a, bb));
        }
      l[t][0] += sum.x;
      l[t][1] += sum.y;
    }
    // O^T: row g of a tile is channel g d/8 + 2 m, row g + 8 the next channel
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t codes[4][HD / 64], scale[4];  // keys 2c, 2c + 1, 2c + 8, 2c + 9; lane g has channels g d/8 ..
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 16 * u + (i & 1) + 4 * (i & 2);    // + 2c
        lds(v_at + at + tok * 16, codes[i]);
        scale[i] = lds8(vs_at + at + tok * (HD / 16));
      }
      uint32_t pa = scale[0] | scale[1] << 8, pb = scale[2] | scale[3] << 8;
      if (!whole) {
        // Keys that no row attends may hold anything: P is 0 there, but 0 * NaN is NaN.
        const int left = L - first - 16 * u - 2 * c;
        pa &= (left > 0 ? 0xffu : 0u) | (left > 1 ? 0xff00u : 0u);
        pb &= (left > 8 ? 0xffu : 0u) | (left > 9 ? 0xff00u : 0u);
      }
      const uint32_t sa = e4m3_pair_f16(pa), sb = e4m3_pair_f16(pb);
#pragma unroll
      for (int w = 0; w < HD / 64; ++w) {                  // eight channels: four tiles
        const uint32_t k0 = codes[0][w], k1 = codes[1][w], k2 = codes[2][w], k3 = codes[3][w];
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        uint32_t ea[4], oa[4], eb[4], ob[4];               // even and odd channels of both key pairs
        unpack_word((k0 & kLow) | ((k1 & kLow) << 4), sa, ea);
        unpack_word(((k0 >> 4) & kLow) | (k1 & ~kLow), sa, oa);
        unpack_word((k2 & kLow) | ((k3 & kLow) << 4), sb, eb);
        unpack_word(((k2 >> 4) & kLow) | (k3 & ~kLow), sb, ob);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t a[4] = {ea[y], oa[y], eb[y], ob[y]};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(o[t][4 * w + y], a, pf[t][u][0], pf[t][u][1]);
        }
      }
    }
  };

  int st = 0;
  for (int i = 0; i < halves; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(F::kStages - 1) : "memory");
    __syncwarp();
    // (the look-ups are up to kStages - 1 halves ahead: in the next 32 already?)
    const bool ahead = (min(i + F::kStages, halves) - 1) >> 5 != i >> 5;
    const int first = __shfl_sync(0xffffffffu, ahead ? first_before : first_l, i & 31);
    if (first >= 0) work(st * F::kStageBytes, first);
    __syncwarp();
    if (i + F::kStages < halves)
      issue(i + F::kStages, st);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
    if (++st == F::kStages) st = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();                         // the rings give way to the warps' O

  // ---- the warps' rows merged: O = sum_w 2^(ref_w - M) O_w, l alike ----
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[t][i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int r = 8 * t + 2 * c + i;
      if (g == 0) {
        s_m[warp][r] = sum > 0.f ? -neg_ref[t][i] : -INFINITY;
        s_l[warp][r] = sum;
      }
#pragma unroll
      for (int m = 0; m < kSteps; m += 2)                  // channels g d/8 + 2 m .. + 3
        *reinterpret_cast<float4*>(s_o + (warp * kRows + r) * HD + g * (HD / 8) + 2 * m) =
            make_float4(o[t][m][i], o[t][m][i + 2], o[t][m + 1][i], o[t][m + 1][i + 2]);
    }
  __syncthreads();
  const bool direct = p.num_splits == 1;
  for (int x = threadIdx.x; x < rows * (HD / 4); x += kThreads) {
    const int r = x / (HD / 4), ch = x % (HD / 4) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][r]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (s_l[w][r] > 0.f) {
        const float wt = ex2_approx(s_m[w][r] - m);
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * kRows + r) * HD + ch);
        sum += wt * s_l[w][r];
        acc.x = fmaf(wt, v.x, acc.x);
        acc.y = fmaf(wt, v.y, acc.y);
        acc.z = fmaf(wt, v.z, acc.z);
        acc.w = fmaf(wt, v.w, acc.w);
      }
    }
    if (direct) {
      const unsigned qi = static_cast<unsigned>(r) / static_cast<unsigned>(p.group), hg = r - qi * p.group;
      const size_t row = static_cast<size_t>(q0 + qi) * p.hq + static_cast<size_t>(h) * p.group + hg;
      const float inv = sum > 0.f ? 1.f / sum : 0.f, g = p.v_scale;      // (g / sum could be a denormal)
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv * g, acc.y * inv * g),
                           hi = __floats2bfloat162_rn(acc.z * inv * g, acc.w * inv * g);
      *reinterpret_cast<uint2*>(p.out + row * HD + ch) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      if (ch == 0 && p.lse != nullptr)
        p.lse[row] = sum > 0.f ? (m + __log2f(sum)) * 0.6931471805599453f : -INFINITY;
    } else {
      const size_t pidx = (static_cast<size_t>(b) * p.hkv + h) * p.num_splits + s;
      const int e = partial_exponent(sum, p.v_scale);
      const float down = __int_as_float((127 - e) << 23), scale = down * p.v_scale;
      *reinterpret_cast<float4*>(p.part_o + (pidx * kMaxRows + r) * HD + ch) =
          make_float4(acc.x * scale, acc.y * scale, acc.z * scale, acc.w * scale);
      if (ch == 0) reinterpret_cast<float2*>(p.part_ml)[pidx * kMaxRows + r] = make_float2(m + static_cast<float>(e), sum * down);
    }
  }
}

template <int HD, int NT>
cudaError_t launch_t(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  static size_t done[64] = {};
  auto kern = attend_packed_few_kernel<HD, NT>;
  const cudaError_t e = ensure_smem_limit(kern, Few<HD, NT>::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.num_splits, p.hkv, num_seqs), dim3(Few<HD, NT>::kThreads), Few<HD, NT>::kSmem, stream, p);
}

}  // namespace

cudaError_t launch_attend_packed_few(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  if (p.max_q * p.group <= 8) return p.head_dim == 128 ? launch_t<128, 1>(p, num_seqs, stream) : launch_t<64, 1>(p, num_seqs, stream);
  return p.head_dim == 128 ? launch_t<128, 2>(p, num_seqs, stream) : launch_t<64, 2>(p, num_seqs, stream);
}

}  // namespace vfy
