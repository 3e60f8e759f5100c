// Attention of a block over a pool of 4-bit chunks, on the tensor cores with the operands exchanged: a tile's 128 keys are
// the M = 128 side of both products and the block's rows (queries x q-heads of one KV head, at most 80) the N side,
//     S^T [128 keys][rows] = K Q^T,    O^T [d][rows] += V^T P^T,
// so that the work follows the rows a block has: one token of G = 4 is N = 16, a block of 17 is N = 80. With the rows as M (as
// in the bf16 layers) a 4-bit tile would be bound by the 128 rows' tensor time.
//
// A value is g s e; s e has 6 significant bits, so the operands in fp16 are exact. Queries are bf16: the tile's are scaled by
// one power of two that puts the largest at 2^14, and fp16 holds all 8 bits of what is above 2^-28 of it. Weights P are
// fp16 too (half a step, 2^-11): a row's reference is put 7 below its maximum (log2), weights grow to 2^15 before the
// reference moves, and what fp16 drops (below 2^-25) is 2^-32 of the largest weight.
//
// One CTA per (split, KV head, sequence and row tile), a contiguous run of tiles of two chunks. Roles:
//   warps 0-3, 4-7   softmax of even / odd tiles: a lane is a key, its 32-bit columns are the rows. Two groups with a
//                    reference, row sums and O of their own, merged at the end; a group has two tiles' time for one.
//   warps 8-11, 12-15   K of even / odd tiles: a lane reads its key's codes and scales, writes fp16 into tensor memory
//                    (the A operand of S)
//   warps 16-19, 20-23  V of even / odd tiles: fp16 into shared memory, channels contiguous (the A operand of O^T, M-major)
//   warp 24          bulk copies of the records (contiguous: no tensor map), and the tiles' geometry
//   warp 25, 26      the MMA issuers of S and of O (25 also holds tensor memory)
#include <cuda_bf16.h>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kGroups = 7;                // warpgroups: softmax 0 and 1, K twice, V twice, the rest
constexpr int kThreads = kGroups * 128;
constexpr int kRegsLaunch = 72, kRegsSoftmax = 152, kRegsUnpack = 40, kRegsRest = 40;
static_assert(2 * kRegsSoftmax + 4 * kRegsUnpack + kRegsRest <= kGroups * kRegsLaunch, "registers the CTA was launched with");
constexpr int kKWarp = 8, kVWarp = 16, kProducerWarp = 24, kMmaWarp = 25;
constexpr int kKeys = 2 * kChunk;         // keys of a tile
constexpr int kFewN = 16, kMaxN = 80;     // rows of a tile (two kernels): the softmax threads hold a partial sum of each
constexpr int kBatch = 16;                // tiles whose chunks a warp's lanes hold; their geometry lies in two such batches
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColK = 0;             // two K tiles of up to 64 columns (two fp16 channels each)
constexpr uint32_t kColS = 128;           // S^T of the two groups, 96 columns apart
constexpr uint32_t kColO = 320;           // O^T of the two groups
constexpr float kTop = 7.f;               // a row's maximum when its reference is set (log2)
constexpr float kLimit = 15.f;            // the reference moves when a weight would pass 2^15
constexpr float kClamp = 24.f;            // weights past the limit are held at 2^24 until they are worked out again
constexpr float kNone = 1e30f;            // minus the reference of a row that has none: every score passes the limit

template <int HD, int NT>
struct Cfg {
  static constexpr int kStages = NT > kFewN ? 4 : 6;
  static constexpr int kRecord = kPackedBytes<HD>;
  static constexpr int kStageBytes = 4 * kRecord;                // K and V of two chunks
  static constexpr int kBoxBytes = kKeys * 128;                  // 64 columns of 128 keys
  static constexpr int kVBytes = 2 * kBoxBytes;                  // M = 128: d = 64 leaves the second box zero
  static constexpr int kPBytes = (NT + 63) / 64 * kBoxBytes;
  static constexpr int kQBoxBytes = NT * 128;
  static constexpr int kQBytes = (HD / 64) * kQBoxBytes;
  static constexpr int kVOffset = 0;
  static constexpr int kPOffset = 2 * kVBytes;
  static constexpr int kQOffset = kPOffset + 2 * kPBytes;
  static constexpr int kStageOffset = kQOffset + kQBytes;
  static constexpr int kBarOffset = kStageOffset + kStages * kStageBytes;
  static constexpr int kBarBytes = 5120;
  static constexpr int kSmemBytes = kBarOffset + kBarBytes + 1024;
  static_assert(kRecord % 16 == 0 && kStageBytes % 128 == 0, "bulk copies");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Shared {
  uint64_t full[6], empty[6];
  uint64_t geo_full[2];
  uint64_t k_ready[2], v_ready[2];
  uint64_t s_done[2];                     // S of a tile: its S^T is there, its K is free
  uint64_t p_ready[2];                    // a tile's P is written, its S^T read
  uint64_t pv_done[2];                    // O^T holds the tile, its P and V are free
  uint64_t q_ready, drain[2], never;
  uint32_t tmem_base;
  int abort;
  unsigned q_top;                         // largest |q| of the tile, as bf16 bits
  int base[2 * kBatch][2];                // position of a chunk's first token, -1: no chunk
  int plain[2 * kBatch];                  // every row attends every key of the tile
  alignas(16) float neg_ref[2][kMaxN];    // [group] minus the rows' reference, log2 units
  alignas(16) float old_ref[2][kMaxN];    // minus the reference before it moved
  alignas(16) float alpha[2][kMaxN];
  alignas(16) float part[2][4][kMaxN];    // [group][warp]: maxima, at the end sums
};
static_assert(sizeof(Shared) <= Cfg<128, kMaxN>::kBarBytes, "barrier block");

struct Work {
  int b, h, s;
  int q0, nq, L;
  int row0, rows;          // block rows of this CTA
  int r0, nres;            // resident list
  int tb, nt;              // tiles
  bool bad;
};

__device__ __forceinline__ Work make_work(const PackedAttnParams& p) {
  Work w;
  w.s = blockIdx.x;
  w.h = blockIdx.y;
  w.b = static_cast<int>(blockIdx.z / static_cast<unsigned>(p.n_tiles));
  const int rt = static_cast<int>(blockIdx.z) - w.b * p.n_tiles;
  const int c0 = p.cu_q[w.b], c1 = p.cu_q[w.b + 1], cr0 = p.cu_res[w.b], cr1 = p.cu_res[w.b + 1];
  w.L = p.seq_len[w.b];
  w.q0 = c0;
  w.nq = c1 - c0;
  w.row0 = rt * p.tile_rows;
  w.r0 = cr0;
  w.nres = max(0, cr1 - cr0);
  w.rows = w.tb = w.nt = 0;
  w.bad = w.nq < 0 || w.nq > p.max_q || w.L < w.nq || static_cast<unsigned>(c0) > static_cast<unsigned>(p.token_cap - w.nq);
  if (w.bad) return w;
  w.rows = min(p.tile_rows, max(0, w.nq * p.group - w.row0));
  if (w.rows == 0) return w;
  const unsigned tiles = (static_cast<unsigned>(w.nres) + 1) / 2, ns = static_cast<unsigned>(p.num_splits);
  // (splits <= 64 and tiles < 2^26: 32-bit products)
  w.tb = static_cast<int>(static_cast<unsigned>(w.s) * tiles / ns);
  w.nt = static_cast<int>(static_cast<unsigned>(w.s + 1) * tiles / ns) - w.tb;
  return w;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes (a 32-bit word) times a scale (in both halves): eight fp16 values, two a register.
__device__ __forceinline__ void unpack_word(uint32_t codes, uint32_t scale2, uint32_t* out) {
  uint32_t a, b, c, d;
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x0;\n\tcvt.rn.f16x2.e2m1x2 %1, x1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, x2;\n\tcvt.rn.f16x2.e2m1x2 %3, x3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(codes));
  out[0] = mul_f16x2(a, scale2);
  out[1] = mul_f16x2(b, scale2);
  out[2] = mul_f16x2(c, scale2);
  out[3] = mul_f16x2(d, scale2);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 pair(const uint32_t* r, int i) {
  return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}
__device__ __forceinline__ uint4 lds_u4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
// (no memory clobber: what is written is read by MMAs alone, behind a proxy fence, and loads may move ahead of it)
__device__ __forceinline__ void sts_u4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
}

// One value per row of eight from 32 lanes: lane r (r < 8, and every lane alike modulo 8) gets row r's sum.
__device__ __forceinline__ float sum_rows8(const float2* l2, int lane) {
  const float l[8] = {l2[0].x, l2[0].y, l2[1].x, l2[1].y, l2[2].x, l2[2].y, l2[3].x, l2[3].y};
  float a[4], b[2], c;
  const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, h4 ? l[i] : l[i + 4], 4);
    a[i] = (h4 ? l[i + 4] : l[i]) + other;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, h2 ? a[i] : a[i + 2], 2);
    b[i] = (h2 ? a[i + 2] : a[i]) + other;
  }
  const float other = __shfl_xor_sync(0xffffffffu, h1 ? b[0] : b[1], 1);
  c = (h1 ? b[1] : b[0]) + other;
  c += __shfl_xor_sync(0xffffffffu, c, 8);
  c += __shfl_xor_sync(0xffffffffu, c, 16);
  return c;
}

template <int HD, int NT>
__global__ void __launch_bounds__(kThreads, 1) attend_packed_kernel(const PackedAttnParams p) {
  using C = Cfg<HD, NT>;
  constexpr int kStages = C::kStages;
  constexpr bool kTrade = NT > kFewN;     // the softmax groups take up registers that the others give up
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));
  uint8_t* sV = smem + C::kVOffset;
  uint8_t* sP = smem + C::kPOffset;
  uint8_t* sQ = smem + C::kQOffset;
  uint8_t* sStage = smem + C::kStageOffset;
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kBarOffset);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == kProducerWarp * 32) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh->full[i], 2);
      mbar_init(&sh->empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->geo_full[i], 1);
      mbar_init(&sh->k_ready[i], 4);
      mbar_init(&sh->v_ready[i], 4);
      mbar_init(&sh->s_done[i], 1);
      mbar_init(&sh->p_ready[i], 4);
      mbar_init(&sh->pv_done[i], 1);
    }
    mbar_init(&sh->q_ready, 8);
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    mbar_init(&sh->never, 1);
    sh->abort = 0;
    sh->q_top = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (HD == 64) {
    // M = 128 with 64 channels: the second box of V stays zero
    for (int x = threadIdx.x; x < 2 * C::kBoxBytes / 16; x += kThreads) {
      const int buf = x / (C::kBoxBytes / 16), at = x % (C::kBoxBytes / 16);
      *reinterpret_cast<uint4*>(sV + buf * C::kVBytes + C::kBoxBytes + at * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sh->tmem_base;
  volatile int* abort = &sh->abort;

  pdl_launch_dependents();
  if (!p.stable_metadata) pdl_wait();
  const Work w = make_work(p);
  if (p.stable_metadata) pdl_wait();
  if (w.bad && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.err, kErrDeviceInput);

  if (warp >= kProducerWarp) {
    if constexpr (kTrade) regs_dec<kRegsRest>();
    if (warp == kProducerWarp) {
      // ------------------------------ records and geometry --------------------------------
      // A lane holds one chunk of sixteen tiles; a tile's two lanes issue its copies, with no word between them.
      const uint64_t pol = l2_policy_evict_first();
      int issued = 0, st = 0, empty_phase = 1;
      bool ok = false;
      const uint8_t *from_k = nullptr, *from_v = nullptr;
      for (int j = 0; j < w.nt; ++j) {
        if (j % kBatch == 0) {
          const int e = (w.tb + j) * 2 + lane;
          const bool in = e < w.nres && e < (w.tb + w.nt) * 2;
          const int cid = in ? __ldg(p.res_ids + w.r0 + e) : -1;
          const int slot = in ? __ldg(p.res_slots + w.r0 + e) : -1;
          ok = cid >= 0 && cid < (1 << 25) && slot >= 0 && slot < p.num_slots;
          if (in && !ok) atomicOr(p.err, kErrDeviceInput);
          const size_t from = (static_cast<size_t>(ok ? slot : 0) * p.hkv + w.h) * C::kRecord;
          from_k = p.k_pool + from;
          from_v = p.v_pool + from;
          // The geometry of the sixteen tiles (the consumers of the sixteen that held these entries have long passed
          // them: at most kStages + 4 tiles lie between this warp and the softmax).
          const bool plain = ok && cid * kChunk + kChunk - 1 <= w.L - w.nq;
          const bool both = __shfl_xor_sync(0xffffffffu, plain ? 1 : 0, 1) != 0 && plain;
          const int at = (j / kBatch & 1) * kBatch + lane / 2;
          sh->base[at][lane & 1] = ok ? cid * kChunk : -1;
          if ((lane & 1) == 0) sh->plain[at] = both ? 1 : 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->geo_full[j / kBatch & 1]);
        }
        if (j >= kStages && !__all_sync(0xffffffffu, mbar_wait_tested(&sh->empty[st], empty_phase, abort, p.err))) break;
        if (lane / 2 == j % kBatch) {
          mbar_arrive_expect_tx(&sh->full[st], ok ? 2 * C::kRecord : 0);
          if (ok) {
            uint8_t* to = sStage + st * C::kStageBytes + (lane & 1) * C::kRecord;
            bulk_load(to, from_k, C::kRecord, &sh->full[st], pol);
            bulk_load(to + 2 * C::kRecord, from_v, C::kRecord, &sh->full[st], pol);
          }
        }
        __syncwarp();
        issued = j + 1;
        if (++st == kStages) st = 0, empty_phase ^= 1;
      }
      // Every copy lands before the CTA can exit.
      if (lane == 0)
        for (int j = max(0, issued - kStages); j < issued; ++j)
          mbar_drain(&sh->full[j % kStages], (j / kStages) & 1, p.err);
      __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ------------------------------ MMA issuers -----------------------------------------
      // One warp for S, one for O: issuing a tile's eight MMAs of one kind with its waits takes 500 to 600 cycles, more
      // than the tensor core does (N = 16: 160 and 320). The whole warp runs the loop (see elect_one). Tensor memory is
      // allocated whole: it starts at column 0.
      const bool is_o = warp != kMmaWarp;
      const int nt = uniform(w.nt), n = (uniform(w.rows) + 15) & ~15;
      if (nt > 0) {
        if (p.timeout_test_ns != 0) mbar_wait_limit(&sh->never, 0, p.timeout_test_ns, abort, p.err);
        bool ok = __all_sync(0xffffffffu, !*abort && mbar_wait(&sh->q_ready, 0, abort, p.err));
        tc_fence_after();
        auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mbar_wait_tested(bar, parity, abort, p.err)); };
        if (!is_o) {
          const uint32_t idesc = idesc_f16_f32(128, n, 0, 0);
          const uint64_t qdesc = sw128_desc(sbase + C::kQOffset, 16, 1024);
          for (int j = 0; j < nt; ++j) {
            // S^T of tile j over its group's buffer: free once the group's P of tile j - 2 is written.
            const int g = j & 1, ph = (j >> 1) & 1;
            if (j > 1) ok = ok && wait(&sh->p_ready[g], ph ^ 1);
            ok = ok && wait(&sh->k_ready[g], ph);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                mma_ts(kColS + g * 96, kColK + g * 64 + kk * 8,
                       qdesc + static_cast<uint64_t>(((kk >> 2) * C::kQBoxBytes + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
              mma_commit(&sh->s_done[g]);
            }
            __syncwarp();
          }
        } else {
          const uint32_t idesc = idesc_f16_f32(128, n, 1, 1);
          const uint64_t vdesc = sw128_desc(sbase + C::kVOffset, C::kBoxBytes, 1024);
          const uint64_t pdesc = sw128_desc(sbase + C::kPOffset, C::kBoxBytes, 1024);
          for (int j = 0; j < nt; ++j) {
            const int g = j & 1, ph = (j >> 1) & 1;
            ok = ok && wait(&sh->v_ready[g], ph) && wait(&sh->p_ready[g], ph);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ss(kColO + g * 96, vdesc + static_cast<uint64_t>((g * C::kVBytes + kk * 2048) >> 4),
                       pdesc + static_cast<uint64_t>((g * C::kPBytes + kk * 2048) >> 4), idesc, (j > 1 || kk > 0) ? 1u : 0u);
              mma_commit(&sh->pv_done[g]);
            }
            __syncwarp();
          }
        }
        // Every MMA issued above completes before tensor memory is freed.
        if (elect_one()) mma_commit(&sh->drain[is_o]);
        __syncwarp();
        mbar_drain(&sh->drain[is_o], 0, p.err);
      }
      __syncwarp();
    }
  } else if (warp >= kKWarp) {
    // ------------------------------ K and V to fp16 -----------------------------------------
    if constexpr (kTrade) regs_dec<kRegsUnpack>();
    const bool is_v = warp >= kVWarp;
    const int g = (warp >> 2) & 1;                       // even or odd tiles; their buffer
    const int key = (warp & 3) * 32 + lane;              // of the tile; a TMEM lane
    const int c = key / kChunk, tok = key % kChunk;
    uint64_t* done = is_v ? &sh->pv_done[g] : &sh->s_done[g];
    uint64_t* ready = is_v ? &sh->v_ready[g] : &sh->k_ready[g];
    const uint32_t rec = sbase + C::kStageOffset + ((is_v ? 2 : 0) + c) * C::kRecord;
    const uint32_t scales_at = rec + kChunk * (HD / 2) + tok * (HD / 16);
    const uint32_t codes_at = rec + tok * 16;
    const uint32_t kto = (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColK + g * 64;
    const uint32_t vto = sbase + C::kVOffset + g * C::kVBytes + key * 128;
    int st = g % kStages, stage_phase = 0;               // (kStages is even)
    for (int j = g; j < w.nt; j += 2) {
      const int u = j >> 1;
      bool ok = mbar_wait_tested(&sh->full[st], stage_phase, abort, p.err);
      if (is_v && j % kBatch == g && ok) ok = mbar_wait_tested(&sh->geo_full[j / kBatch & 1], j / kBatch >> 1 & 1, abort, p.err);
      if (ok && u > 0) ok = mbar_wait_tested(done, (u - 1) & 1, abort, p.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t at = st * C::kStageBytes;
      // Keys that no row attends may hold anything: P is 0 there, but 0 * NaN is NaN.
      bool keep = true;
      if (is_v && !sh->plain[j % (2 * kBatch)]) {
        const int base = sh->base[j % (2 * kBatch)][c];
        keep = base >= 0 && base + tok < w.L;
      }
      if (!is_v) tc_fence_after();
#pragma unroll
      for (int y = 0; y < HD / 64; ++y) {                // 64 channels: two words of codes, four scales
        // (both words loaded before the first store: the compiler keeps loads behind stores)
        const uint4 codes[2] = {lds_u4(codes_at + at + 2 * y * kChunk * 16), lds_u4(codes_at + at + (2 * y + 1) * kChunk * 16)};
        const uint32_t scales = keep ? lds_u32(scales_at + at + 4 * y) : 0u;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t two = e4m3_pair_f16(x == 0 ? scales & 0xffffu : scales >> 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {                  // 16 channels: one scale
            const uint32_t sc = __byte_perm(two, two, i == 0 ? 0x1010 : 0x3232);
            uint32_t out[8];
            unpack_word(i == 0 ? codes[x].x : codes[x].z, sc, out);
            unpack_word(i == 0 ? codes[x].y : codes[x].w, sc, out + 4);
            if (!is_v) {
              tmem_st8_async(kto + (4 * y + 2 * x + i) * 8, out);
            } else {
#pragma unroll
              for (int z = 0; z < 2; ++z)                // 16-byte words of the 128-byte row
                sts_u4(vto + y * C::kBoxBytes + (((x * 4 + 2 * i + z) ^ (key & 7)) << 4),
                       make_uint4(out[4 * z], out[4 * z + 1], out[4 * z + 2], out[4 * z + 3]));
            }
          }
        }
      }
      if (is_v) {
        fence_proxy_async_smem();
      } else {
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh->empty[st]);
        mbar_arrive(ready);
      }
      st += 2;
      if (st >= kStages) st -= kStages, stage_phase ^= 1;
    }
  } else {
    // ------------------------------ softmax ---------------------------------------------------
    if constexpr (kTrade) regs_inc<kRegsSoftmax>();
    const int grp = warp >> 2, wq = warp & 3, tg = threadIdx.x & 127;
    const int key = tg;
    const int bar = 2 + grp;                             // named barrier of the group; 1: both groups
    // Q: words of 8 channels, all of a thread's in registers while the tile's largest value is found
    constexpr int kWords = (NT * HD / 8 + 255) / 256;
    float q_scale;                                       // of a score: softmax scale, g of K, the queries' power of two
    {
      uint4 qv[kWords];
      unsigned top = 0u;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int x = threadIdx.x + i * 256;
        const int r = x / (HD / 8), cw = x % (HD / 8);
        qv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < w.rows) {
          const unsigned rg = static_cast<unsigned>(w.row0 + r), ug = static_cast<unsigned>(p.group);
          const unsigned qi = rg / ug, hg = rg - qi * ug;
          qv[i] = __ldg(reinterpret_cast<const uint4*>(
                            p.q + (static_cast<size_t>(w.q0 + qi) * p.hq + static_cast<size_t>(w.h) * p.group + hg) * HD) + cw);
        }
        const uint32_t ws[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(ws[e] & 0x7fffu, (ws[e] >> 16) & 0x7fffu));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) atomicMax(&sh->q_top, top);
      named_sync(1, 256);
      const int qe = max(static_cast<int>(sh->q_top >> 7) - 127 - 14, -100);
      const float down = __int_as_float((127 - qe) << 23);
      q_scale = p.scale_log2 * __int_as_float((127 + qe) << 23);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int x = threadIdx.x + i * 256;
        const int r = x / (HD / 8), cw = x % (HD / 8);
        const uint32_t ws[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_f16(__uint_as_float(ws[e] << 16) * down, __uint_as_float(ws[e] & 0xffff0000u) * down);
        if (r < NT)
          *reinterpret_cast<uint4*>(sQ + (cw >> 3) * C::kQBoxBytes + r * 128 + (((cw & 7) ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_ready);
    }
    // (rows past the block, Q = 0, keep weight 1: never read)
    if (tg < NT) sh->neg_ref[grp][tg] = tg < w.rows ? kNone : 0.f;
    named_sync(bar, 128);

    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_at = lane_base + kColS + grp * 96, o_at = lane_base + kColO + grp * 96;
    const uint32_t prow = sbase + C::kPOffset + grp * C::kPBytes + key * 128;
    const int p0 = w.L - w.nq;
    const float2 sc2 = make_float2(q_scale, q_scale);
    float2 l[NT / 2];
#pragma unroll
    for (int r = 0; r < NT / 2; ++r) l[r] = make_float2(0.f, 0.f);
    bool dead = false;                                   // a wait of this warp gave up
    int u = 0;                                           // tiles of this group so far
    for (int j = grp; j < w.nt; j += 2, ++u) {
      if (j % kBatch == grp && !mbar_wait_tested(&sh->geo_full[j / kBatch & 1], j / kBatch >> 1 & 1, abort, p.err)) dead = true;
      const int geo = j % (2 * kBatch);
      const bool whole = sh->plain[geo] != 0;
      int n_min = 0;
      if (!whole) {
        // Rows from n_min on attend this lane's key: row n is of block query (row0 + n) / G, at position p0 + that.
        const int base = sh->base[geo][key / kChunk], pos = base + key % kChunk;
        if (base < 0 || pos >= w.L)
          n_min = NT;
        else if (pos > p0)
          n_min = min(static_cast<long long>(NT), max(0ll, static_cast<long long>(pos - p0) * p.group - w.row0));
      }
      if (u > 0 && !mbar_wait_tested(&sh->pv_done[grp], (u - 1) & 1, abort, p.err)) dead = true;   // P is free, O complete
      if (!mbar_wait_tested(&sh->s_done[grp], u & 1, abort, p.err)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      tc_fence_after();
      // Weights P = 2^(s scale - ref), their sums, and the largest exponent: sixteen rows at a time, the next sixteen's
      // scores on their way. `undo` takes the weights against the old references off the sums first.
      auto weigh = [&](bool undo) -> float {
        float top[2] = {-INFINITY, -INFINITY};
        uint32_t buf[2][16];
        tmem_ld_async(s_at, buf[0]);
#pragma unroll
        for (int cb = 0; cb < NT / 16; ++cb) {
          if (cb * 16 < w.rows) {
            uint32_t(&s)[16] = buf[cb & 1];
            tmem_wait_ld(s);
            if (cb + 1 < NT / 16 && (cb + 1) * 16 < w.rows) tmem_ld_async(s_at + (cb + 1) * 16, buf[(cb + 1) & 1]);
            if (!whole) {                                // 2^-inf = 0
#pragma unroll
              for (int e = 0; e < 16; ++e) s[e] = cb * 16 + e >= n_min ? s[e] : 0xff800000u;
            }
            if (undo) {
              const float2* old = reinterpret_cast<const float2*>(&sh->old_ref[grp][cb * 16]);
              const float2* al = reinterpret_cast<const float2*>(&sh->alpha[grp][cb * 16]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 x = fma_f32x2(pair(s, 2 * e), sc2, old[e]);
                float2& sum = l[cb * 8 + e];
                sum.x = (sum.x - ex2_approx(fminf(x.x, kClamp))) * al[e].x;
                sum.y = (sum.y - ex2_approx(fminf(x.y, kClamp))) * al[e].y;
              }
            }
            const float4* nr = reinterpret_cast<const float4*>(&sh->neg_ref[grp][cb * 16]);
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 f = nr[e];
              float2 a = fma_f32x2(pair(s, 4 * e), sc2, make_float2(f.x, f.y));
              float2 b = fma_f32x2(pair(s, 4 * e + 2), sc2, make_float2(f.z, f.w));
              top[0] = fmaxf(fmaxf(top[0], a.x), a.y);
              top[1] = fmaxf(fmaxf(top[1], b.x), b.y);
              a.x = ex2_approx(fminf(a.x, kClamp));
              a.y = ex2_approx(fminf(a.y, kClamp));
              b.x = ex2_approx(fminf(b.x, kClamp));
              b.y = ex2_approx(fminf(b.y, kClamp));
              l[cb * 8 + 2 * e] = add_f32x2(l[cb * 8 + 2 * e], a);
              l[cb * 8 + 2 * e + 1] = add_f32x2(l[cb * 8 + 2 * e + 1], b);
              pk[2 * e] = pack_f16(a.x, a.y);
              pk[2 * e + 1] = pack_f16(b.x, b.y);
            }
            const uint32_t box = prow + (cb >> 2) * C::kBoxBytes;
            const int word = (cb & 3) * 2;               // 16-byte word of the key's rows: 8 words a box
            sts_u4(box + ((word ^ (key & 7)) << 4), make_uint4(pk[0], pk[1], pk[2], pk[3]));
            sts_u4(box + (((word + 1) ^ (key & 7)) << 4), make_uint4(pk[4], pk[5], pk[6], pk[7]));
          }
        }
        return fmaxf(top[0], top[1]);
      };
      // (the first tile sets the references: its weights are worked out once they are)
      const bool moves = u == 0 || (!dead && weigh(false) > kLimit);
      if (named_any(bar, 128, moves || dead)) {
        // A row's weights passed the limit (or it has no reference yet): the rows' maxima over the tile, new
        // references for those rows, O scaled, the tile weighed again. All warps of the group come here or none.
        if (named_any(bar, 128, dead)) break;
#pragma unroll 1
        for (int r = 0; r < w.rows; r += 8) {
          uint32_t sr[8];
          tmem_ld8(s_at + r, sr);
          float mine = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float m = warp_max(r + e >= n_min ? __uint_as_float(sr[e]) : -INFINITY);
            mine = lane == e ? m : mine;
          }
          if (lane < 8) sh->part[grp][wq][r + lane] = mine;
        }
        named_sync(bar, 128);
        if (tg < NT) {
          const float old = sh->neg_ref[grp][tg];
          float a = 1.f;
          if (tg < w.rows) {
            const float m = fmaxf(fmaxf(sh->part[grp][0][tg], sh->part[grp][1][tg]),
                                  fmaxf(sh->part[grp][2][tg], sh->part[grp][3][tg])) * q_scale;
            if (m + old > kLimit) {
              a = old == kNone ? 0.f : ex2_approx(kTop - m - old);
              sh->neg_ref[grp][tg] = kTop - m;
            }
          }
          sh->old_ref[grp][tg] = old;
          sh->alpha[grp][tg] = a;
        }
        named_sync(bar, 128);
        if (u > 0) {
#pragma unroll 1
          for (int r = 0; r < w.rows; r += 8) {
            uint32_t o[8];
            tmem_ld8(o_at + r, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sh->alpha[grp][r + e]);
            tmem_st8_async(o_at + r, o);
          }
          tmem_wait_st();
        }
        weigh(u > 0);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_ready[grp]);
    }
    // ---- epilogue: the groups' sums and O merged into the split's partial (m, l, O not normalised) ----
    if (u > 0 && !dead) dead = !__all_sync(0xffffffffu, mbar_wait(&sh->pv_done[grp], (u - 1) & 1, abort, p.err));
#pragma unroll
    for (int cb = 0; cb < NT / 8; ++cb) {
      if (cb * 8 < w.rows) {
        const float sum = sum_rows8(&l[cb * 4], lane);
        if (lane < 8) sh->part[grp][wq][cb * 8 + lane] = sum;
      }
    }
    tc_fence_before();
    named_sync(1, 256);
    tc_fence_after();
    if (static_cast<int>(threadIdx.x) < w.rows) {
      const int r = threadIdx.x;
      float lg[2], ref[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        lg[g] = (sh->part[g][0][r] + sh->part[g][1][r]) + (sh->part[g][2][r] + sh->part[g][3][r]);
        ref[g] = lg[g] > 0.f ? -sh->neg_ref[g][r] : -INFINITY;
      }
      const float m = fmaxf(ref[0], ref[1]);
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float wt = lg[g] > 0.f ? ex2_approx(ref[g] - m) : 0.f;
        sum += wt * lg[g];
        sh->alpha[g][r] = wt * p.v_scale;
      }
      const int rg = w.row0 + r;
      const size_t pidx = ((static_cast<size_t>(w.b) * p.row_tiles + rg / kMaxRows) * p.hkv + w.h) * p.num_splits + w.s;
      reinterpret_cast<float2*>(p.part_ml)[pidx * kMaxRows + rg % kMaxRows] = make_float2(m, sum);
    }
    named_sync(1, 256);
    if (w.nt > 0 && wq * 32 < HD) {
      // lane = channel: 32 neighbouring channels of a row are one 128-byte store. The groups take rows of eight in turn.
#pragma unroll 1
      for (int r0 = grp * 8; r0 < w.rows; r0 += 16) {
        uint32_t o0[8], o1[8];
        tmem_ld8(lane_base + kColO + r0, o0);
        tmem_ld8(lane_base + kColO + 96 + r0, o1);
        const int rg = w.row0 + r0;                      // (a multiple of 8: the eight lie in one of the combine's tiles)
        float* dst = p.part_o +
                     ((((static_cast<size_t>(w.b) * p.row_tiles + rg / kMaxRows) * p.hkv + w.h) * p.num_splits + w.s) * kMaxRows +
                      rg % kMaxRows) * HD + wq * 32 + lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (r0 + e < w.rows) {
            const float w0 = sh->alpha[0][r0 + e], w1 = sh->alpha[1][r0 + e];
            dst[e * HD] = (w0 > 0.f ? w0 * __uint_as_float(o0[e]) : 0.f) + (w1 > 0.f ? w1 * __uint_as_float(o1[e]) : 0.f);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

template <int HD, int NT>
cudaError_t launch_t(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  static size_t done[64] = {};
  static bool registers = false;
  auto kern = attend_packed_kernel<HD, NT>;
  if (!registers) {
    // The warpgroups trade registers; a kernel launched with fewer than they take up would wait for ever.
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    if (NT > kFewN && a.numRegs < kRegsLaunch) return cudaErrorNotSupported;
    registers = true;
  }
  const cudaError_t e = ensure_smem_limit(kern, Cfg<HD, NT>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.num_splits, p.hkv, num_seqs * p.n_tiles);
  return launch_pdl(kern, grid, dim3(kThreads), Cfg<HD, NT>::kSmemBytes, stream, p);
}

}  // namespace

int packed_tile_rows() { return kMaxN; }

cudaError_t launch_attend_packed(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  if (p.tile_rows <= kFewN)
    return p.head_dim == 128 ? launch_t<128, kFewN>(p, num_seqs, stream) : launch_t<64, kFewN>(p, num_seqs, stream);
  return p.head_dim == 128 ? launch_t<128, kMaxN>(p, num_seqs, stream) : launch_t<64, kMaxN>(p, num_seqs, stream);
}

}  // namespace vfy
