// Attention of a block over a pool of 4-bit chunks, on the tensor cores with the operands exchanged: a tile's 128 keys are
// the M = 128 side of both products and the block's rows (queries x q-heads of one KV head, at most 72) the N side,
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
//   softmax          a lane is a key, its 32-bit columns are the rows. Each warpgroup has up to 24 (8) of the rows, with their
//                    reference, sums and columns of O: the groups meet only in the MMAs. While a tile's weights are
//                    worked out, the next tile's scores are on their way and the vote whether one of them passes the limit.
//   K, V             two warpgroups each, which take tiles in turn: a lane reads its key's codes and scales, writes fp16
//                    into tensor memory (K, the A operand of S) or shared memory (V, channels contiguous: the A operand
//                    of O^T, M-major)
//   one warp         bulk copies of the records (contiguous: no tensor map), and the tiles' geometry
//   two warps        the MMA issuers of S and of O
#include <cuda_bf16.h>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kKeys = 2 * kChunk;         // keys of a tile
constexpr int kFewN = 16, kMaxN = 72;     // rows of a tile (two kernels)
constexpr int kBatch = 16;                // tiles whose chunks a warp's lanes hold; their geometry lies in two such batches
constexpr uint32_t kTmemCols = 512;
constexpr float kTop = 7.f;               // a row's maximum when its reference is set (log2)
constexpr float kLimit = 15.f;            // the reference moves when a weight would pass 2^15
constexpr float kNone = 1e30f;            // minus the reference of a row that has none: every score passes the limit

template <int HD, int NT>
struct Cfg {
  static constexpr bool kFew = NT <= kFewN;
  static constexpr int kSoftmax = kFew ? 2 : 3;                  // warpgroups of softmax
  static constexpr int kRowsT = NT / kSoftmax;                   // rows of a softmax thread
  static constexpr int kUnpack = 2;                              // warpgroups of K, and of V
  static constexpr int kGroups = kSoftmax + 2 * kUnpack + 1;
  static constexpr int kThreads = kGroups * 128;
  static constexpr int kKWarp = 4 * kSoftmax, kVWarp = kKWarp + 4 * kUnpack;
  static constexpr int kProducerWarp = kVWarp + 4 * kUnpack, kMmaWarp = kProducerWarp + 1;
  // Registers: with 72 rows the softmax groups take up what the others give up.
  static constexpr bool kTrade = !kFew;
  static constexpr int kRegsLaunch = 64, kRegsSoftmax = 104, kRegsUnpack = 40, kRegsRest = 40;
  static_assert(!kTrade || kSoftmax * kRegsSoftmax + 2 * kUnpack * kRegsUnpack + kRegsRest <= kGroups * kRegsLaunch,
                "registers the CTA was launched with");
  static constexpr int kN = (NT + 15) / 16 * 16;                 // N of the MMAs: multiples of 16
  static constexpr int kStages = 4;
  static constexpr int kKBufs = kFew ? 4 : 2, kSBufs = kFew ? 4 : 3;   // in tensor memory
  static constexpr int kVBufs = kFew ? 3 : 2;
  // columns: K tiles of up to 64 (two fp16 channels each), S^T, O^T
  static constexpr uint32_t kColS = kKBufs * 64, kColO = kColS + kSBufs * kN;
  static_assert(kColO + kN <= kTmemCols && kStages % kUnpack == 0, "tensor memory, stages");
  static constexpr int kRecord = kPackedBytes<HD>;
  static constexpr int kStageBytes = 4 * kRecord;                // K and V of two chunks
  static constexpr int kBoxBytes = kKeys * 128;                  // 64 columns of 128 keys
  static constexpr int kVBytes = 2 * kBoxBytes;                  // M = 128: d = 64 leaves the second box zero
  static constexpr int kPBytes = (kN + 63) / 64 * kBoxBytes;
  static constexpr int kQBoxBytes = kN * 128;
  static constexpr int kQBytes = (HD / 64) * kQBoxBytes;
  static constexpr int kVOffset = 0;
  static constexpr int kPOffset = kVBufs * kVBytes;
  static constexpr int kQOffset = kPOffset + 2 * kPBytes;
  static constexpr int kStageOffset = kQOffset + kQBytes;
  static constexpr int kBarOffset = kStageOffset + kStages * kStageBytes;
  static constexpr int kBarBytes = 6144;
  static constexpr int kSmemBytes = kBarOffset + kBarBytes + 1024;
  static_assert(kRecord % 16 == 0 && kStageBytes % 128 == 0, "bulk copies");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Shared {
  uint64_t full[4], empty[4];
  uint64_t geo_full[2];
  uint64_t k_ready[4], k_free[4];
  uint64_t s_done[4], s_free[4];          // S^T written; read
  uint64_t v_ready[3], v_free[3];
  uint64_t p_ready[2], pv_done[2];        // P written; O^T holds the tile, its P is free
  uint64_t vote[3], meet[3];              // [softmax group]: of one tile; where a reference moves
  uint64_t q_ready, drain[2], never;
  uint32_t tmem_base;
  int abort;
  unsigned q_top;                         // largest |q| of the tile, as bf16 bits
  int moves[3][2];                        // [softmax group][tile parity]: a weight would pass the limit
  int base[2 * kBatch][2];                // position of a chunk's first token, -1: no chunk
  int plain[2 * kBatch];                  // every row attends every key of the tile
  alignas(16) float neg_ref[kMaxN];       // minus the rows' reference, log2 units
  alignas(16) float alpha[kMaxN];
  alignas(16) float part[4][kMaxN];       // [lane quarter]: maxima, at the end sums
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
__global__ void __launch_bounds__(Cfg<HD, NT>::kThreads, 1) attend_packed_kernel(const PackedAttnParams p) {
  using C = Cfg<HD, NT>;
  constexpr int kStages = C::kStages, kThreads = C::kThreads;
  constexpr int kKWarp = C::kKWarp, kVWarp = C::kVWarp, kProducerWarp = C::kProducerWarp, kMmaWarp = C::kMmaWarp;
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
    for (int i = 0; i < C::kKBufs; ++i) {
      mbar_init(&sh->k_ready[i], 4);
      mbar_init(&sh->k_free[i], 1);
    }
    for (int i = 0; i < C::kSBufs; ++i) {
      mbar_init(&sh->s_done[i], 1);
      mbar_init(&sh->s_free[i], 4 * C::kSoftmax);
    }
    for (int i = 0; i < C::kVBufs; ++i) {
      mbar_init(&sh->v_ready[i], 4);
      mbar_init(&sh->v_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->geo_full[i], 1);
      mbar_init(&sh->p_ready[i], 4 * C::kSoftmax);
      mbar_init(&sh->pv_done[i], 1);
    }
    for (int i = 0; i < C::kSoftmax; ++i) {
      mbar_init(&sh->vote[i], 4);
      mbar_init(&sh->meet[i], 4);
      sh->moves[i][0] = sh->moves[i][1] = 0;
    }
    mbar_init(&sh->q_ready, 4 * C::kSoftmax);
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
    for (int x = threadIdx.x; x < C::kVBufs * C::kBoxBytes / 16; x += kThreads) {
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
    if constexpr (C::kTrade) regs_dec<C::kRegsRest>();
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
          int sb = 0, s_phase = 1;                       // S buffer; the parity of its earlier use
          for (int j = 0; j < nt; ++j) {
            const int kb = j % C::kKBufs;
            ok = wait(&sh->k_ready[kb], j / C::kKBufs & 1) && (j < C::kSBufs || wait(&sh->s_free[sb], s_phase));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                mma_ts(C::kColS + sb * C::kN, kb * 64 + kk * 8,
                       qdesc + static_cast<uint64_t>(((kk >> 2) * C::kQBoxBytes + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
              mma_commit(&sh->s_done[sb]);
              mma_commit(&sh->k_free[kb]);
            }
            __syncwarp();
            if (++sb == C::kSBufs) sb = 0, s_phase ^= 1;
          }
        } else {
          const uint32_t idesc = idesc_f16_f32(128, n, 1, 1);
          const uint64_t vdesc = sw128_desc(sbase + C::kVOffset, C::kBoxBytes, 1024);
          const uint64_t pdesc = sw128_desc(sbase + C::kPOffset, C::kBoxBytes, 1024);
          int vb = 0, v_phase = 0;
          for (int j = 0; j < nt; ++j) {
            const int g = j & 1, ph = (j >> 1) & 1;
            ok = wait(&sh->v_ready[vb], v_phase) && wait(&sh->p_ready[g], ph);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ss(C::kColO, vdesc + static_cast<uint64_t>((vb * C::kVBytes + kk * 2048) >> 4),
                       pdesc + static_cast<uint64_t>((g * C::kPBytes + kk * 2048) >> 4), idesc, (j > 0 || kk > 0) ? 1u : 0u);
              mma_commit(&sh->pv_done[g]);
              mma_commit(&sh->v_free[vb]);
            }
            __syncwarp();
            if (++vb == C::kVBufs) vb = 0, v_phase ^= 1;
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
    if constexpr (C::kTrade) regs_dec<C::kRegsUnpack>();
    const bool is_v = warp >= kVWarp;
    const int wg = (warp >> 2) - (is_v ? kVWarp : kKWarp) / 4;   // takes tiles wg, wg + kUnpack, ...
    const int key = (warp & 3) * 32 + lane;              // of the tile; a TMEM lane
    const int c = key / kChunk, tok = key % kChunk;
    const int bufs = is_v ? C::kVBufs : C::kKBufs;
    uint64_t* free_bar = is_v ? sh->v_free : sh->k_free;
    uint64_t* ready_bar = is_v ? sh->v_ready : sh->k_ready;
    const uint32_t rec = sbase + C::kStageOffset + ((is_v ? 2 : 0) + c) * C::kRecord;
    const uint32_t scales_at = rec + kChunk * (HD / 2) + tok * (HD / 16);
    const uint32_t codes_at = rec + tok * 16;
    int st = wg, stage_phase = 0;
    int buf = wg, free_phase = 1;                        // of this WG's next tile; its buffer's earlier use
    for (int j = wg; j < w.nt; j += C::kUnpack) {
      bool ok = mbar_wait_tested(&sh->full[st], stage_phase, abort, p.err);
      if (is_v && j % kBatch < C::kUnpack && ok)
        ok = mbar_wait_tested(&sh->geo_full[j / kBatch & 1], j / kBatch >> 1 & 1, abort, p.err);
      if (ok && j >= bufs) ok = mbar_wait_tested(&free_bar[buf], free_phase, abort, p.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t kto = (static_cast<uint32_t>((warp & 3) * 32) << 16) + buf * 64;
      const uint32_t vto = sbase + C::kVOffset + buf * C::kVBytes + key * 128;
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
        mbar_arrive(&ready_bar[buf]);
      }
      st += C::kUnpack;
      if (st >= C::kStages) st -= C::kStages, stage_phase ^= 1;
      buf += C::kUnpack;
      if (buf >= bufs) buf -= bufs, free_phase ^= 1;
    }
  } else {
    // ------------------------------ softmax ---------------------------------------------------
    if constexpr (C::kTrade) regs_inc<C::kRegsSoftmax>();
    constexpr int kAll = 128 * C::kSoftmax;
    const int grp = warp >> 2, wq = warp & 3;
    const int rows_each = ((w.rows + C::kSoftmax - 1) / C::kSoftmax + 7) & ~7;
    const int row_first = grp * rows_each;
    const int my_rows = max(0, min(rows_each, w.rows - row_first));
    const int tg = threadIdx.x & 127;                    // thread of the group; its key of a tile
    const int key = tg;
    // Q: words of 8 channels, all of a thread's in registers while the tile's largest value is found
    constexpr int kWords = (C::kN * HD / 8 + kAll - 1) / kAll;
    float q_scale;                                       // of a score: softmax scale, g of K, the queries' power of two
    {
      uint4 qv[kWords];
      unsigned top = 0u;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int x = threadIdx.x + i * kAll;
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
      named_sync(1, kAll);
      const int qe = max(static_cast<int>(sh->q_top >> 7) - 127 - 14, -100);
      const float down = __int_as_float((127 - qe) << 23);
      q_scale = p.scale_log2 * __int_as_float((127 + qe) << 23);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int x = threadIdx.x + i * kAll;
        const int r = x / (HD / 8), cw = x % (HD / 8);
        const uint32_t ws[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_f16(__uint_as_float(ws[e] << 16) * down, __uint_as_float(ws[e] & 0xffff0000u) * down);
        if (r < C::kN)
          *reinterpret_cast<uint4*>(sQ + (cw >> 3) * C::kQBoxBytes + r * 128 + (((cw & 7) ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_ready);
    }
    // (rows past the block, Q = 0, keep weight 1: never read)
    if (static_cast<int>(threadIdx.x) < NT) sh->neg_ref[threadIdx.x] = static_cast<int>(threadIdx.x) < w.rows ? kNone : 0.f;
    named_sync(1, kAll);

    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t o_at = lane_base + C::kColO + row_first;
    const uint32_t prow = sbase + C::kPOffset + key * 128;
    const int p0 = w.L - w.nq;
    const float2 sc2 = make_float2(q_scale, q_scale);
    float2 l[C::kRowsT / 2];
#pragma unroll
    for (int r = 0; r < C::kRowsT / 2; ++r) l[r] = make_float2(0.f, 0.f);
    auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mbar_wait_tested(bar, parity, abort, p.err)); };
    int met = 0;                                         // the group's meetings so far
    auto meet = [&]() {                                  // all warps of the group, what they wrote to shared memory seen
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->meet[grp]);
      return wait(&sh->meet[grp], met++ & 1);
    };
    // Rows from n_min on attend this lane's key of tile j: row n is of block query (row0 + n) / G, at position p0 + that.
    auto first_row = [&](int j) -> int {
      const int geo = j % (2 * kBatch);
      if (sh->plain[geo]) return 0;
      const int base = sh->base[geo][key / kChunk], pos = base + key % kChunk;
      if (base < 0 || pos >= w.L) return NT;
      return pos > p0 ? min(static_cast<long long>(NT), max(0ll, static_cast<long long>(pos - p0) * p.group - w.row0)) : 0;
    };
    auto s_address = [&](int buf) { return lane_base + C::kColS + buf * C::kN + row_first; };
    auto load_scores = [&](uint32_t(&x)[C::kRowsT], int buf) {
      tc_fence_after();
#pragma unroll
      for (int r = 0; r < C::kRowsT; r += 8) tmem_ld8_async(s_address(buf) + r, *reinterpret_cast<uint32_t(*)[8]>(x + r));
    };
    // Scores to exponents s scale - ref, masked keys to -inf; the largest.
    auto exponents = [&](uint32_t(&x)[C::kRowsT], int n_min) -> float {
      tmem_wait_ld(x);
      if (!__all_sync(0xffffffffu, n_min == 0)) {
#pragma unroll
        for (int r = 0; r < C::kRowsT; ++r) x[r] = row_first + r >= n_min ? x[r] : 0xff800000u;
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int r = 0; r < C::kRowsT; r += 8) {
        if (r < my_rows) {
          const float4* nr = reinterpret_cast<const float4*>(&sh->neg_ref[row_first + r]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 f = nr[e];
            const float2 a = fma_f32x2(pair(x, r + 4 * e), sc2, make_float2(f.x, f.y));
            const float2 b = fma_f32x2(pair(x, r + 4 * e + 2), sc2, make_float2(f.z, f.w));
            top[0] = fmaxf(fmaxf(top[0], a.x), a.y);
            top[1] = fmaxf(fmaxf(top[1], b.x), b.y);
            x[r + 4 * e] = __float_as_uint(a.x);
            x[r + 4 * e + 1] = __float_as_uint(a.y);
            x[r + 4 * e + 2] = __float_as_uint(b.x);
            x[r + 4 * e + 3] = __float_as_uint(b.y);
          }
        }
      }
      return fmaxf(top[0], top[1]);
    };
    auto vote = [&](float top, int j) {
      if (top > kLimit) sh->moves[grp][j & 1] = 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->vote[grp]);
    };
    int sb = 0;                                          // S buffer of the current tile
    int next_buf = 0, next_phase = 0;                    // and of the next
    auto step_buf = [&]() { if (++next_buf == C::kSBufs) next_buf = 0, next_phase ^= 1; };
    // One tile: its exponents are in `x` and their vote is under way; those of the next come into `next`.
    auto tile = [&](uint32_t(&x)[C::kRowsT], uint32_t(&next)[C::kRowsT], int j) -> bool {
      const int g = j & 1;
      const bool more = j + 1 < w.nt;
      bool loading = false;
      if (more) {
        loading = __all_sync(0xffffffffu, mbar_test_wait(&sh->s_done[next_buf], next_phase));
        if (loading) load_scores(next, next_buf);
      }
      if (!wait(&sh->vote[grp], j & 1)) return false;
      if (sh->moves[grp][g]) {
        // A weight would pass the limit, or a row has no reference yet: the rows' maxima over the tile, new references for
        // those rows, their sums and O scaled, the exponents again. All warps of the group come here or none.
        const int n_min = first_row(j);
#pragma unroll 1
        for (int r = 0; r < my_rows; r += 8) {
          uint32_t sr[8];
          tmem_ld8(s_address(sb) + r, sr);
          float mine = -INFINITY;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float m = warp_max(row_first + r + e >= n_min ? __uint_as_float(sr[e]) : -INFINITY);
            mine = lane == e ? m : mine;
          }
          if (lane < 8) sh->part[wq][row_first + r + lane] = mine;
        }
        if (!meet()) return false;
        if (tg == 0) sh->moves[grp][g] = 0;
        if (tg < my_rows) {
          const int r = row_first + tg;
          const float m = fmaxf(fmaxf(sh->part[0][r], sh->part[1][r]), fmaxf(sh->part[2][r], sh->part[3][r])) * q_scale;
          const float old = sh->neg_ref[r];
          float a = 1.f;
          if (m + old > kLimit) {
            a = old == kNone ? 0.f : ex2_approx(kTop - m - old);
            sh->neg_ref[r] = kTop - m;
          }
          sh->alpha[r] = a;
        }
        if (!meet()) return false;
        if (j > 0) {
          if (!wait(&sh->pv_done[g ^ 1], ((j - 1) >> 1) & 1)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int r = 0; r < my_rows; r += 8) {
            uint32_t o[8];
            tmem_ld8(o_at + r, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sh->alpha[row_first + r + e]);
            tmem_st8_async(o_at + r, o);
          }
          tmem_wait_st();
#pragma unroll
          for (int r = 0; r < C::kRowsT; r += 2) {
            if (r < my_rows) {
              const float2 a = *reinterpret_cast<const float2*>(&sh->alpha[row_first + r]);
              l[r / 2].x *= a.x;
              l[r / 2].y *= a.y;
            }
          }
        }
        load_scores(x, sb);
        exponents(x, n_min);
      }
      tc_fence_before();
      if (lane == 0) mbar_arrive(&sh->s_free[sb]);
      if (more) {
        if (j % kBatch == kBatch - 1 && !wait(&sh->geo_full[(j + 1) / kBatch & 1], (j + 1) / kBatch >> 1 & 1)) return false;
        if (!loading) {
          if (!__all_sync(0xffffffffu, mbar_wait(&sh->s_done[next_buf], next_phase, abort, p.err))) return false;
          load_scores(next, next_buf);
        }
        vote(exponents(next, first_row(j + 1)), j + 1);
      }
      sb = next_buf;
      step_buf();
      // Weights 2^x to shared memory, and their sums
      if (j >= 2 && !wait(&sh->pv_done[g], ((j >> 1) - 1) & 1)) return false;
#pragma unroll
      for (int r = 0; r < C::kRowsT; r += 8) {
        if (r < my_rows) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 a = pair(x, r + 2 * e);
            a.x = ex2_approx(a.x);
            a.y = ex2_approx(a.y);
            l[r / 2 + e] = add_f32x2(l[r / 2 + e], a);
            pk[e] = pack_f16(a.x, a.y);
          }
          const int word = (row_first + r) / 8;          // 16-byte word of the key's rows: 8 words a box
          sts_u4(prow + g * C::kPBytes + (word >> 3) * C::kBoxBytes + (((word & 7) ^ (key & 7)) << 4),
                 make_uint4(pk[0], pk[1], pk[2], pk[3]));
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_ready[g]);
      return true;
    };
    bool ok = true;
    if (w.nt > 0) {
      uint32_t xa[C::kRowsT], xb[C::kRowsT];
      ok = wait(&sh->geo_full[0], 0) && wait(&sh->s_done[0], 0);
      if (ok) {
        load_scores(xa, 0);
        vote(exponents(xa, first_row(0)), 0);
        step_buf();
        for (int j = 0; ok && j < w.nt; j += 2) {
          ok = tile(xa, xb, j);
          if (ok && j + 1 < w.nt) ok = tile(xb, xa, j + 1);
        }
      }
    }
    // ---- epilogue: the split's partial (m, l, O not normalised) ----
    if (ok && w.nt > 0) ok = wait(&sh->pv_done[(w.nt - 1) & 1], ((w.nt - 1) >> 1) & 1);
    tc_fence_after();
#pragma unroll
    for (int r = 0; r < C::kRowsT; r += 8) {
      if (r < my_rows) {
        const float sum = sum_rows8(&l[r / 2], lane);
        if (lane < 8) sh->part[wq][row_first + r + lane] = sum;
      }
    }
    named_sync(1, kAll);
    if (static_cast<int>(threadIdx.x) < w.rows) {
      const int r = threadIdx.x;
      const float sum = (sh->part[0][r] + sh->part[1][r]) + (sh->part[2][r] + sh->part[3][r]);
      const int rg = w.row0 + r;
      const size_t pidx = ((static_cast<size_t>(w.b) * p.row_tiles + rg / kMaxRows) * p.hkv + w.h) * p.num_splits + w.s;
      reinterpret_cast<float2*>(p.part_ml)[pidx * kMaxRows + rg % kMaxRows] =
          make_float2(sum > 0.f ? -sh->neg_ref[r] : -INFINITY, sum);
    }
    if (w.nt > 0 && wq * 32 < HD) {
      // lane = channel: 32 neighbouring channels of a row are one 128-byte store
#pragma unroll 1
      for (int r = 0; r < my_rows; r += 8) {
        uint32_t o[8];
        tmem_ld8(o_at + r, o);
        const int rg = w.row0 + row_first + r;           // (a multiple of 8: the eight lie in one of the combine's tiles)
        float* dst = p.part_o +
                     ((((static_cast<size_t>(w.b) * p.row_tiles + rg / kMaxRows) * p.hkv + w.h) * p.num_splits + w.s) * kMaxRows +
                      rg % kMaxRows) * HD + wq * 32 + lane;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (r + e < my_rows) dst[e * HD] = __uint_as_float(o[e]) * p.v_scale;
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
    if (Cfg<HD, NT>::kTrade && a.numRegs < Cfg<HD, NT>::kRegsLaunch) return cudaErrorNotSupported;
    registers = true;
  }
  const cudaError_t e = ensure_smem_limit(kern, Cfg<HD, NT>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.num_splits, p.hkv, num_seqs * p.n_tiles);
  return launch_pdl(kern, grid, dim3(Cfg<HD, NT>::kThreads), Cfg<HD, NT>::kSmemBytes, stream, p);
}

}  // namespace

int packed_tile_rows() { return kMaxN; }

cudaError_t launch_attend_packed(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  if (p.tile_rows <= kFewN)
    return p.head_dim == 128 ? launch_t<128, kFewN>(p, num_seqs, stream) : launch_t<64, kFewN>(p, num_seqs, stream);
  return p.head_dim == 128 ? launch_t<128, kMaxN>(p, num_seqs, stream) : launch_t<64, kMaxN>(p, num_seqs, stream);
}

}  // namespace vfy
