// Attention of a block over a pool of 4-bit chunks, more than 16 rows a KV head, on the tensor cores with the operands
// exchanged: a tile's 128 keys are the M = 128 side of both products and the block's rows (queries x q-heads of one KV head,
// at most 72) the N side,
//     S^T [128 keys][rows] = K Q^T,    O^T [d][rows] += V^T P^T,
// so that the work follows the rows a block has: a block of 17 with G = 4 is N = 80 (68 rows). With the rows as M (as in the
// bf16 layers) a 4-bit tile would be bound by the 128 rows' tensor time.
//
// A value is g s e; s e has 6 significant bits, so the operands in fp16 are exact. Queries are bf16: the tile's are scaled by
// one power of two that puts the largest at 2^14, and fp16 holds all 8 bits of what is above 2^-28 of it. Weights P are
// fp16 too (half a step, 2^-11): a row's reference is put 7 below its maximum (log2), weights grow to 2^15 before the
// reference moves, and what fp16 drops (below 2^-25) is 2^-32 of the largest weight.
//
// One CTA per (split, KV head, sequence and row tile), a contiguous run of tiles of two chunks. Roles:
//   softmax          of even / odd tiles: a lane is a key, its 32-bit columns are the rows. Two groups with a reference, row
//                    sums and O of their own, merged at the end; a group has two tiles' time for one. A group is two
//                    warpgroups, each with half of the rows, all of them in registers; a vote of the group says whether a
//                    reference has to move, which is rare: then the tile is read again from tensor memory.
//   K                a lane reads its key's codes and scales, writes fp16 into tensor memory (the A operand of S)
//   V                the same into shared memory, channels contiguous (the A operand of O^T, M-major)
//   one warp         bulk copies of the records (contiguous: no tensor map), and the tiles' geometry
//   two warps        the MMA issuers of S and of O
//
// 17 rows, 16 q-heads over 4 KV heads, d = 128: 256K tokens in 58.9 us, 8K in 13.2, eight ragged sequences of 12K to 48K in
// 64.5. A tile takes 1.8 thousand cycles. Shared memory moves 1.35 of them (V written and read 512, P and Q 450, records
// 290), the schedulers issue 1.2 (K and V to fp16 a third, weights a third); the records alone, from HBM, would be 0.8.
#include <cuda_bf16.h>

#include <type_traits>

#include "packed.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kGroups = 8;                // warpgroups: softmax (0-3), K, V (of even, of odd tiles), the rest
constexpr int kThreads = kGroups * 128, kVGroups = 2;
constexpr int kRegsLaunch = 64, kRegsSoftmax = 96, kRegsUnpack = 32, kRegsRest = 32;
static_assert(4 * kRegsSoftmax + (1 + kVGroups) * kRegsUnpack + kRegsRest <= kGroups * kRegsLaunch, "registers the CTA was launched with");
constexpr int kKWarp = 16, kVWarp = 20, kProducerWarp = 28, kMmaWarp = 29;
constexpr int kKeys = 2 * kChunk;         // keys of a tile
constexpr int kMaxN = 72, kN = 80;        // rows of a tile; N of the MMAs, a multiple of 16
static_assert(kMaxN == 72, "rows of the two halves of a group");
constexpr int kRowsT = kMaxN / 2;         // rows of a softmax thread, which holds their scores and sums
constexpr int kStages = 4;
constexpr int kBatch = 16;                // tiles whose chunks a warp's lanes hold; their geometry lies in two such batches
constexpr uint32_t kTmemCols = 512;
constexpr float kTop = 7.f;               // a row's maximum when its reference is set (log2)
constexpr float kLimit = 15.f;            // the reference moves when a weight would pass 2^15
// columns of tensor memory: two K tiles of up to 64 (two fp16 channels each), S^T and O^T of the two groups
constexpr uint32_t kColS = 128, kColO = kColS + 2 * kN;
static_assert(kColO + 2 * kN <= kTmemCols, "tensor memory");

template <int HD>
struct Cfg {
  static constexpr int kRecord = kPackedBytes<HD>;
  static constexpr int kStageBytes = 4 * kRecord;                // K and V of two chunks
  static constexpr int kBoxBytes = kKeys * 128;                  // 64 columns of 128 keys
  static constexpr int kVBytes = 2 * kBoxBytes;                  // M = 128: d = 64 leaves the second box zero
  static constexpr int kPBytes = 2 * kBoxBytes;
  static constexpr int kQBoxBytes = kN * 128;
  static constexpr int kQBytes = (HD / 64) * kQBoxBytes;
  static constexpr int kVOffset = 0;
  static constexpr int kPOffset = 2 * kVBytes;
  static constexpr int kQOffset = kPOffset + 2 * kPBytes;
  static constexpr int kStageOffset = kQOffset + kQBytes;
  static constexpr int kBarOffset = kStageOffset + kStages * kStageBytes;
  static constexpr int kBarBytes = 6144;
  static constexpr int kSmemBytes = kBarOffset + kBarBytes + 1024;
  static_assert(kRecord % 16 == 0 && kStageBytes % 128 == 0, "bulk copies");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t geo_full[2];
  // of even / odd tiles
  uint64_t k_ready[2], s_done[2], s_free[2];   // K written; S^T written and K free; S^T read
  uint64_t v_ready[2], p_ready[2];
  uint64_t pv_done[2];                    // O^T holds the tile, its P and V are free
  uint64_t q_ready, drain[2], never;
  uint32_t tmem_base;
  int abort;
  unsigned q_top;                         // largest |q| of the tile, as bf16 bits
  int base[2 * kBatch][2];                // position of a chunk's first token, -1: no chunk
  // [group]: each group writes and reads its own, with its own barrier between (a group without tiles meets no other wait)
  int seq[2];                             // of the batch
  int4 geom[2];                           // length, position of the block's first token, first row, rows: read
                                          // where they are needed, registers are short
  int plain[2 * kBatch];                  // every row attends every key of the tile
  alignas(16) float neg_ref[2][kMaxN];    // [group] minus the rows' reference, log2 units
  alignas(16) float alpha[2][kMaxN];      // a factor of what was summed before the reference moved
  alignas(16) float part[2][4][kMaxN];    // [group][lane quarter]: maxima, at the end sums
};
static_assert(sizeof(Shared) <= Cfg<128>::kBarBytes, "barrier block");

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
  const int z = static_cast<int>(blockIdx.z / static_cast<unsigned>(p.n_tiles));
  const int rt = static_cast<int>(blockIdx.z) - z * p.n_tiles;
  const SequenceMeta meta = longest_first(p.cu_q, p.cu_res, p.seq_len, p.num_seqs, z, threadIdx.x & 31);
  const int c0 = meta.c0, c1 = meta.c1, cr0 = meta.r0, cr1 = meta.r1;
  w.b = meta.b;
  w.L = meta.len;
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
__device__ __forceinline__ void sts_u2(uint32_t at, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y));
}
// (no memory clobber: what is written is read by MMAs alone, behind a proxy fence, and loads may move ahead of it)
__device__ __forceinline__ void sts_u4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
}

// One value per row of four from 32 lanes: lane r (and every lane alike modulo 4) gets row r's sum.
__device__ __forceinline__ float sum_rows4(const float2* l2, int lane) {
  const bool h2 = lane & 2, h1 = lane & 1;
  const float2 mine = h2 ? l2[1] : l2[0], theirs = h2 ? l2[0] : l2[1];
  const float a = mine.x + __shfl_xor_sync(0xffffffffu, theirs.x, 2), b = mine.y + __shfl_xor_sync(0xffffffffu, theirs.y, 2);
  float c = (h1 ? b : a) + __shfl_xor_sync(0xffffffffu, h1 ? a : b, 1);
  c += __shfl_xor_sync(0xffffffffu, c, 4);
  c += __shfl_xor_sync(0xffffffffu, c, 8);
  c += __shfl_xor_sync(0xffffffffu, c, 16);
  return c;
}

// The K or V role of a warpgroup: tiles first, first + step, ... A lane has one key of the tile (a lane of tensor memory).
template <int HD, bool V>
__device__ __forceinline__ void unpack_tiles(const PackedAttnParams& p, const Work& w, Shared* sh, uint32_t sbase, int first,
                                             int step) {
  using C = Cfg<HD>;
  volatile int* abort = &sh->abort;
  const int lane = threadIdx.x & 31, key = threadIdx.x & 127;
  const int c = key / kChunk, tok = key % kChunk;
  const uint32_t rec = sbase + C::kStageOffset + ((V ? 2 : 0) + c) * C::kRecord;
  const uint32_t scales_at = rec + kChunk * (HD / 2) + tok * (HD / 16), codes_at = rec + tok * 16;
  // (a row of 128 bytes starts with zeros in the bits that the swizzle changes: one XOR a word)
  const uint32_t to = V ? sbase + C::kVOffset + key * 128 + ((key & 7) << 4) : static_cast<uint32_t>((key & 96) << 16);
  for (int j = first; j < w.nt; j += step) {
    const int st = j % kStages, g = j & 1;
    bool ok = mbar_wait_tested(&sh->full[st], j / kStages & 1, abort, p.err);
    if (V && j % kBatch == first && ok) ok = mbar_wait_tested(&sh->geo_full[j / kBatch & 1], j / kBatch >> 1 & 1, abort, p.err);
    if (ok && j >= 2) ok = mbar_wait_tested(V ? &sh->pv_done[g] : &sh->s_done[g], (j >> 1 & 1) ^ 1, abort, p.err);
    if (!__all_sync(0xffffffffu, ok)) break;
    const uint32_t at = st * C::kStageBytes;
    // Keys that no row attends may hold anything: P is 0 there, but 0 * NaN is NaN.
    bool keep = true;
    if (V && !sh->plain[j % (2 * kBatch)]) {
      const int base = sh->base[j % (2 * kBatch)][c];
      keep = base >= 0 && base + tok < w.L;
    }
    if (!V) tc_fence_after();
#pragma unroll
    for (int y = 0; y < HD / 64; ++y) {                  // 64 channels: two words of codes, four scales
      uint32_t scales = lds_u32(scales_at + at + 4 * y);
      if (V && !keep) scales = 0u;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 cw = lds_u4(codes_at + at + (2 * y + x) * kChunk * 16);
        const uint32_t two = e4m3_pair_f16(x == 0 ? scales & 0xffffu : scales >> 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {                    // 16 channels: one scale
          const uint32_t sc = __byte_perm(two, two, i == 0 ? 0x1010 : 0x3232);
          uint32_t out[8];
          unpack_word(i == 0 ? cw.x : cw.z, sc, out);
          unpack_word(i == 0 ? cw.y : cw.w, sc, out + 4);
          if constexpr (V) {
#pragma unroll
            for (int z = 0; z < 2; ++z)                  // 16-byte words of the 128-byte row
              sts_u4(((to + g * C::kVBytes) ^ ((x * 4 + 2 * i + z) << 4)) + y * C::kBoxBytes,
                     make_uint4(out[4 * z], out[4 * z + 1], out[4 * z + 2], out[4 * z + 3]));
          } else {
            tmem_st8_async(to + g * 64 + (4 * y + 2 * x + i) * 8, out);
          }
        }
      }
    }
    if constexpr (V) {
      fence_proxy_async_smem();
    } else {
      tmem_wait_st();
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh->empty[st]);
      mbar_arrive(V ? &sh->v_ready[g] : &sh->k_ready[g]);
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) attend_packed_kernel(const PackedAttnParams p) {
  using C = Cfg<HD>;
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
      mbar_init(&sh->s_done[i], 1);
      mbar_init(&sh->s_free[i], 8);
      mbar_init(&sh->v_ready[i], 4);
      mbar_init(&sh->p_ready[i], 8);
      mbar_init(&sh->pv_done[i], 1);
    }
    mbar_init(&sh->q_ready, 16);
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
    regs_dec<kRegsRest>();
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
      // One warp for S, one for O: issuing a tile's eight MMAs of one kind with its waits takes 500 to 600 cycles, as long as
      // the tensor core does. The whole warp runs the loop (see elect_one). Tensor memory is
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
          for (int j = 0; ok && j < nt; ++j) {
            const int g = j & 1, ph = j >> 1 & 1;
            ok = wait(&sh->k_ready[g], ph) && (j < 2 || wait(&sh->s_free[g], ph ^ 1));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                mma_ts(kColS + g * kN, g * 64 + kk * 8,
                       qdesc + static_cast<uint64_t>(((kk >> 2) * C::kQBoxBytes + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
              mma_commit(&sh->s_done[g]);
            }
            __syncwarp();
          }
        } else {
          const uint32_t idesc = idesc_f16_f32(128, n, 1, 1);
          const uint64_t vdesc = sw128_desc(sbase + C::kVOffset, C::kBoxBytes, 1024);
          const uint64_t pdesc = sw128_desc(sbase + C::kPOffset, C::kBoxBytes, 1024);
          for (int j = 0; ok && j < nt; ++j) {
            const int g = j & 1, ph = j >> 1 & 1;
            ok = wait(&sh->v_ready[g], ph) && wait(&sh->p_ready[g], ph);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ss(kColO + g * kN, vdesc + static_cast<uint64_t>((g * C::kVBytes + kk * 2048) >> 4),
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
    regs_dec<kRegsUnpack>();
    // (V waits for O of two tiles before: with one warpgroup for it a tile took 3% longer)
    if (warp >= kVWarp)
      unpack_tiles<HD, true>(p, w, sh, sbase, (warp - kVWarp) >> 2, kVGroups);
    else
      unpack_tiles<HD, false>(p, w, sh, sbase, 0, 1);
  } else {
    // ------------------------------ softmax ---------------------------------------------------
    regs_inc<kRegsSoftmax>();
    constexpr int kAll = 512, kGroup = 256;
    const int grp = warp >> 3, half = warp >> 2 & 1, wq = warp & 3;
    // Rows of this thread: every other eight of the first 64, four of the last eight.
    const int row_lo = half * 8, row_hi = 64 + half * 4;
    auto row_of = [&](int r) { return r < 32 ? (r >> 3) * 16 + row_lo + (r & 7) : row_hi + r - 32; };
    const int tg = threadIdx.x & 255;                    // thread of the group
    const int key = threadIdx.x & 127;
    const int bar = 2 + grp;                             // named barrier of the group; 1: both groups
    // Q: words of 8 channels, all of a thread's in registers while the tile's largest value is found
    constexpr int kWords = (kN * HD / 8 + kAll - 1) / kAll;
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
      const int qe = query_exponent(sh->q_top);
      const PowerOfTwo down(-qe);
      q_scale = score_scale(p.scale_log2, p.scale_exp, qe);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int x = threadIdx.x + i * kAll;
        const int r = x / (HD / 8), cw = x % (HD / 8);
        const uint32_t ws[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_f16(down.times(__uint_as_float(ws[e] << 16)), down.times(__uint_as_float(ws[e] & 0xffff0000u)));
        if (r < kN)
          *reinterpret_cast<uint4*>(sQ + (cw >> 3) * C::kQBoxBytes + r * 128 + (((cw & 7) ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_ready);
    }
    // No reference yet. Rows past the block weigh 0, whatever their scores hold: all 36 rows of a thread are computed
    // without a branch.
    if (tg < kMaxN) sh->neg_ref[grp][tg] = tg < w.rows ? 0.f : -INFINITY;
    if (tg == 0) {
      sh->seq[grp] = w.b;
      sh->geom[grp] = make_int4(w.L, w.L - w.nq, w.row0, w.rows);
    }
    bool has_ref = tg >= w.rows;                         // of row tg
    bool all_have = false;                               // of the group
    named_sync(bar, kGroup);

    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_at = lane_base + kColS + grp * kN;
    const uint32_t prow = sbase + C::kPOffset + grp * C::kPBytes + key * 128 + (((key & 7) ^ half) << 4);   // word `half` of the row
    const float2 sc2 = make_float2(q_scale, q_scale);
    float2 l[kRowsT / 2];
#pragma unroll
    for (int r = 0; r < kRowsT / 2; ++r) l[r] = make_float2(0.f, 0.f);
    bool dead = false;                                   // a wait of this warp gave up
    int u = 0;                                           // tiles of this group so far
    // R: rows of a thread. Up to 32 rows in all need no more than 16 (4 rows over 256K 49 us, with 36 of a thread 54.7; the second
    // loop costs the first half a microsecond: 17 rows 59.7 -> 60.2).
    auto tiles = [&](auto rows_of_thread) {
      constexpr int R = decltype(rows_of_thread)::value;
      for (int j = grp; j < w.nt; j += 2, ++u) {
        if (j % kBatch == grp && !mbar_wait_tested(&sh->geo_full[j / kBatch & 1], j / kBatch >> 1 & 1, abort, p.err)) dead = true;
        if (!mbar_wait_tested(&sh->s_done[grp], u & 1, abort, p.err)) dead = true;
        dead = __any_sync(0xffffffffu, dead);
        tc_fence_after();
        uint32_t s[R];
        const int geo = j % (2 * kBatch);
        bool pv = u == 0 || mbar_test_wait(&sh->pv_done[grp], (u - 1) & 1);
        pv = __all_sync(0xffffffffu, pv);
        bool stop = false;                                 // a warp of the group gave up
        for (bool again = false;; again = true) {
          // s = score - reference (log2)
#pragma unroll
          for (int r = 0; r < R / 8 * 8; r += 8) tmem_ld8_async(s_at + row_of(r), s + r);
          if constexpr (R % 8 != 0) tmem_ld4_async(s_at + row_hi, s + 32);
          tmem_wait_ld(s);
          if (!sh->plain[geo]) {
            // Rows from n_min on attend this lane's key: row n is of block query (row0 + n) / G, at position p0 + that.
            const int base = sh->base[geo][key / kChunk], pos = base + key % kChunk;
            const int4 gm = sh->geom[grp];
            int n_min = 0;
            if (base < 0 || pos >= gm.x)
              n_min = kMaxN;
            else if (pos > gm.y)
              n_min = min(static_cast<long long>(kMaxN), max(0ll, static_cast<long long>(pos - gm.y) * p.group - gm.z));
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = row_of(r) >= n_min ? s[r] : 0xff800000u;   // 2^-inf = 0
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sh->neg_ref[grp][row_of(r)]);
            const float2 a = fma_f32x2(pair(s, r), sc2, make_float2(f.x, f.y));
            const float2 b = fma_f32x2(pair(s, r + 2), sc2, make_float2(f.z, f.w));
            s[r] = __float_as_uint(a.x);
            s[r + 1] = __float_as_uint(a.y);
            s[r + 2] = __float_as_uint(b.x);
            s[r + 3] = __float_as_uint(b.y);
            top[r / 2 % 4] = fmaxf(fmaxf(top[r / 2 % 4], a.x), a.y);
            top[r / 2 % 4 + 1] = fmaxf(fmaxf(top[r / 2 % 4 + 1], b.x), b.y);
          }
          if (again) break;
          const bool moves = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > kLimit;
          if (all_have && !named_any(bar, kGroup, moves || dead)) break;
          // A row's weights would pass the limit, or a row has no reference yet: the rows' maxima over the tile, new
          // references for those rows, their sums and O scaled, and once more. All warps of the group come here or none.
          stop = named_any(bar, kGroup, dead);
          if (stop) break;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float m = warp_max(__uint_as_float(s[r]));
            if (lane == 0) sh->part[grp][wq][row_of(r)] = m;
          }
          named_sync(bar, kGroup);
          const int rows = sh->geom[grp].w;
          if (tg < rows) {
            const float m = fmaxf(fmaxf(sh->part[grp][0][tg], sh->part[grp][1][tg]),
                                  fmaxf(sh->part[grp][2][tg], sh->part[grp][3][tg]));
            float a = 1.f;
            if (m > (has_ref ? kLimit : -INFINITY)) {
              const float old = -sh->neg_ref[grp][tg], ref = old + (m - kTop);
              a = has_ref ? ex2_approx(old - ref) : 0.f;
              sh->neg_ref[grp][tg] = -ref;
              has_ref = true;
              if (!(fabsf(ref) < kMostScore)) atomicOr(p.err, kErrDeviceInput);
            }
            sh->alpha[grp][tg] = a;
          }
          all_have = !named_any(bar, kGroup, !has_ref);
          if (u > 0) {
            dead = !__all_sync(0xffffffffu, mbar_wait_tested(&sh->pv_done[grp], (u - 1) & 1, abort, p.err));
            pv = true;
            tc_fence_after();
            if (!dead) {
#pragma unroll 1
              for (int r = 0; r < R; r += 4) {
                const int row = row_of(r);
                if (row >= rows) break;
                uint32_t o[4];
                tmem_ld4_async(s_at + (kColO - kColS) + row, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sh->alpha[grp][row + e]);
                tmem_st4_async(s_at + (kColO - kColS) + row, o);
              }
              tmem_wait_st();
            }
#pragma unroll
            for (int r = 0; r < R; r += 2) {
              if (row_of(r) < rows) {
                const float2 a = *reinterpret_cast<const float2*>(&sh->alpha[grp][row_of(r)]);
                l[r / 2].x *= a.x;
                l[r / 2].y *= a.y;
              }
            }
          }
        }
        if (stop) break;
        tc_fence_before();
        if (lane == 0) mbar_arrive(&sh->s_free[grp]);
        // P = 2^s, and its sums
        if (!pv) dead = !__all_sync(0xffffffffu, mbar_wait_tested(&sh->pv_done[grp], (u - 1) & 1, abort, p.err));
        auto weigh4 = [&](int r) {                         // four rows' weights, as fp16
          const float2 a = make_float2(ex2_approx(__uint_as_float(s[r])), ex2_approx(__uint_as_float(s[r + 1])));
          const float2 b = make_float2(ex2_approx(__uint_as_float(s[r + 2])), ex2_approx(__uint_as_float(s[r + 3])));
          l[r / 2] = add_f32x2(l[r / 2], a);
          l[r / 2 + 1] = add_f32x2(l[r / 2 + 1], b);
          return make_uint2(pack_f16(a.x, a.y), pack_f16(b.x, b.y));
        };
        // (eight rows are a 16-byte word of the key's; 64 rows a box)
#pragma unroll
        for (int r = 0; r < R / 8 * 8; r += 8) {
          const uint2 a = weigh4(r), b = weigh4(r + 4);
          sts_u4(prow ^ (r << 2), make_uint4(a.x, a.y, b.x, b.y));
        }
        if constexpr (R % 8 != 0) sts_u2((prow ^ (half << 4)) + C::kBoxBytes + half * 8, weigh4(32));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !dead) mbar_arrive(&sh->p_ready[grp]);
      }
    };
    if (w.rows <= 32)
      tiles(std::integral_constant<int, 16>());
    else
      tiles(std::integral_constant<int, kRowsT>());
    // ---- epilogue: the groups' sums and O merged into the split's partial (m, l, O not normalised) ----
    const int4 gm = sh->geom[grp];
    const int b = sh->seq[grp];
    if (u > 0 && !dead) dead = !__all_sync(0xffffffffu, mbar_wait(&sh->pv_done[grp], (u - 1) & 1, abort, p.err));
#pragma unroll
    for (int r = 0; r < kRowsT; r += 4) {
      if (row_of(r) < gm.w) {
        const float sum = sum_rows4(&l[r / 2], lane);
        if (lane < 4) sh->part[grp][wq][row_of(r) + lane] = sum;
      }
    }
    tc_fence_before();
    named_sync(1, kAll);
    tc_fence_after();
    if (static_cast<int>(threadIdx.x) < gm.w) {
      const int r = threadIdx.x;
      float lg[2], ref[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        lg[g] = (sh->part[g][0][r] + sh->part[g][1][r]) + (sh->part[g][2][r] + sh->part[g][3][r]);
        ref[g] = lg[g] > 0.f ? -sh->neg_ref[g][r] : -INFINITY;
      }
      const float m = fmaxf(ref[0], ref[1]);
      float wt[2], sum = 0.f;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        wt[g] = lg[g] > 0.f ? ex2_approx(ref[g] - m) : 0.f;
        sum += wt[g] * lg[g];
      }
      const int e = partial_exponent(sum, p.v_scale);
      const float down = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int g = 0; g < 2; ++g) sh->alpha[g][r] = wt[g] * down * p.v_scale;
      const int rg = gm.z + r;
      const size_t pidx = ((static_cast<size_t>(b) * p.row_tiles + rg / kMaxRows) * p.hkv + blockIdx.y) * p.num_splits + blockIdx.x;
      reinterpret_cast<float2*>(p.part_ml)[pidx * kMaxRows + rg % kMaxRows] = make_float2(m + static_cast<float>(e), sum * down);
    }
    named_sync(1, kAll);
    if (w.nt > 0 && wq * 32 < HD) {
      // lane = channel: 32 neighbouring channels of a row are one 128-byte store. The warpgroups take rows of eight in turn.
#pragma unroll 1
      for (int r0 = (warp >> 2) * 8; r0 < gm.w; r0 += 32) {
        uint32_t o0[8], o1[8];
        tmem_ld8(lane_base + kColO + r0, o0);
        tmem_ld8(lane_base + kColO + kN + r0, o1);
        const int rg = gm.z + r0;                      // (a multiple of 8: the eight lie in one of the combine's tiles)
        float* dst = p.part_o +
                     ((((static_cast<size_t>(b) * p.row_tiles + rg / kMaxRows) * p.hkv + blockIdx.y) * p.num_splits + blockIdx.x) * kMaxRows +
                      rg % kMaxRows) * HD + wq * 32 + lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (r0 + e < gm.w) {
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

template <int HD>
cudaError_t launch_hd(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  static size_t done[64] = {};
  static bool registers = false;
  auto kern = attend_packed_kernel<HD>;
  if (!registers) {
    // The warpgroups trade registers; a kernel launched with fewer than they take up would wait for ever.
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    if (a.numRegs < kRegsLaunch) return cudaErrorNotSupported;
    registers = true;
  }
  const cudaError_t e = ensure_smem_limit(kern, Cfg<HD>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.num_splits, p.hkv, num_seqs * p.n_tiles);
  return launch_pdl(kern, grid, dim3(kThreads), Cfg<HD>::kSmemBytes, stream, p);
}

}  // namespace

int packed_tile_rows() { return kMaxN; }

cudaError_t launch_attend_packed(const PackedAttnParams& p, int num_seqs, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_hd<128>(p, num_seqs, stream) : launch_hd<64>(p, num_seqs, stream);
}

}  // namespace vfy
