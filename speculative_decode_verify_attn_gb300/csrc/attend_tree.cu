// Tree attention of full layers for large blocks: split-KV flash-decode with 256 block rows per CTA.
//
// A tree of more than 128 / G nodes has more rows per KV head than one M = 128 MMA holds. Here one CTA
// takes two row tiles of 128 (a pair), so that every K/V byte that reaches shared memory serves 256 rows:
// with d = 128 a 128-key tile is 64 KB for 4 * 128 * 128 * 128 multiply-adds, 1.4 us of one SM's HBM share
// and 1.1 us of its tensor core -- the two bounds meet.
//
// The work is one list of tiles: item (sequence b, KV head h, pair t) has T_b tiles of two resident chunks
// each, and the persistent CTAs cut the list of all items' tiles into equal runs. So a ragged batch is as
// balanced as one sequence, whatever the lengths. A CTA's run is a sequence of segments, each inside one
// item; a segment that covers its item writes O and the LSE itself, others write fp32 partials (m, l,
// unnormalised O) that the combine kernel merges:
//     O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  LSE = ln2 * (M + log2 sum_s 2^(m_s - M) l_s)
// A run has at most two partial segments, its first and its last: 2 slots per CTA.
//
// Warps: 0-3 softmax and epilogue of row tile 0, 4-7 of row tile 1 (TMEM lane = row, one thread per row),
// 8 K producer and tile geometry, 9 V producer, 10 and 11 MMA issuers, one per row tile. A tile's two chunks
// are two steps. Tensor memory per row tile: two S buffers of 64 columns (P, bf16, over the first half of its
// S) and O. S of step s+1 is issued before PV of step s, so the tensor core works on one step while the
// softmax works on the other, and the two row tiles run free of each other. An MMA costs its issuer 50 to 110
// cycles beside busy softmax warps, more than its 32 or 64 cycles in the tensor pipe: hence two issuers. In a
// segment of at most 128 rows the second row tile's warps only keep the barrier protocol, so that every role
// sees every phase of every barrier it waits on.
#include <cuda_bf16.h>

#include <type_traits>

#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 384;
constexpr int kKWarp = 8;
constexpr int kVWarp = 9;
constexpr int kMmaWarp = 10;              // and 11
constexpr int kVRelayWarp = 3;            // softmax warp of a row tile whose P arrival waits for V
constexpr int kPairRows = 2 * kMaxRows;
constexpr int kKeys = 2 * kChunk;         // keys per tile
constexpr int kGeo = 8;                   // tile-geometry ring
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;             // [row tile][chunk]: S buffers of kChunk columns
constexpr uint32_t kColO = 256;           // [row tile]: O accumulators of d columns, 128 apart
constexpr int kPrefetch = 3;              // tiles prefetched into L2 beyond the shared-memory stages
// A row keeps a stale reference maximum until a tile's maximum exceeds it by this much (log2 units).
constexpr float kRescaleLog2 = 8.0f;

template <int HD>
struct Cfg {
  static constexpr int kBoxes = HD / 64;                // 128-byte (64-column) boxes per row
  static constexpr int kBoxBytes = kKeys * 128;
  static constexpr int kChunkRowsBytes = kChunk * 128;  // one chunk's rows within a box
  static constexpr int kChunkBytes = kChunk * HD * 2;
  static constexpr int kTileBytes = kKeys * HD * 2;
  static constexpr int kQBoxBytes = kMaxRows * 128;
  static constexpr int kQTileBytes = kMaxRows * HD * 2;
  // A K stage frees as soon as both row tiles' S have read it, a V stage only after their last PV.
  static constexpr int kKStages = HD == 128 ? 2 : 4;
  static constexpr int kVStages = HD == 128 ? 3 : 4;
  static constexpr int kBarOffset = 2 * kQTileBytes + (kKStages + kVStages) * kTileBytes;
  static constexpr int kSmemBytes = kBarOffset + 2048 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static_assert(kKStages + 3 <= kGeo && kKStages <= 4 && kVStages <= 4, "rings");
};

struct Bars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t geo_full[kGeo];
  uint64_t s_full[2][2];   // [row tile][chunk], one phase per tile
  uint64_t p_full[2][2];   // [row tile][chunk]: P is written (and V has landed, its outside rows zeroed)
  uint64_t o_full[2];      // [row tile]: one phase per step, after its PV
  uint64_t o_done[2];      // [row tile]: one phase per segment with rows in it, after its last PV
  uint64_t q_ready[2];     // [row tile]: one phase per segment
  uint64_t drain[2], never;
  uint32_t tmem_base;
  int abort;
  int base[kGeo][2];       // position of each chunk's first key
  int valid[kGeo][2];
  int plain[kGeo];         // every key lies before the block: all rows attend all of them
  int zero[kGeo];          // some key lies outside the sequence: its V row is to be zeroed
};
static_assert(sizeof(Bars) <= 2048, "barrier block");

// One sequence's share of the list.
struct Seq {
  int q0, nq, L, r0, nres, rows, pairs, tiles;    // tiles of one (head, pair)
};

__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  Seq s;
  s.q0 = p.cu_q[b];
  const int q1 = p.cu_q[b + 1];
  s.L = p.seq_len[b];
  s.r0 = p.cu_res[b];
  s.nres = max(0, p.cu_res[b + 1] - s.r0);
  s.nq = q1 - s.q0;
  const bool bad = s.nq < 0 || s.nq > p.max_q || s.L < s.nq || s.q0 < 0;
  if (bad) s.nq = 0;
  s.rows = s.nq * p.group;
  s.pairs = (s.rows + kPairRows - 1) / kPairRows;
  // a sequence without a resident chunk has one tile without keys, which writes its empty rows
  s.tiles = s.rows > 0 ? max(1, (s.nres + 1) / 2) : 0;
  return s;
}
__device__ __forceinline__ bool seq_is_bad(const AttnParams& p, int b) {
  const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0;
  return nq < 0 || nq > p.max_q || p.seq_len[b] < nq || q0 < 0;
}

// Tiles of all sequences, and where tile x lies: its sequence and the tiles before that sequence. Every
// lane of the warp takes part (32 sequences a round).
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ long long seq_work(const AttnParams& p, int b) {
  if (b >= p.num_seqs) return 0;
  const Seq s = load_seq(p, b);
  return static_cast<long long>(s.tiles) * s.pairs * p.hkv;
}
__device__ __forceinline__ long long total_work(const AttnParams& p, int lane) {
  long long total = 0;
  for (int b0 = 0; b0 < p.num_seqs; b0 += 32)
    total += __shfl_sync(0xffffffffu, warp_scan(seq_work(p, b0 + lane), lane), 31);
  return total;
}
// (x below the total)
__device__ __forceinline__ void locate(const AttnParams& p, int lane, long long x, int* b, long long* before) {
  long long done = 0;
  for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
    const long long w = seq_work(p, b0 + lane), incl = done + warp_scan(w, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, incl > x);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      *b = b0 + l;
      *before = __shfl_sync(0xffffffffu, incl - w, l);
      return;
    }
    done = __shfl_sync(0xffffffffu, incl, 31);
  }
  *b = p.num_seqs;
  *before = done;
}
// Runs that the list is cut into: no run is empty, so that an item's pieces are those of all CTAs between its ends.
__device__ __forceinline__ int runs_of(long long total, int ctas) {
  return total < ctas ? static_cast<int>(total) : ctas;
}
__device__ __forceinline__ long long run_start(long long total, int cta, int ctas) { return total * cta / ctas; }
// the CTA whose run holds tile x
__device__ __forceinline__ int cta_of(long long total, long long x, int ctas) {
  return static_cast<int>(((x + 1) * ctas - 1) / total);
}

// A CTA's walk over its run: every role takes the same steps.
struct Walk {
  Seq s;
  int b, h, t, k;          // item and first tile of the segment
  int nt;                  // tiles of the segment
  int index;               // segment number
  long long left;          // tiles of the run from this segment on

  __device__ __forceinline__ void begin(const AttnParams& p, int lane, int cta, int ctas) {
    const long long total = total_work(p, lane);
    ctas = runs_of(total, ctas);
    index = 0;
    nt = 0;
    b = h = t = k = 0;
    left = 0;
    if (cta >= ctas) return;
    const long long x0 = run_start(total, cta, ctas);
    left = run_start(total, cta + 1, ctas) - x0;
    long long before;
    locate(p, lane, x0, &b, &before);
    s = load_seq(p, b);
    const long long x = x0 - before;
    const int item = static_cast<int>(x / s.tiles);
    k = static_cast<int>(x - static_cast<long long>(item) * s.tiles);
    h = item / s.pairs;
    t = item - h * s.pairs;
    set();
  }
  __device__ __forceinline__ void set() { nt = static_cast<int>(min(left, static_cast<long long>(s.tiles - k))); }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const AttnParams& p) {
    left -= nt;
    ++index;
    if (left <= 0) return;
    k = 0;                                     // the segment ended its item
    if (++t == s.pairs) {
      t = 0;
      if (++h == p.hkv) {
        h = 0;
        do s = load_seq(p, ++b); while (s.tiles == 0);
      }
    }
    set();
  }
  __device__ __forceinline__ int rows() const { return min(kPairRows, s.rows - t * kPairRows); }
  __device__ __forceinline__ bool single() const { return rows() <= kMaxRows; }
  __device__ __forceinline__ bool whole() const { return k == 0 && nt == s.tiles; }
};

struct Chunk {
  int y, base;
  bool present, valid;
};
__device__ __forceinline__ Chunk chunk_at(const AttnParams& p, const Walk& w, int j, int c) {
  Chunk t;
  const int e = 2 * (w.k + j) + c;
  t.present = e < w.s.nres;
  const int cid = t.present ? p.res_ids[w.s.r0 + e] : -1;
  const int slot = t.present ? p.res_slots[w.s.r0 + e] : -1;
  t.valid = t.present && cid >= 0 && cid < (1 << 25) && slot >= 0 && slot < p.num_slots;
  t.y = (t.valid ? slot * p.hkv + w.h : w.h) * kChunk;
  t.base = t.valid ? cid * kChunk : 0;
  return t;
}

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
// Which of the 32 keys from position pos on a row attends: those before the block (p0) and the block rows
// of its mask `words`; the 32 block bits from j = pos - p0 on straddle two words.
__device__ __forceinline__ uint32_t keep32(const uint32_t* words, int pos, int p0, int L) {
  uint32_t keep = low_bits(p0 - pos);
  const int j = pos - p0;
  if (j > -32 && pos < L) {
    const int at = j >> 5;
    const uint32_t w0 = at >= 0 ? __ldg(words + at) : 0u;
    const uint32_t w1 = at + 1 < VFY_TREE_WORDS ? __ldg(words + at + 1) : 0u;
    keep |= __funnelshift_r(w0, w1, j & 31) & low_bits(L - pos);
  }
  return keep;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tree_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * C::kQTileBytes;
  uint8_t* sV = sK + C::kKStages * C::kTileBytes;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBarOffset);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == kKWarp * 32) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);       // both issuers
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 2);
    }
    for (int i = 0; i < kGeo; ++i) mbar_init(&bars->geo_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(&bars->s_full[i][k], 1);
        mbar_init(&bars->p_full[i][k], 128);
      }
      mbar_init(&bars->drain[i], 1);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->o_done[i], 1);
      mbar_init(&bars->q_ready[i], 128);
    }
    mbar_init(&bars->never, 1);
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  volatile int* abort = &bars->abort;

  pdl_launch_dependents();
  if (!p.stable_metadata) pdl_wait();
  Walk w;
  w.begin(p, lane, blockIdx.x, gridDim.x);
  if (p.stable_metadata) pdl_wait();
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.num_seqs; b += kThreads)
      if (seq_is_bad(p, b)) atomicOr(p.err, kErrDeviceInput);
  }

  if (warp == kKWarp) {
    // ------------------------------ K producer and tile geometry --------------------------------
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      uint32_t n = 0;                        // tiles so far
      bool ok = true, reported = false;
      for (; ok && w.more(); w.next(p)) {
        for (int j = 0; j < w.nt; ++j, ++n) {
          const int st = n % C::kKStages;
          if (n >= C::kKStages) ok = mbar_wait(&bars->k_empty[st], (n / C::kKStages - 1) & 1, abort, p.err);
          if (!ok) break;
          const int g = n % kGeo;
          const int p0 = w.s.L - w.s.nq;
          Chunk c[2];
          int present = 0;
          bool plain = true, zero = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            c[i] = chunk_at(p, w, j, i);
            if (c[i].present && !c[i].valid && !reported) {
              atomicOr(p.err, kErrDeviceInput);
              reported = true;
            }
            bars->base[g][i] = c[i].base;
            bars->valid[g][i] = c[i].valid ? 1 : 0;
            plain = plain && c[i].valid && c[i].base + kChunk <= p0;
            zero = zero || !c[i].valid || c[i].base + kChunk > w.s.L;
            present += c[i].present ? 1 : 0;
          }
          bars->plain[g] = plain ? 1 : 0;
          bars->zero[g] = zero ? 1 : 0;
          mbar_arrive(&bars->geo_full[g]);
          // a chunk the sequence lacks is not loaded: the mask and the zeroed V rows cover its stale rows
          mbar_arrive_expect_tx(&bars->k_full[st], present * C::kChunkBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!c[i].present) continue;
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_2d(sK + st * C::kTileBytes + bx * C::kBoxBytes + i * C::kChunkRowsBytes, &tmap_k,
                          &bars->k_full[st], bx * 64, c[i].y, pol);
          }
          // more of the stream in flight from HBM than the stages hold
          const int f = j + kPrefetch + C::kKStages - 1;
          if (f < w.nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const Chunk a = chunk_at(p, w, f, i);
              if (!a.present) continue;
#pragma unroll
              for (int bx = 0; bx < C::kBoxes; ++bx) {
                tma_prefetch_2d(&tmap_k, bx * 64, a.y);
                tma_prefetch_2d(&tmap_v, bx * 64, a.y);
              }
            }
          }
        }
      }
      // every copy lands before the CTA can exit, also when the pipeline was aborted
      for (uint32_t i = n > C::kKStages ? n - C::kKStages : 0; i < n; ++i)
        mbar_drain(&bars->k_full[i % C::kKStages], (i / C::kKStages) & 1, p.err);
    }
  } else if (warp == kVWarp) {
    // ------------------------------ V producer --------------------------------------------------
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      uint32_t n = 0;
      bool ok = true;
      for (; ok && w.more(); w.next(p)) {
        for (int j = 0; j < w.nt; ++j, ++n) {
          const int st = n % C::kVStages;
          if (n >= C::kVStages) ok = mbar_wait(&bars->v_empty[st], (n / C::kVStages - 1) & 1, abort, p.err);
          if (!ok) break;
          Chunk c[2];
          int present = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            c[i] = chunk_at(p, w, j, i);
            present += c[i].present ? 1 : 0;
          }
          mbar_arrive_expect_tx(&bars->v_full[st], present * C::kChunkBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!c[i].present) continue;
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_2d(sV + st * C::kTileBytes + bx * C::kBoxBytes + i * C::kChunkRowsBytes, &tmap_v,
                          &bars->v_full[st], bx * 64, c[i].y, pol);
          }
        }
      }
      for (uint32_t i = n > C::kVStages ? n - C::kVStages : 0; i < n; ++i)
        mbar_drain(&bars->v_full[i % C::kVStages], (i / C::kVStages) & 1, p.err);
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------ MMA issuers (one lane each) ---------------------------------
    if (lane == 0) {
      const int h = warp - kMmaWarp;         // row tile
      if (h == 0 && p.timeout_test_ns != 0) mbar_wait_limit(&bars->never, 0, p.timeout_test_ns, abort, p.err);
      bool ok = !*abort;
      const uint32_t idesc_s = idesc_bf16_f32(128, kChunk, 0, 0);
      const uint32_t idesc_pv = idesc_bf16_f32(128, HD, 0, 1);
      const uint64_t qd = sw128_desc(smem_u32(sQ + h * C::kQTileBytes), 16, 1024);
      const uint64_t kd = sw128_desc(smem_u32(sK), 16, 1024);
      const uint64_t vd = sw128_desc(smem_u32(sV), C::kBoxBytes, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(qd), q_hi = static_cast<uint32_t>(qd >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(kd), k_hi = static_cast<uint32_t>(kd >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(vd), v_hi = static_cast<uint32_t>(vd >> 32);
      const uint32_t col_s = tbase + kColS + h * 128, col_o = tbase + kColO + h * 128;
      uint32_t n = 0;                        // tiles of the run before the segment's
      uint32_t segs = 0;                     // segments so far
      for (; ok && w.more(); w.next(p)) {
        const bool idle = h == 1 && w.single();      // no rows here: the barriers only
        // S of step s: chunk s & 1 of tile n + s / 2; with a tile's second chunk its K stage is read
        auto issue_s = [&](int s) {
          const uint32_t st = (n + (s >> 1)) % C::kKStages;
          if (idle) {
            mbar_arrive(&bars->s_full[h][s & 1]);
            if (s & 1) mbar_arrive(&bars->k_empty[st]);
            return;
          }
          const uint32_t k0 = k_lo + ((st * C::kTileBytes + (s & 1) * C::kChunkRowsBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_ss_lo(col_s + (s & 1) * kChunk, q_lo + (((kk >> 2) * C::kQBoxBytes + (kk & 3) * 32) >> 4), q_hi,
                      k0 + (((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4), k_hi, idesc_s, kk > 0 ? 1u : 0u);
          mma_commit(&bars->s_full[h][s & 1]);
          if (s & 1) mma_commit(&bars->k_empty[st]);
        };
        auto wait_k = [&](uint32_t i) {
          const bool got = mbar_wait(&bars->k_full[i % C::kKStages], (i / C::kKStages) & 1, abort, p.err);
          tc_fence_after();
          return got;
        };
        const int ns = 2 * w.nt;
        ok = mbar_wait(&bars->q_ready[h], segs++ & 1, abort, p.err) && wait_k(n);
        if (!ok) break;
        issue_s(0);
        for (int s = 0; s < ns; ++s) {
          if (s + 1 < ns) {
            if (s & 1) ok = wait_k(n + ((s + 1) >> 1));
            if (!ok) break;
            issue_s(s + 1);
          }
          const int c = s & 1;
          const uint32_t i = n + (s >> 1), st = i % C::kVStages;
          ok = mbar_wait(&bars->p_full[h][c], i & 1, abort, p.err);
          // (an idle row tile gives a V stage back once per load too, as its PV would)
          if (idle && c == 1) ok = ok && mbar_wait(&bars->v_full[st], (i / C::kVStages) & 1, abort, p.err);
          if (!ok) break;
          if (idle) {
            mbar_arrive(&bars->o_full[h]);
            if (c == 1) mbar_arrive(&bars->v_empty[st]);
            continue;
          }
          tc_fence_after();
          const uint32_t v0 = v_lo + ((st * C::kTileBytes + c * C::kChunkRowsBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk)
            mma_ts_lo(col_o, col_s + c * kChunk + kk * 8, v0 + ((16 * kk * 128) >> 4), v_hi, idesc_pv,
                      (s > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&bars->o_full[h]);
          if (c == 1) mma_commit(&bars->v_empty[st]);
          if (s + 1 == ns) mma_commit(&bars->o_done[h]);
        }
        n += w.nt;
      }
      // every MMA completes before TMEM is freed
      mma_commit(&bars->drain[h]);
      mbar_drain(&bars->drain[h], 0, p.err);
    }
    __syncwarp();
  } else {
    // ------------------------------ softmax / epilogue ------------------------------------------
    const int h = warp >> 2;                           // row tile
    const int lr = (warp & 3) * 32 + lane;             // row of the tile and TMEM lane
    const uint32_t lane_base = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const unsigned ug = static_cast<unsigned>(p.group);
    uint8_t* sq = sQ + h * C::kQTileBytes;
    bool ok = true;
    uint32_t n = 0;                                    // tiles before this segment
    // Q of a segment's row tile -> shared memory, in the 128-byte swizzle
    auto stage_q = [&](const Walk& v) {
      const int r = h * kMaxRows + lr;
      const bool rv = r < v.rows();
      const unsigned br = static_cast<unsigned>(v.t * kPairRows + (rv ? r : 0));
      const unsigned qi = br / ug, g = br - qi * ug;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<size_t>(v.s.q0 + qi) * p.hq + static_cast<size_t>(v.h) * p.group + g) * HD);
#pragma unroll
      for (int half = 0; half < HD / 64; ++half) {
        uint4 x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = rv ? __ldg(src + half * 8 + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(sq + half * C::kQBoxBytes + lr * 128 + ((c ^ (lr & 7)) << 4)) = x[c];
      }
      fence_proxy_async_smem();
    };
    uint32_t segs = 0;                                 // segments with rows in this tile
    if (w.more()) {
      if (h == 0 || !w.single()) stage_q(w);
      mbar_arrive(&bars->q_ready[h]);
    }
    while (ok && w.more()) {
      const bool idle = h == 1 && w.single();
      const int r = h * kMaxRows + lr;
      const bool rv = r < w.rows();
      const bool active = __any_sync(0xffffffffu, rv);
      const unsigned br = static_cast<unsigned>(w.t * kPairRows + (rv ? r : 0));
      const unsigned qi = br / ug;
      const int p0 = w.s.L - w.s.nq;
      const uint32_t* words = p.tree_mask + static_cast<size_t>(w.s.q0 + qi) * VFY_TREE_WORDS;
      float m_ref = -INFINITY, l = 0.f;
      const int ns = 2 * w.nt;
      bool plain = true, zero = false;                 // of the tile
      for (int s = 0; s < ns; ++s) {
        const int j = s >> 1, c = s & 1;
        const uint32_t i = n + j;
        const int gs = i % kGeo;
        if (c == 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->geo_full[gs], (i / kGeo) & 1, abort, p.err));
          if (!ok) break;
          plain = bars->plain[gs] != 0;
          zero = bars->zero[gs] != 0;
        }
        uint32_t keep[2] = {0u, 0u};
        if (!plain && bars->valid[gs][c] != 0 && rv) {
          keep[0] = keep32(words, bars->base[gs][c], p0, w.s.L);
          keep[1] = keep32(words, bars->base[gs][c] + 32, p0, w.s.L);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[h][c], i & 1, abort, p.err));
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const uint32_t ts = lane_base + kColS + h * 128 + c * kChunk;
          float sv[kChunk];
          {
            uint32_t sr[kChunk];
            tmem_ld64(ts, sr);
#pragma unroll
            for (int e = 0; e < kChunk; ++e) sv[e] = __uint_as_float(sr[e]);
          }
          if (!plain) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e) sv[e] = (keep[e >> 5] >> (e & 31)) & 1u ? sv[e] : -INFINITY;
          }
          float mx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = sv[e];
#pragma unroll
          for (int e = 8; e < kChunk; ++e) mx[e & 7] = fmaxf(mx[e & 7], sv[e]);
          const float m_tile = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                     fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * p.scale_log2;
          const bool raise = m_tile > m_ref + kRescaleLog2;
          const bool scale_o = raise && m_ref != -INFINITY;
          float alpha = 1.f;
          if (raise) {
            alpha = ex2_approx(m_ref - m_tile);        // 0 where m_ref = -inf
            l *= alpha;
            m_ref = m_tile;
          }
          if (__any_sync(0xffffffffu, scale_o)) {
            // O holds the steps before s. PV(s-2) was issued before S(s) and PV(s) needs this step's P: the
            // barrier of PV(s-1) is in that phase or the one after.
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_full[h], (2 * n + s - 1) & 1, abort, p.err));
            if (!ok) break;
            tc_fence_after();
            const float a = scale_o ? alpha : 1.f;
#pragma unroll 1
            for (int x = 0; x < HD / 32; ++x) {
              uint32_t o[32];
              tmem_ld32(lane_base + kColO + h * 128 + x * 32, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st32(lane_base + kColO + h * 128 + x * 32, o);
            }
          }
          // p = 2^(s * scale * log2e - m_ref), packed over the first half of this S
          const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
          const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), neg2 = make_float2(neg, neg);
          float2 ps[4];
          uint32_t pk[kChunk / 2];
#pragma unroll
          for (int e = 0; e < kChunk / 2; ++e) {
            float2 x = fma_f32x2(make_float2(sv[2 * e], sv[2 * e + 1]), scale2, neg2);
            x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            ps[e & 3] = e < 4 ? x : add_f32x2(ps[e & 3], x);
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(x.x, x.y);
            pk[e] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          const float2 sum = add_f32x2(add_f32x2(ps[0], ps[1]), add_f32x2(ps[2], ps[3]));
          l += sum.x + sum.y;
          tmem_st32(ts, pk);
        }
        tc_fence_before();
        // One warp's arrival waits for the tile's V, so the issuer's wait for P covers V too.
        if (!idle && (zero || ((warp & 3) == kVRelayWarp && c == 0))) {
          const int sv = i % C::kVStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[sv], (i / C::kVStages) & 1, abort, p.err));
          if (!ok) break;
          if (zero) {
            // V rows of keys outside the sequence may hold anything, and 0 * NaN is NaN on the tensor core. Both
            // row tiles zero them (the same zeros), each before its own P.
            const int key = lr >> 1;                   // two threads per key
            if (bars->valid[gs][c] == 0 || bars->base[gs][c] + key >= w.s.L) {
              uint8_t* row = sV + sv * C::kTileBytes + c * C::kChunkRowsBytes + key * 128;
#pragma unroll
              for (int x = (lr & 1) * C::kBoxes * 4; x < ((lr & 1) + 1) * C::kBoxes * 4; ++x)
                *reinterpret_cast<uint4*>(row + (x >> 3) * C::kBoxBytes + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        mbar_arrive(&bars->p_full[h][c]);
      }
      if (!ok) break;
      // the next segment's first S may run during this one's epilogue: every S here has read Q
      Walk nx = w;
      nx.next(p);
      if (nx.more()) {
        if (h == 0 || !nx.single()) stage_q(nx);
        mbar_arrive(&bars->q_ready[h]);
      }
      if (idle) {
        n += w.nt;
        w = nx;
        continue;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_done[h], segs++ & 1, abort, p.err));
      if (!ok) break;
      tc_fence_after();
      if (active) {
        const uint32_t to = lane_base + kColO + h * 128;
        if (w.whole()) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const int t = w.s.q0 + static_cast<int>(qi);
          const int hq = w.h * p.group + static_cast<int>(br - qi * ug);
          const bool wr = rv && t < p.token_cap;
          uint16_t* dst = p.out + (static_cast<size_t>(wr ? t : 0) * p.hq + hq) * HD;
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
            if (!wr) continue;
            uint32_t out[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float a = l > 0.f ? __uint_as_float(o[2 * e]) * inv : 0.f;
              const float b = l > 0.f ? __uint_as_float(o[2 * e + 1]) * inv : 0.f;
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
              out[e] = *reinterpret_cast<const uint32_t*>(&h2);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(dst + c * 32 + 2 * e) = make_uint4(out[e], out[e + 1], out[e + 2], out[e + 3]);
          }
          if (wr && p.lse != nullptr)
            p.lse[static_cast<size_t>(t) * p.hq + hq] = l > 0.f ? (m_ref + __log2f(l)) * 0.6931471805599453f : -INFINITY;
        } else {
          const size_t at = (2 * static_cast<size_t>(blockIdx.x) + (w.index > 0 ? 1 : 0)) * kPairRows + r;
          float* dst = p.part_o + at * HD;
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + c * 32, o);
            if (!rv || !(l > 0.f)) continue;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(dst + c * 32 + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          if (rv) reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(l > 0.f ? m_ref : -INFINITY, l);
        }
      }
      tc_fence_before();
      n += w.nt;
      w = nx;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// ------------------------------ merge of the partial segments ------------------------------------
// One 128-thread CTA per output row. Its item's tiles lie in the runs of CTAs c0 .. c1; if that is one CTA,
// it wrote the row itself. Otherwise warp x takes pieces c0 + x, c0 + x + 4, ... eight at a time, and the
// four warps' sums meet in shared memory.
constexpr int kAhead = 8;

template <int HD>
__global__ void __launch_bounds__(128) combine_tree_kernel(const AttnParams p, int ctas) {
  constexpr int kPer = HD / 32;
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  __shared__ float s_m[4], s_l[4], s_acc[4][HD];
  pdl_launch_dependents();
  if (!p.stable_metadata) pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = static_cast<int>(blockIdx.x / p.hq);
  const int hq = static_cast<int>(blockIdx.x % p.hq);
  const int tokens = p.cu_q[p.num_seqs];
  long long total = 0, before = 0;             // tiles of all sequences, of those before the row's
  int b = -1;
  for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
    const int mine = b0 + lane;
    const long long work = seq_work(p, mine);
    const long long incl = total + warp_scan(work, lane);
    const bool here = mine < p.num_seqs && p.cu_q[mine] <= t && t < p.cu_q[mine + 1];
    const unsigned hit = __ballot_sync(0xffffffffu, here);
    if (hit != 0u && b < 0) {
      const int l = __ffs(hit) - 1;
      b = b0 + l;
      before = __shfl_sync(0xffffffffu, incl - work, l);
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }
  if (p.stable_metadata) pdl_wait();
  if (b < 0 || t >= tokens || t >= p.token_cap) return;
  const Seq s = load_seq(p, b);
  if (s.tiles == 0) return;
  const int h = hq / p.group;
  const int br = (t - s.q0) * p.group + (hq - h * p.group);
  const int pair = br / kPairRows, r = br - pair * kPairRows;
  ctas = runs_of(total, ctas);
  const long long x0 = before + (static_cast<long long>(h) * s.pairs + pair) * s.tiles;
  const int c0 = cta_of(total, x0, ctas), c1 = cta_of(total, x0 + s.tiles - 1, ctas);
  if (c0 == c1) return;
  const bool c0_first = run_start(total, c0, ctas) == x0;      // the item opens c0's run
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int c = c0 + warp; c <= c1; c += 4 * kAhead) {
    float2 a[kAhead];
    Vec v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int x = min(c + 4 * u, c1);
      const size_t at = (2 * static_cast<size_t>(x) + (x == c0 && !c0_first ? 1 : 0)) * kPairRows + r;
      a[u] = __ldcg(ml + at);
      v[u] = __ldcg(reinterpret_cast<const Vec*>(p.part_o + at * HD) + lane);
      if (c + 4 * u > c1) a[u] = make_float2(-INFINITY, 0.f);
    }
    float mm = m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) mm = a[u].y > 0.f ? fmaxf(mm, a[u].x) : mm;
    const float old = l > 0.f ? ex2_approx(m - mm) : 0.f;
    l *= old;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= old;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      // a piece without a key for this row holds no O: its zero weight selects it out
      const bool use = a[u].y > 0.f;
      const float wgt = use ? ex2_approx(a[u].x - mm) : 0.f;
      l = use ? fmaf(wgt, a[u].y, l) : l;
      const float* f = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = use ? fmaf(wgt, f[e], acc[e]) : acc[e];
    }
    m = mm;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_acc[warp][lane * kPer + e] = acc[e];
  __syncthreads();
  if (warp != 0) return;
  float mmax = -INFINITY;
#pragma unroll
  for (int x = 0; x < 4; ++x) mmax = s_l[x] > 0.f ? fmaxf(mmax, s_m[x]) : mmax;
  float sc[4], lsum = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    sc[x] = s_l[x] > 0.f ? ex2_approx(s_m[x] - mmax) : 0.f;
    lsum += sc[x] * s_l[x];
  }
  const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
  uint32_t o[kPer / 2];
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) {
    float a = 0.f, c = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      a = fmaf(sc[x], s_acc[x][lane * kPer + 2 * e], a);
      c = fmaf(sc[x], s_acc[x][lane * kPer + 2 * e + 1], c);
    }
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(a * inv, c * inv);
    o[e] = *reinterpret_cast<const uint32_t*>(&h2);
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (static_cast<size_t>(t) * p.hq + hq) * HD) + lane * (kPer / 2);
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) dst[e] = o[e];
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<size_t>(t) * p.hq + hq] = lsum > 0.f ? (mmax + __log2f(lsum)) * 0.6931471805599453f : -INFINITY;
}

template <int HD>
cudaError_t launch_hd(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int ctas,
                      cudaStream_t stream) {
  static size_t done[64] = {};
  auto kern = attend_tree_kernel<HD>;
  cudaError_t e = ensure_smem_limit(kern, Cfg<HD>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(ctas), dim3(kThreads), Cfg<HD>::kSmemBytes, stream, p, tk, tv);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.token_cap) * p.hq;
  return launch_pdl(combine_tree_kernel<HD>, dim3(static_cast<unsigned>(rows)), dim3(128), 0, stream, p, ctas);
}

}  // namespace

cudaError_t launch_attend_tree(int head_dim, const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               int ctas, cudaStream_t stream) {
  return head_dim == 128 ? launch_hd<128>(p, tk, tv, ctas, stream) : launch_hd<64>(p, tk, tv, ctas, stream);
}

}  // namespace vfy
