// Tree attention of full layers for large blocks (d = 128): split-KV flash-decode with 256 block rows per
// CTA pair.
//
// A tree of more than 128 / G nodes has more rows per KV head than one M = 128 MMA holds. Here two CTAs of a
// cluster take two row tiles of 128, one each, as the halves of M = 256 MMAs (cta_group::2): every K/V byte is
// fetched by one of the two SMs (K: a chunk each; V: half of the columns each) and serves 256 rows.
//
// The work is one list of tiles: item (sequence b, KV head h, pair of row tiles t) has T_b tiles of two
// resident chunks each, and the persistent CTA pairs cut the list of all items' tiles into equal runs. So a
// ragged batch is as balanced as one sequence, whatever the lengths. A run is a sequence of segments, each
// inside one item; a segment that covers its item writes O and the LSE itself, others write fp32 partials
// (m, l, unnormalised O) that the combine kernel merges:
//     O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  LSE = ln2 * (M + log2 sum_s 2^(m_s - M) l_s)
// A run has at most two partial segments, its first and its last: 2 slots per pair.
//
// Warps of each CTA: 0-3 and 4-7 two softmax warpgroups (TMEM lane = row of the CTA's row tile, one thread
// per row and warpgroup), 8 K producer and tile geometry, 9 V producer; in the leading CTA 10 issues the S
// MMAs and 11 the PV MMAs. Warpgroup g takes chunk g of every tile, with a running maximum, a row sum and an
// O of its own (O_g += P_g V_g); the halves merge once, at the segment's end. S of a tile (128 columns, P as
// bf16 over the first half of each chunk's) has two buffers, so S of the next tile runs during the softmax of
// this one. An MMA costs its issuer 50 to 110 cycles beside busy softmax warps, more than the pair's 64 in the
// tensor pipes: hence two issuers (one for everything: 2360 cycles a tile, in the linear block's kernel).
//
// P is rounded to bf16 for the second MMA (half a step, 2^-8, of each weight, and O once more at the end; its sum l is
// that of the unrounded weights), as V's type asks; P in two bf16 parts would double that MMA. Against fp64 the
// outputs are off by 0.0023 of their norm, rounding O alone costs 0.0017.
//
// GB300, 4 KV heads, G = 4, one layer with its merge, replayed in a graph: 64 nodes over 4096 resident chunks (537 MB)
// 109 us, 4.9 TB/s and 1.26 PFLOP/s of full row tiles (the linear block's kernel with its best splits 146); 8 ragged
// sequences of 48 nodes up to 48K 110 us (147). Calls in a loop on the stream take 120 and 115. A tile of 128 keys
// takes a pair 1880 to 1910 cycles, of which its MMAs fill 1024 and the copies at the HBM rate would 1400: the bound is
// the loop P(n) -> PV(n) -> S(n + 2) -> P(n + 2), two tiles long, and beside it the softmax warps' own time (1160 cycles
// of a tile are arithmetic, the rest barrier operations; a wait for a phase that is complete takes 145 cycles on an idle
// SM, 70 when it is tested first, both twice that here). So every wait and index in that loop counts: rings of 4 stages
// (6 of K, or 5 of V, cost 4 to 6 us for the division), V's wait before S's, where the warp waits anyway (3 us), tests
// first, no wait for the geometry of most tiles (1 us each).
// Measured and not kept, against 117 then: P in columns of its own, so that S(n + 1) runs as soon as S(n) is loaded,
// 128 with one S buffer, 140 with two and one O for both warpgroups (which then have to agree on each row's maximum);
// one lane waiting for its warp 131; spinning without suspending 116; the issuing warp converged, with predicated
// MMAs, 119.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int HD = 128;
constexpr int kThreads = 384;
constexpr int kKWarp = 8;
constexpr int kVWarp = 9;
constexpr int kMmaWarp = 10;              // and 11
constexpr int kVRelayWarp = 3;            // softmax warp of a warpgroup whose P arrival waits for V
constexpr int kPairRows = 2 * kMaxRows;
constexpr int kKeys = 2 * kChunk;         // keys per tile
constexpr int kGeo = 16;                  // tile-geometry ring
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;             // [tile parity]: S of kKeys columns
constexpr uint32_t kColO = 256;           // [chunk]: O of 128 columns
// A row keeps a stale reference maximum until a tile's maximum exceeds it by this much (log2 units).
constexpr float kRescaleLog2 = 8.0f;

// Shared memory of one CTA: its row tile of Q; K stages of its chunk (64 keys x 128); V stages of its 64
// columns (128 keys x 64). Each is made of 128-byte rows in the 128-byte swizzle.
constexpr int kBoxBytes = kChunk * 128;               // 64 rows of 128 bytes
constexpr int kQBoxBytes = kMaxRows * 128;
constexpr int kQBytes = 2 * kQBoxBytes;
constexpr int kStageBytes = 2 * kBoxBytes;            // of K (two column boxes) and of V (two chunks)
constexpr int kKStages = 4, kVStages = 4;
constexpr int kBarOffset = kQBytes + (kKStages + kVStages) * kStageBytes;
constexpr int kBarBytes = 4096;
constexpr int kSmemBytes = kBarOffset + kBarBytes + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(kKStages + 4 <= kGeo, "geometry ring");

struct Bars {
  uint64_t k_full[kKStages];   // in the leading CTA: both CTAs' chunks
  uint64_t k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t geo_full[kGeo];
  uint64_t s_full[2], s_free[2];   // [tile parity]: S is there; its P has been read (leading CTA)
  uint64_t p_full[2];          // in the leading CTA, [tile parity]: P is written in both CTAs (and V has landed)
  uint64_t o_done;             // one phase per segment, after its last PV
  uint64_t q_ready;            // in the leading CTA, one phase per segment: Q is staged in both CTAs
  uint64_t half_ready[4];      // [lane quarter], one phase per segment: both warpgroups' (m, l)
  uint64_t o_read;             // one phase per segment: both warpgroups have read both O
  uint64_t drain[2], never;
  uint32_t tmem_base;
  int abort;
  int base[kGeo][2];           // position of each chunk's first key
  int valid[kGeo][2];
  uint32_t plain_tag[kGeo];    // tile + 1 if every key of the tile lies before the block: all rows attend them
  int zero[kGeo];              // some key lies outside the sequence: its V row is to be zeroed
  float xm[2][128], xl[2][128];
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

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
  const bool bad = s.nq < 0 || s.nq > p.max_q || s.L < s.nq || s.q0 < 0 || s.q0 > p.token_cap - s.nq;
  if (bad) s.nq = 0;
  s.rows = s.nq * p.group;
  s.pairs = (s.rows + kPairRows - 1) / kPairRows;
  // a sequence without a resident chunk has one tile without keys, which writes its empty rows
  s.tiles = s.rows > 0 ? max(1, (s.nres + 1) / 2) : 0;
  return s;
}
__device__ __forceinline__ bool seq_is_bad(const AttnParams& p, int b) {
  const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0;
  return nq < 0 || nq > p.max_q || p.seq_len[b] < nq || q0 < 0 || q0 > p.token_cap - nq;
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
  int ctas;                // runs
  long long left;          // tiles of the run from this segment on
  long long total, end;    // tiles of all runs, of the runs up to this one's end

  __device__ __forceinline__ void begin(const AttnParams& p, int lane, int cta, int pairs) {
    total = total_work(p, lane);
    ctas = runs_of(total, pairs);
    end = 0;
    index = 0;
    nt = 0;
    b = h = t = k = 0;
    left = 0;
    if (cta >= ctas) return;
    const long long x0 = run_start(total, cta, ctas);
    end = run_start(total, cta + 1, ctas);
    left = end - x0;
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
  __device__ __forceinline__ bool whole() const { return k == 0 && nt == s.tiles; }
  // the item starts here and goes on in the next run: the run that holds its last tile
  __device__ __forceinline__ bool cut() const { return k == 0 && nt < s.tiles; }
  __device__ __forceinline__ int last_cta() const { return cta_of(total, end + (s.tiles - nt) - 1, ctas); }
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

// A copy lands within microseconds; after an abort the producers keep their CTA for a thousand times that.
__device__ __forceinline__ void let_copies_land() {
  const unsigned long long t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attend_tree_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v) {
  extern __shared__ uint8_t smem_raw[];
  // (the pair's descriptors need the same offsets in both CTAs: the dynamic block starts at one address in all)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kQBytes;
  uint8_t* sV = sK + kKStages * kStageBytes;
  Bars* bars = reinterpret_cast<Bars*>(smem + kBarOffset);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
  auto leader = [&](const uint64_t* bar) { return dsmem_addr(smem_u32(bar), 0); };

  if (threadIdx.x == kKWarp * 32) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 1);
    }
    for (int i = 0; i < kGeo; ++i) mbar_init(&bars->geo_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 1);
      mbar_init(&bars->p_full[i], 16);                                   // all softmax warps, both CTAs
      mbar_init(&bars->drain[i], 1);
    }
    mbar_init(&bars->o_done, 1);
    mbar_init(&bars->q_ready, 16);                                       // all softmax warps, both CTAs
    for (int i = 0; i < 4; ++i) mbar_init(&bars->half_ready[i], 2);
    mbar_init(&bars->o_read, 8);
    mbar_init(&bars->never, 1);
    for (int i = 0; i < kGeo; ++i) bars->plain_tag[i] = 0;
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  __syncwarp();
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&bars->tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                          // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  volatile int* abort = &bars->abort;

  pdl_launch_dependents();
  if (!p.stable_metadata) pdl_wait();
  Walk w;
  w.begin(p, lane, pair, pairs);
  if (p.stable_metadata) pdl_wait();
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.num_seqs; b += kThreads)
      if (seq_is_bad(p, b)) atomicOr(p.err, kErrDeviceInput);
  }
  bool ok = true;

  if (warp == kKWarp) {
    // ------------------------------ K producer and tile geometry --------------------------------
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      uint32_t n = 0;                        // tiles so far
      bool reported = rank != 0;
      if (rank == 0) p.tree_pieces[pair].rows = 0;
      for (; ok && w.more(); w.next(p)) {
        if (rank == 0 && w.cut()) {
          TreePiece x = {};
          x.rows = w.rows();
          x.row0 = w.t * kPairRows;
          x.q0 = w.s.q0;
          x.head0 = w.h * p.group;
          x.slot = 2 * pair + (w.index > 0 ? 1 : 0);
          x.last = w.last_cta();
          p.tree_pieces[pair] = x;
        }
        for (int j = 0; j < w.nt; ++j, ++n) {
          const int st = n % kKStages;
          Chunk c[2] = {chunk_at(p, w, j, 0), chunk_at(p, w, j, 1)};       // (read while the stage empties)
          if (n >= kKStages) ok = mbar_wait(&bars->k_empty[st], (n / kKStages - 1) & 1, abort, p.err);
          if (!ok) break;
          const int g = n % kGeo;
          const int p0 = w.s.L - w.s.nq;
          int present = 0;
          bool plain = true, zero = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (c[i].present && !c[i].valid && !reported) {
              atomicOr(p.err, kErrDeviceInput);
              reported = true;
            }
            bars->base[g][i] = c[i].base;
            bars->valid[g][i] = c[i].valid ? 1 : 0;
            // (the last chunk ends at 2^31: no sums with its base)
            plain = plain && c[i].valid && c[i].base <= p0 - kChunk;
            zero = zero || !c[i].valid || c[i].base > w.s.L - kChunk;
            present += c[i].present ? 1 : 0;
          }
          bars->zero[g] = zero ? 1 : 0;
          if (plain) *reinterpret_cast<volatile uint32_t*>(&bars->plain_tag[g]) = n + 1;
          mbar_arrive(&bars->geo_full[g]);
          // a chunk the sequence lacks is not loaded: the mask and the zeroed V rows cover its stale rows
          if (rank == 0) mbar_arrive_expect_tx(&bars->k_full[st], present * kStageBytes);
          const Chunk mine = rank == 0 ? c[0] : c[1];
          if (mine.present) {
#pragma unroll
            for (int bx = 0; bx < 2; ++bx)
              tma_load_2d_pair(sK + st * kStageBytes + bx * kBoxBytes, &tmap_k, leader(&bars->k_full[st]), bx * 64,
                               mine.y, pol);
          }
        }
      }
      // Every copy has been read when the run ends as it should. After a wait that ran out, copies of either CTA
      // may be in flight, and the leading CTA's barriers count both CTAs': they get time to land.
      if (!ok) let_copies_land();
    }
  } else if (warp == kVWarp) {
    // ------------------------------ V producer --------------------------------------------------
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      uint32_t n = 0;
      for (; ok && w.more(); w.next(p)) {
        for (int j = 0; j < w.nt; ++j, ++n) {
          const int st = n % kVStages;
          Chunk c[2] = {chunk_at(p, w, j, 0), chunk_at(p, w, j, 1)};
          if (n >= kVStages) ok = mbar_wait(&bars->v_empty[st], (n / kVStages - 1) & 1, abort, p.err);
          if (!ok) break;
          const int present = (c[0].present ? 1 : 0) + (c[1].present ? 1 : 0);
          mbar_arrive_expect_tx(&bars->v_full[st], present * kBoxBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (c[i].present)
              tma_load_2d(sV + st * kStageBytes + i * kBoxBytes, &tmap_v, &bars->v_full[st], rank * 64, c[i].y, pol);
        }
      }
      if (!ok) let_copies_land();
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------ MMA issuers (one lane each, leading CTA) --------------------
    if (lane == 0 && rank == 0) {
      const bool s_issuer = warp == kMmaWarp;
      if (p.timeout_test_ns != 0) mbar_wait_limit(&bars->never, 0, p.timeout_test_ns, abort, p.err);
      ok = !*abort;
      uint32_t n = 0, segs = 0;              // tiles and segments so far
      if (s_issuer) {
        const uint32_t idesc = idesc_bf16_f32(256, kKeys, 0, 0);
        const uint64_t qdesc = sw128_desc(smem_u32(sQ), 16, 1024);
        const uint64_t kdesc = sw128_desc(smem_u32(sK), 16, 1024);
        for (; ok && w.more(); w.next(p)) {
          ok = mbar_wait(&bars->q_ready, segs++ & 1, abort, p.err);
          for (int j = 0; ok && j < w.nt; ++j, ++n) {
            const uint32_t ks = n % kKStages, sb = n & 1;
            ok = mbar_wait_tested(&bars->k_full[ks], (n / kKStages) & 1, abort, p.err);
            if (n >= 2)
              ok = ok && mbar_wait_tested(&bars->s_free[sb], ((n >> 1) - 1) & 1, abort, p.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              mma_ss_pair(tbase + kColS + sb * kKeys,
                          qdesc + static_cast<uint64_t>(((kk >> 2) * kQBoxBytes + (kk & 3) * 32) >> 4),
                          kdesc + ((ks * kStageBytes + (kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4),
                          idesc, kk > 0 ? 1u : 0u);
            mma_commit_pair(&bars->s_full[sb]);
            mma_commit_pair(&bars->k_empty[ks]);
          }
        }
      } else {
        const uint32_t idesc = idesc_bf16_f32(256, HD, 0, 1);
        const uint64_t vdesc = sw128_desc(smem_u32(sV), kStageBytes, 1024);
        for (; ok && w.more(); w.next(p)) {
          for (int j = 0; j < w.nt; ++j, ++n) {
            const uint32_t vs = n % kVStages, sb = n & 1;
            ok = mbar_wait_tested(&bars->p_full[sb], (n >> 1) & 1, abort, p.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int kk = 0; kk < kChunk / 16; ++kk)
                mma_ts_pair(tbase + kColO + c * 128, tbase + kColS + sb * kKeys + c * kChunk + kk * 8,
                            vdesc + ((vs * kStageBytes + c * kBoxBytes + 16 * kk * 128) >> 4), idesc,
                            (j > 0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(&bars->s_free[sb]);
            mma_commit_pair(&bars->v_empty[vs]);
            if (j == w.nt - 1) mma_commit_pair(&bars->o_done);
          }
        }
      }
      // every MMA completes before TMEM is freed
      mma_commit_pair(&bars->drain[warp - kMmaWarp]);
      mbar_drain(&bars->drain[warp - kMmaWarp], 0, p.err);
    }
    __syncwarp();
  } else {
    // ------------------------------ softmax / epilogue ------------------------------------------
    const int g = warp >> 2;                           // warpgroup: its chunk of every tile
    const int quarter = warp & 3;
    const int lr = quarter * 32 + lane;                // row of the CTA's row tile and TMEM lane
    const int r = rank * kMaxRows + lr;                // row of the pair
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
    const unsigned ug = static_cast<unsigned>(p.group);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_tested(bar, parity, abort, p.err)) != 0;
    };
    uint32_t n = 0, segs = 0;                          // tiles and segments so far
    // Q of a segment's rows -> shared memory, in the 128-byte swizzle: warpgroup g takes columns [64 g, 64 g + 64)
    auto stage_q = [&](const Walk& v) {
      const bool rv = r < v.rows();
      const unsigned br = static_cast<unsigned>(v.t * kPairRows + (rv ? r : 0));
      const unsigned qi = br / ug, gq = br - qi * ug;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<size_t>(v.s.q0 + qi) * p.hq + static_cast<size_t>(v.h) * p.group + gq) * HD) + g * 8;
      uint4 x[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = rv ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(sQ + g * kQBoxBytes + lr * 128 + ((c ^ (lr & 7)) << 4)) = x[c];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader(&bars->q_ready));
    };
    if (w.more()) stage_q(w);
    while (w.more()) {
      const bool rv = r < w.rows();
      const bool active = __any_sync(0xffffffffu, rv);
      const unsigned br = static_cast<unsigned>(w.t * kPairRows + (rv ? r : 0));
      const unsigned qi = br / ug;
      const int p0 = w.s.L - w.s.nq;
      const uint32_t* words = p.tree_mask + static_cast<size_t>(w.s.q0 + qi) * VFY_TREE_WORDS;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < w.nt; ++j, ++n) {
        const int gs = n % kGeo;
        const uint32_t sb = n & 1;
        // One warp waits for the tile's V in this CTA before it arrives for P, so the issuer's wait for P covers V too.
        if (warp == kVRelayWarp) {
          ok = wait(&bars->v_full[n % kVStages], (n / kVStages) & 1);
          if (!ok) break;
        }
        // (a tag that names the tile says all there is to know: most tiles need no wait for their geometry)
        const bool plain =
            __all_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&bars->plain_tag[gs]) == n + 1) != 0;
        bool zero = false;
        uint32_t keep[2] = {0u, 0u};
        if (!plain) {
          ok = wait(&bars->geo_full[gs], (n / kGeo) & 1);
          if (!ok) break;
          zero = bars->zero[gs] != 0;
          if (bars->valid[gs][g] != 0 && rv) {
            keep[0] = keep32(words, bars->base[gs][g], p0, w.s.L);
            keep[1] = keep32(words, bars->base[gs][g] + 32, p0, w.s.L);
          }
        }
        ok = wait(&bars->s_full[sb], (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const uint32_t ts = lane_base + kColS + sb * kKeys + g * kChunk;
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
            alpha = ex2_approx(m_ref - m_tile);      // 0 where m_ref = -inf
            l *= alpha;
            m_ref = m_tile;
          }
          if (__any_sync(0xffffffffu, scale_o)) {
            // O holds the tiles before this one: PV of the last one is waited for, which gives its V stage back. (PV of
            // this tile needs its P, so the stage's barrier is in that phase or the one after.)
            const uint32_t last = n - 1;
            ok = wait(&bars->v_empty[last % kVStages], (last / kVStages) & 1);
            if (!ok) break;
            tc_fence_after();
            const float a = scale_o ? alpha : 1.f;
#pragma unroll 1
            for (int x = 0; x < HD / 32; ++x) {
              uint32_t o[32];
              tmem_ld32(lane_base + kColO + g * 128 + x * 32, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st32(lane_base + kColO + g * 128 + x * 32, o);
            }
          }
          // p = 2^(s * scale * log2e - m_ref), packed over the first half of this chunk's S
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
          tmem_st32(ts, pk);
          const float2 sum = add_f32x2(add_f32x2(ps[0], ps[1]), add_f32x2(ps[2], ps[3]));
          l += sum.x + sum.y;
        }
        tc_fence_before();
        if (zero) {
          // V rows of keys outside the sequence may hold anything, and 0 * NaN is NaN on the tensor core: two threads
          // zero a key's row (its CTA's columns) before P.
          const int sv = n % kVStages;
          ok = wait(&bars->v_full[sv], (n / kVStages) & 1);
          if (!ok) break;
          const int key = lr >> 1;
          if (bars->valid[gs][g] == 0 || bars->base[gs][g] + key >= w.s.L) {
            uint8_t* row = sV + sv * kStageBytes + g * kBoxBytes + key * 128 + (lr & 1) * 64;
#pragma unroll
            for (int x = 0; x < 4; ++x) *reinterpret_cast<uint4*>(row + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(leader(&bars->p_full[sb]));
      }
      if (!ok) break;
      // ---- the segment's end: merge the two warpgroups' halves ----
      bars->xm[g][lr] = l > 0.f ? m_ref : -INFINITY;
      bars->xl[g][lr] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->half_ready[quarter]);
      ok = wait(&bars->half_ready[quarter], segs & 1);
      if (!ok) break;
      const float m0 = bars->xm[0][lr], m1 = bars->xm[1][lr], l0 = bars->xl[0][lr], l1 = bars->xl[1][lr];
      const float m_row = fmaxf(m0, m1);
      const float w0 = l0 > 0.f ? ex2_approx(m0 - m_row) : 0.f, w1 = l1 > 0.f ? ex2_approx(m1 - m_row) : 0.f;
      const float l_row = w0 * l0 + w1 * l1;
      ok = wait(&bars->o_done, segs & 1);
      if (!ok) break;
      tc_fence_after();
      // every S of the segment has read Q: the next one's first S may run during this one's epilogue
      Walk nx = w;
      nx.next(p);
      if (nx.more()) stage_q(nx);
      if (active) {
        // warpgroup g writes columns [64 g, 64 g + 64); a half without a key has no weight, and its O may be anything
        const bool whole = w.whole();
        const float inv = whole ? (l_row > 0.f ? 1.f / l_row : 0.f) : 1.f;
        const float a0 = w0 * inv, a1 = w1 * inv;
        const int t = w.s.q0 + static_cast<int>(qi);
        const int hq = w.h * p.group + static_cast<int>(br - qi * ug);
        const bool wr = rv && (!whole || t < p.token_cap);
        const size_t at = (2 * static_cast<size_t>(pair) + (w.index > 0 ? 1 : 0)) * kPairRows + r;
        uint16_t* out = p.out + (static_cast<size_t>(wr ? t : 0) * p.hq + hq) * HD + g * 64;
        float* part = p.part_o + at * HD + g * 64;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t o0[32], o1[32];
          tmem_ld32x2(lane_base + kColO + g * 64 + x * 32, lane_base + kColO + 128 + g * 64 + x * 32, o0, o1);
          if (!wr) continue;
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v[e] = l0 > 0.f ? a0 * __uint_as_float(o0[e]) : 0.f;
            v[e] = l1 > 0.f ? fmaf(a1, __uint_as_float(o1[e]), v[e]) : v[e];
          }
          if (whole) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
              pk[e] = *reinterpret_cast<const uint32_t*>(&h2);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(out + x * 32 + 2 * e) = make_uint4(pk[e], pk[e + 1], pk[e + 2], pk[e + 3]);
          } else if (l_row > 0.f) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(part + x * 32 + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
        if (wr && g == 0) {
          if (!whole)
            reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(l_row > 0.f ? m_row : -INFINITY, l_row);
          else if (p.lse != nullptr)
            p.lse[static_cast<size_t>(t) * p.hq + hq] =
                l_row > 0.f ? (m_row + __log2f(l_row)) * 0.6931471805599453f : -INFINITY;
        }
      }
      // the next segment's PV writes O, and its end (m, l): both warpgroups are done with both
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_read);
      ok = wait(&bars->o_read, segs & 1);
      if (!ok) break;
      ++segs;
      w = nx;
    }
  }
  // A wait that ran out ends the other CTA's waits too; both leave together (remote arrivals, pair MMAs).
  if (!ok && lane == 0) st_dsmem_u32(dsmem_addr(smem_u32(&bars->abort), rank ^ 1), 1u);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // The issuers' commits arrive in both CTAs, and neither leaves before it has the last ones. (By a warp without
  // other work: the same wait in a softmax warp or in the second CTA's producers cost 1.6 to 2.6 us of 110.)
  if (warp == kMmaWarp) {
    if (lane < 2) mbar_drain(&bars->drain[lane], 0, p.err);
    __syncwarp();
  }
  cluster_sync_all();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, kTmemCols);
  }
}

// ------------------------------ merge of the partial segments ------------------------------------
// A warp merges one row of an item that several runs hold; CTA (x, y) has rows [8 y, 8 y + 8) of the item that
// starts in run x and ends in a later one, if there is one. (A grid over all output rows, most of which no run
// boundary cuts in a large batch, took 27 us for 8 sequences of 64 nodes and 47 us for 16.)
constexpr int kMergeRows = 8;
constexpr int kAhead = 10;                     // pieces loaded at once

__global__ void __launch_bounds__(kMergeRows * 32) combine_tree_kernel(const AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int r = static_cast<int>(blockIdx.y) * kMergeRows + static_cast<int>(threadIdx.x >> 5);
  const TreePiece* rec = p.tree_pieces + blockIdx.x;
  const int4 r0 = __ldcg(reinterpret_cast<const int4*>(rec)), r1 = __ldcg(reinterpret_cast<const int4*>(rec) + 1);
  if (r >= r0.x) return;
  const unsigned br = static_cast<unsigned>(r0.y + r), ug = static_cast<unsigned>(p.group);
  const int t = r0.z + static_cast<int>(br / ug), hq = r0.w + static_cast<int>(br % ug);
  if (t >= p.token_cap) return;
  const int c0 = static_cast<int>(blockIdx.x), c1 = r1.y;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; c += kAhead) {
    float2 a[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int x = min(c + u, c1);
      const size_t at = static_cast<size_t>(x == c0 ? r1.x : 2 * x) * kPairRows + r;
      a[u] = __ldcg(ml + at);
      v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * HD) + lane);
      if (c + u > c1) a[u] = make_float2(-INFINITY, 0.f);
    }
    float mm = m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) mm = a[u].y > 0.f ? fmaxf(mm, a[u].x) : mm;
    const float old = l > 0.f ? ex2_approx(m - mm) : 0.f;
    l *= old;
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (a[u].y <= 0.f) continue;             // a piece without a key for this row holds no O
      const float w = ex2_approx(a[u].x - mm);
      l = fmaf(w, a[u].y, l);
      acc = make_float4(fmaf(w, v[u].x, acc.x), fmaf(w, v[u].y, acc.y), fmaf(w, v[u].z, acc.z), fmaf(w, v[u].w, acc.w));
    }
    m = mm;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint16_t* dst = p.out + (static_cast<size_t>(t) * p.hq + hq) * HD + lane * 4;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<size_t>(t) * p.hq + hq] = l > 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

// CTA pairs that can be resident at once on the current device (one CTA per SM), cached per device.
int attend_tree_pairs() {
  static int count[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (count[dev] != 0) return count[dev];
  static size_t done[64] = {};
  if (ensure_smem_limit(attend_tree_kernel, kSmemBytes, done) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, attend_tree_kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  count[dev] = n;
  return n;
}

cudaError_t launch_attend_tree(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int pairs,
                               cudaStream_t stream) {
  static size_t done[64] = {};
  cudaError_t e = ensure_smem_limit(attend_tree_kernel, kSmemBytes, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attend_tree_kernel, dim3(2 * pairs), dim3(kThreads), kSmemBytes, stream, p, tk, tv);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine_tree_kernel, dim3(pairs, kPairRows / kMergeRows), dim3(kMergeRows * 32), 0, stream, p);
}

}  // namespace vfy
