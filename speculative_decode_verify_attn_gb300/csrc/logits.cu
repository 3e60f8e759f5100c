// Rules on the target's logits before the acceptance: penalties for tokens a sequence holds already,
// biases and grammar masks, for every row of the block; and the token counts behind the penalties.
//
// process_logits: with c = generated count of token v + how often v is drafted on the row's path,
//     x = seen ? (x > 0 ? x / r : x r) : x;  x -= f c + (c > 0 ? q : 0);  x += bias_v;  masked -> -inf
// A row reads V logits and V / 32 mask words and writes V floats; the counts and biases belong to
// the sequence. So a CTA takes one vocabulary segment of one sequence and runs over the block's rows:
// what a column's count and biases do to it is worked out once. What differs between rows are the
// drafted tokens on their paths: the main loop leaves out the few columns of the segment that any node
// drafts, and at the end a thread per (row, such column) counts the drafting nodes in the row's mask.
// Every entry is read and written by one thread, so the call may work in place.
// Bound by bytes in flight and, in a batch, by issue slots, half of which are taken. So the first rows' logits are
// loaded before the rules, the masks of 32 rows at a time go through shared memory (one wait instead of one per batch),
// staged from each row's first column on, so that a thread's bits are two shifts; four rows of eight columns are in
// flight per thread; and entries take the steps of the rules in use only. GB300: 17 x 131072 fp32 8.4 us (the bytes
// alone 2.7); 339 rows x 100003 bf16 of 16 sequences 56.0 us (3.8 TB/s; 47.7 us with a vocabulary of 100000, whose rows
// all start alike, 37.8 of it without rules). Loading eight neighbouring columns per thread (half-sector stores),
// per-thread mask loads, and columns past a row's end in a loop of their own each cost 15 to 40 us of the batch;
// refilling each row's registers as soon as it is done, instead of four rows at a time, 20, loading a batch ahead 5.
// Five CTAs per SM or six made no difference to the batch; fp32 rows take five (four: 17 rows 10.4 us).
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 8;                       // columns per thread: two groups of four neighbours, so that a
constexpr int kGroup = kThreads * 4;           // warp's 16-byte stores cover whole sectors
constexpr int kSeg = kThreads * kCols;         // columns per CTA
constexpr int kWords = VFY_TREE_WORDS;
constexpr int kNone = 0x7fffffff;
constexpr int kSpan = kSeg + 3;                // columns a CTA keeps
constexpr int kBiasAhead = 4;                  // bias entries in flight per thread
constexpr int kSegWords = kSeg / 32;           // words of a row's staged mask
constexpr int kSpanIters = (kSpan + kThreads - 1) / kThreads;

// A thread's eight columns of one row, as they were loaded: rows in flight cost registers. Bit e of `valid`:
// column e lies in the row (the others read 0). `vec`: the groups are aligned to their four-entry words.
// (Plain loads, not the read-only path: the logits may be the output.)
template <bool BF16>
struct Raw {
  uint32_t w[BF16 ? 4 : 8];
};
template <bool BF16>
__device__ __forceinline__ void load_row(const char* at, bool vec, uint32_t valid, Raw<BF16>& d) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const char* s = at + g * kGroup * (BF16 ? 2 : 4);
    const uint32_t ok = (valid >> (4 * g)) & 15u;
    if (vec && ok == 15u) {
      if constexpr (BF16) {
        const uint2 a = *reinterpret_cast<const uint2*>(s);
        d.w[2 * g] = a.x, d.w[2 * g + 1] = a.y;
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(s);
        d.w[4 * g] = a.x, d.w[4 * g + 1] = a.y, d.w[4 * g + 2] = a.z, d.w[4 * g + 3] = a.w;
      }
    } else if constexpr (BF16) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(s);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t lo = (ok >> (2 * e)) & 1u ? h[2 * e] : 0u, hi = (ok >> (2 * e + 1)) & 1u ? h[2 * e + 1] : 0u;
        d.w[2 * g + e] = lo | (hi << 16);
      }
    } else {
      const uint32_t* f = reinterpret_cast<const uint32_t*>(s);
#pragma unroll
      for (int e = 0; e < 4; ++e) d.w[4 * g + e] = (ok >> e) & 1u ? f[e] : 0u;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ float entry_of(const Raw<BF16>& d, int e) {
  if constexpr (BF16)
    return __uint_as_float(e & 1 ? d.w[e >> 1] & 0xffff0000u : d.w[e >> 1] << 16);
  else
    return __uint_as_float(d.w[e]);
}
// column e of a thread's eight, from its first
__device__ __forceinline__ constexpr int col_of(int e) { return (e >> 2) * kGroup + (e & 3); }

// ONE: every sequence has one row, as when a request starts or decodes without drafts: node 0 is in the counts, so
// no token is drafted. Seven CTAs per SM then hold 8 rows of 131072 columns in one wave (8 requests' first rows with
// their prompt counts 9.8 us, 14.3 with the general kernel).
template <bool BF16, bool ONE>
__global__ void __launch_bounds__(kThreads, ONE ? 7 : 5) process_logits_kernel(const LogitParams p) {
  constexpr int kNodes = ONE ? 1 : VFY_MAX_TREE_NODES;
  constexpr int kMaskRows = ONE ? 1 : 32;      // rows whose mask words are staged at a time
  constexpr int kMaskIters = (kMaskRows * kSegWords + kThreads - 1) / kThreads;
  // Columns seg0 - 3 .. seg0 + kSeg - 1 of the sequence (a row uses kSeg of them, see below).
  __shared__ int32_t s_count[kSpan];
  __shared__ float s_bias[kSpan];
  __shared__ int s_entry[ONE ? 1 : kSpan];     // lowest node (less one) that drafts the column
  __shared__ int s_turn[kSpan];                // lowest bias entry of the column still to be added
  __shared__ uint32_t s_set[kNodes][kWords];   // per entry: the nodes that draft its token
  __shared__ int s_mask[kNodes];               // per row: its grammar mask, -1 = none
  __shared__ int s_drafted[kNodes];            // the drafted columns, once each
  __shared__ uint32_t s_lets[kMaskRows][kSegWords];   // masks of a chunk of this CTA's rows, from the row's first column on
  __shared__ int s_num_drafted;
  pdl_launch_dependents();
  pdl_wait();
  const vfy_logit_rules& r = p.rules;
  const int tid = static_cast<int>(threadIdx.x);
  int b = blockIdx.y;
  if (!ONE && p.num_seqs > 1 && p.num_seqs <= 32) {
    // The sequences with the most rows go first, so that the last CTAs are short ones (the ragged batch 67.4 -> 60.8 us,
    // one of equal lengths 95.2 -> 96.1).
    const int lane = tid & 31;
    const bool have = lane < p.num_seqs;
    const int rows = have ? p.cu_rows[lane + 1] - p.cu_rows[lane] : 0;
    int rank = 0;
    for (int i = 0; i < p.num_seqs; ++i) {
      const int other = __shfl_sync(0xffffffffu, rows, i);
      rank += other > rows || (other == rows && i < lane) ? 1 : 0;
    }
    b = __ffs(__ballot_sync(0xffffffffu, have && rank == b)) - 1;
  }
  const int r0 = p.cu_rows[b];
  const int n = p.cu_rows[b + 1] - r0;
  const bool report = blockIdx.x == 0 && blockIdx.z == 0;
  // (r0 < b: an earlier sequence has no row, and the drafts of this one would start before the list)
  if (n < 1 || n > kNodes || r0 < b || r0 > p.max_rows - n) {
    if (report && tid == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  // This CTA's rows: r0 + i = z (mod step). Rows start at different places of a four-entry word unless
  // the vocabulary is a multiple of 4, and a thread's four columns shift with them so that they stay one
  // aligned word of `out`. The rows run in passes of equal shift, so that a column's state is taken from
  // shared memory once per pass: four passes over every fourth row, or one where all rows shift alike.
  const int step = gridDim.z;
  const int i0 = (static_cast<int>(blockIdx.z) - r0 % step + step) % step;
  if (i0 >= n && !report) return;
  const int passes = ONE || ((p.vocab & 3) == 0 && (p.stride & 3) == 0) || (step & 3) == 0 ? 1 : 4;
  const int stride = passes * step;            // rows of one pass
  const int seg0 = static_cast<int>(blockIdx.x) * kSeg;
  const long long out_base = static_cast<long long>(reinterpret_cast<uintptr_t>(p.out) >> 2);
  const long long in_base = static_cast<long long>(reinterpret_cast<uintptr_t>(p.logits) >> (BF16 ? 1 : 2));
  auto shift_of = [&](int i) { return static_cast<int>(((r0 + static_cast<long long>(i)) * p.vocab + out_base) & 3); };

  // A batch: kRows rows of a pass at the columns v0 + {0 .. 3} and v0 + kGroup + {0 .. 3} of this thread:
  // 64 or 128 bytes of logits in flight per thread, 20 warps per SM. Columns past the row's ends are
  // left out one by one, within the same batches.
  constexpr int kRows = ONE ? 1 : 4;
  constexpr int kSize = BF16 ? 2 : 4;
  const uint32_t words_per_mask = (static_cast<uint32_t>(p.vocab) + 31u) / 32u;
  const long long in_pitch = static_cast<long long>(stride) * p.stride * kSize;
  const long long out_pitch = static_cast<long long>(stride) * p.vocab;
  auto valid_of = [&](int v0) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kCols; ++e) m |= (v0 + col_of(e) >= 0 && v0 + col_of(e) < p.vocab ? 1u : 0u) << e;
    return m;
  };
  Raw<BF16> x[kRows];
  auto load_rows = [&](int ib, int rows, int v0, uint32_t valid) {     // rows: of the chunk, from ib on
    const long long at = (r0 + static_cast<long long>(ib)) * p.stride + v0;
    const bool vec = ((at + in_base) & 3) == 0;
    const char* src = static_cast<const char*>(p.logits) + at * kSize;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (u * passes < rows) load_row<BF16>(src, vec, valid, x[u]);
      src += in_pitch;
    }
  };
  const bool grammar = r.grammar != nullptr;
  int v0 = seg0 - shift_of(i0) + 4 * tid;
  uint32_t valid = valid_of(v0);
  if (i0 < n) load_rows(i0, min((n - i0 + step - 1) / step, kMaskRows), v0, valid);     // while the rules are read

  // ---- the sequence's rules for these columns ----
  const bool penalties = r.counts != nullptr;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  int e0 = 0, e1 = 0;                          // bias entries
  if (r.cu_bias != nullptr) {
    e0 = r.cu_bias[b];
    e1 = r.cu_bias[b + 1];
    if (e0 < 0 || e1 < e0) {
      if (report && tid == 0) atomicOr(p.err, kErrDeviceInput);
      e0 = e1 = 0;
    }
  }
  constexpr int kNodeIters = (kNodes + kThreads - 1) / kThreads;
  int draft_col[kNodeIters];                   // this thread's nodes tid + 1, ... (node 0 is in the counts)
  if (penalties) {
    if (r.repetition != nullptr) rep = r.repetition[b];
    if (r.frequency != nullptr) freq = r.frequency[b];
    if (r.presence != nullptr) pres = r.presence[b];
  }
#pragma unroll
  for (int k = 0; k < kNodeIters; ++k) {
    draft_col[k] = -1;
    const int at = k * kThreads + tid;
    if (penalties && r.drafts != nullptr && at + 1 < n) {
      const int tok = r.drafts[r0 - b + at];
      if (tok < 0 || tok >= p.vocab) {
        if (report) atomicOr(p.err, kErrDeviceInput);
      } else if (tok >= seg0 - 3 && tok < seg0 + kSeg) {
        draft_col[k] = tok - seg0 + 3;
      }
    }
    if (at < n) {
      int mask = !grammar ? -1 : r.mask_index != nullptr ? r.mask_index[r0 + at] : r0 + at;
      if (mask < -1 || (mask >= r.num_masks && grammar)) {
        if (report) atomicOr(p.err, kErrDeviceInput);
        mask = -1;
      }
      s_mask[at] = mask;
    }
  }
  int bias_col[kBiasAhead];
  float bias_val[kBiasAhead];
  auto load_bias = [&](int base) {
#pragma unroll
    for (int u = 0; u < kBiasAhead; ++u) {
      const unsigned e = static_cast<unsigned>(base) + u * kThreads + tid;     // (past 2^31 behind the longest list)
      bias_col[u] = -1;
      bias_val[u] = 0.f;
      if (e >= static_cast<unsigned>(e1)) continue;
      const int tok = r.bias_token[e];
      bias_val[u] = r.bias_value[e];
      if (tok < 0 || tok >= p.vocab) {
        if (report) atomicOr(p.err, kErrDeviceInput);
      } else if (tok >= seg0 - 3 && tok < seg0 + kSeg) {
        bias_col[u] = tok - seg0 + 3;
      }
    }
  };
  load_bias(e0);
  // (all of a thread's counts and mask words at once: a wait for memory less each)
  int32_t count[kSpanIters];
#pragma unroll
  for (int u = 0; u < kSpanIters; ++u) {
    const int v = seg0 - 3 + tid + u * kThreads;
    count[u] = penalties && v >= 0 && v < p.vocab && tid + u * kThreads < kSpan
                   ? __ldg(r.counts + static_cast<size_t>(b) * p.vocab + v)
                   : 0;
  }
  const int my_rows = i0 < n ? (n - i0 + step - 1) / step : 0;
  // the masks of rows j0 .. j1 - 1 of this CTA, into s_lets; mask_of(i) = the mask of row i, -1 = none
  auto stage_masks = [&](int j0, int j1, auto mask_of) {
    uint32_t lo[kMaskIters], hi[kMaskIters];
#pragma unroll
    for (int u = 0; u < kMaskIters; ++u) {
      const int x = tid + u * kThreads, j = x / kSegWords, w = x % kSegWords;
      lo[u] = hi[u] = 0xffffffffu;
      if (j < j1 - j0) {
        const int i = i0 + (j0 + j) * step, mask = mask_of(i), shift = shift_of(i);
        const int at = (seg0 >> 5) + w - (shift > 0 ? 1 : 0);        // the word of this one's first column
        if (mask >= 0) {
          const uint32_t* words = r.grammar + static_cast<uint64_t>(static_cast<uint32_t>(mask)) * words_per_mask;
          if (at >= 0 && at < static_cast<int>(words_per_mask)) lo[u] = __ldg(words + at);
          if (shift > 0 && at + 1 < static_cast<int>(words_per_mask)) hi[u] = __ldg(words + at + 1);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kMaskIters; ++u) {
      const int x = tid + u * kThreads, j = x / kSegWords;
      const int shift = shift_of(i0 + (j0 + j) * step);
      if (j < j1 - j0) (&s_lets[0][0])[x] = shift > 0 ? __funnelshift_r(lo[u], hi[u], 32 - shift) : lo[u];
    }
  };
  if (grammar)
    stage_masks(0, min(my_rows, kMaskRows), [&](int i) {
      const int mask = r.mask_index != nullptr ? __ldg(r.mask_index + r0 + i) : r0 + i;
      return mask < r.num_masks ? mask : -1;
    });
#pragma unroll
  for (int u = 0; u < kSpanIters; ++u) {
    const int c = tid + u * kThreads;
    if (c >= kSpan) break;
    s_count[c] = count[u];
    s_bias[c] = -0.f;
    if constexpr (!ONE) s_entry[c] = kNone;
    s_turn[c] = kNone;
  }
  if (tid == 0) s_num_drafted = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kNodeIters; ++k) {
    if (ONE || draft_col[k] < 0) continue;
    if (atomicMin(&s_entry[draft_col[k]], k * kThreads + tid) == kNone)
      s_drafted[atomicAdd(&s_num_drafted, 1)] = draft_col[k];
  }
  // Biases are added up in list order: of the entries with one token the lowest goes first, a round per
  // repetition.
  for (int base = e0;;) {
    bool pending = false;
#pragma unroll
    for (int u = 0; u < kBiasAhead; ++u) {
      if (bias_col[u] < 0) continue;
      pending = true;
      atomicMin(&s_turn[bias_col[u]], base + u * kThreads + tid);
    }
    bool todo = __syncthreads_or(pending) != 0;     // (most chunks hold nothing for this segment)
    while (todo) {
      bool turn[kBiasAhead];
#pragma unroll
      for (int u = 0; u < kBiasAhead; ++u)
        turn[u] = bias_col[u] >= 0 && s_turn[bias_col[u]] == base + u * kThreads + tid;
      __syncthreads();
      bool more = false;
#pragma unroll
      for (int u = 0; u < kBiasAhead; ++u) {
        if (turn[u]) {
          s_bias[bias_col[u]] += bias_val[u];
          s_turn[bias_col[u]] = kNone;
          bias_col[u] = -1;
        }
        more = more || bias_col[u] >= 0;
      }
      todo = __syncthreads_or(more) != 0;
      if (!todo) break;
#pragma unroll
      for (int u = 0; u < kBiasAhead; ++u)
        if (bias_col[u] >= 0) atomicMin(&s_turn[bias_col[u]], base + u * kThreads + tid);
      __syncthreads();
    }
    if (e1 - base <= kThreads * kBiasAhead) break;
    base += kThreads * kBiasAhead;
    load_bias(base);
  }
  const int num_drafted = ONE ? 0 : s_num_drafted;       // (the bias rounds passed at least one barrier)
  if (num_drafted > 0) {
    for (int w = tid; w < kNodes * kWords; w += kThreads) s_set[0][w] = 0u;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kNodeIters; ++k) {
      const int node = k * kThreads + tid + 1;
      if (draft_col[k] >= 0) atomicOr(&s_set[s_entry[draft_col[k]]][node >> 5], 1u << (node & 31));
    }
    __syncthreads();
  }

  // What the rules do to an entry: x m + add, m = seen ? (x > 0 ? 1 / rep : rep) : 1, with one rounding
  // for the product and the sum; 1 / rep is rounded once more. A column that no rule touches has m = 1
  // and add = -0: x stays x, the sign of a zero too.
  const bool rules = penalties || r.cu_bias != nullptr;
  const float inv = 1.f / rep;
  auto addend = [&](int32_t word, float bias) {
    const float c = static_cast<float>(word & 0x7fffffff);
    return bias - (word != 0 ? fmaf(freq, c, c > 0.f ? pres : 0.f) : 0.f);
  };
  auto rule = [&](float v, bool seen, float add) {
    return fmaf(v, seen ? (v > 0.f ? inv : rep) : 1.f, add);
  };
  // ---- the rows, kMaskRows of this CTA's at a time (row j: i = i0 + j step) ----
  for (int j0 = 0; j0 < my_rows; j0 += kMaskRows) {
    const int j1 = min(my_rows, j0 + kMaskRows);
    if (grammar && j0 > 0) {
      __syncthreads();
      stage_masks(j0, j1, [&](int i) { return s_mask[i]; });
      __syncthreads();
    }
    for (int pass = 0; pass < passes; ++pass) {
      const int first = j0 + pass;               // of the pass; its rows are `passes` apart
      if (first >= j1) break;
      if (j0 + pass > 0) {
        v0 = seg0 - shift_of(i0 + first * step) + 4 * tid;
        valid = valid_of(v0);
      }
      if (valid == 0u) continue;
      const int c0 = v0 - seg0 + 3;
      uint32_t seen = 0, mine = valid;           // bit e: column e is seen; this loop writes it
      float add[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) {
        const int c = c0 + col_of(e);
        const int32_t word = s_count[c];
        if (word != 0) seen |= 1u << e;
        add[e] = addend(word, s_bias[c]);
        if (!ONE && num_drafted > 0 && s_entry[c] != kNone) mine &= ~(1u << e);
      }
      float* dst = p.out + ((r0 + static_cast<long long>(i0 + first * step)) * p.vocab + v0);
      for (int jb = first; jb < j1; jb += kRows * passes) {
        if (jb > 0) load_rows(i0 + jb * step, j1 - jb, v0, valid);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int j = jb + u * passes;
          if (j >= j1) break;
          float y[kCols];
#pragma unroll
          for (int e = 0; e < kCols; ++e) y[e] = entry_of<BF16>(x[u], e);
          if (rules) {
#pragma unroll
            for (int e = 0; e < kCols; ++e) y[e] = rule(y[e], (seen >> e) & 1u, add[e]);
          }
          if (grammar) {
            const uint32_t* words = s_lets[j - j0] + (tid >> 3);
            const uint32_t a = words[0] >> (4 * (tid & 7)), c = words[kGroup / 32] >> (4 * (tid & 7));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = (a >> e) & 1u ? y[e] : -INFINITY;
              y[e + 4] = (c >> e) & 1u ? y[e + 4] : -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            if (((mine >> e) & 15u) == 15u) {
              *reinterpret_cast<float4*>(dst + col_of(e)) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            } else {
#pragma unroll
              for (int f = e; f < e + 4; ++f)
                if ((mine >> f) & 1u) dst[col_of(f)] = y[f];
            }
          }
          dst += out_pitch;
        }
      }
    }
  }

  // ---- the drafted columns, a thread per (row, column): the row's own path counts too ----
  if constexpr (!ONE) {
    for (int x = tid; x < my_rows * num_drafted; x += kThreads) {
      const int i = i0 + (x / num_drafted) * step, c = s_drafted[x % num_drafted];
      const long long row = r0 + static_cast<long long>(i);
      const int v = seg0 - 3 + c;
      const int shift = shift_of(i);
      if (v < seg0 - shift || v >= seg0 - shift + kSeg) continue;      // another CTA's column in this row
      const uint32_t* set = s_set[s_entry[c]];
      int extra = 0;
  #pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint32_t path = r.tree_mask != nullptr ? __ldg(r.tree_mask + row * kWords + w)
                              : i >= 32 * w + 31     ? 0xffffffffu     // a chain's path: nodes 0 .. i
                              : i < 32 * w           ? 0u
                                                     : (2u << (i - 32 * w)) - 1u;
        extra += __popc(path & set[w]);
      }
      const int32_t word = s_count[c] + extra;                         // bit 31 stays: counts stay below 2^31
      const long long at = row * p.stride + v;
      const float in = BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.logits)[at]) << 16)
                            : static_cast<const float*>(p.logits)[at];
      float y = rule(in, word != 0, addend(word, s_bias[c]));      // (drafts come with counts)
      if (s_mask[i] >= 0) {
        const uint64_t word0 = static_cast<uint64_t>(static_cast<uint32_t>(s_mask[i])) * words_per_mask;
        const uint32_t bits = __ldg(r.grammar + word0 + (v >> 5));
        if (!((bits >> (v & 31)) & 1u)) y = -INFINITY;
      }
      p.out[row * p.vocab + v] = y;
    }
  }
}

__global__ void __launch_bounds__(kThreads) count_tokens_kernel(const CountParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int total = p.cu_tokens[p.num_seqs];
  const long long t = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (t == 0 && total > p.max_tokens) atomicOr(p.err, kErrDeviceInput);
  if (t >= total || t >= p.max_tokens) return;
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_tokens[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int tok = p.tokens[t];
  if (t < p.cu_tokens[lo] || t >= p.cu_tokens[lo + 1] || tok < -1 || tok >= p.vocab) {
    atomicOr(p.err, kErrDeviceInput);
    return;
  }
  if (tok < 0) return;
  int32_t* word = p.counts + static_cast<size_t>(lo) * p.vocab + tok;
  if (p.as_prompt) {
    if (!(__ldcg(word) & static_cast<int32_t>(0x80000000u)))
      atomicOr(reinterpret_cast<unsigned int*>(word), 0x80000000u);
  } else {
    atomicAdd(word, 1);
  }
}

// Counts from scratch (reset): a CTA owns one segment of one sequence's counts in shared memory, runs over
// all of the sequence's tokens and writes the segment out whole, so nothing is zeroed first and no
// global atomics run. The tokens are read once per segment, from L2.
constexpr int kHistThreads = 1024;
constexpr int kHistAhead = 16;         // tokens in flight per thread

__global__ void __launch_bounds__(kHistThreads) rebuild_counts_kernel(const CountParams p) {
  extern __shared__ uint32_t s_count[];
  pdl_launch_dependents();
  const int seg0 = static_cast<int>(blockIdx.x) * p.seg;
  const int seg = min(p.seg, p.vocab - seg0);
  for (int c = threadIdx.x; c < seg; c += kHistThreads) s_count[c] = 0u;
  pdl_wait();
  const int b = blockIdx.y;
  const int t0 = p.cu_tokens[b];
  int t1 = p.cu_tokens[b + 1];                           // (up to 2^31 - 1: places past it are unsigned)
  bool bad = false;
  if (t0 < 0 || t1 < t0 || t1 > p.max_tokens) {        // its counts become zero
    bad = true;
    t1 = t0 < 0 ? 0 : t0;
  }
  __syncthreads();
  const unsigned end = static_cast<unsigned>(t1);
  for (unsigned base = static_cast<unsigned>(t0); base < end; base += kHistThreads * kHistAhead) {
    int tok[kHistAhead];
#pragma unroll
    for (int u = 0; u < kHistAhead; ++u) {
      const unsigned at = base + u * kHistThreads + threadIdx.x;
      tok[u] = at < end ? __ldg(p.tokens + at) : -1;
    }
#pragma unroll
    for (int u = 0; u < kHistAhead; ++u) {
      bad = bad || tok[u] < -1 || tok[u] >= p.vocab;
      const unsigned c = static_cast<unsigned>(tok[u]) - static_cast<unsigned>(seg0);
      if (tok[u] < 0 || c >= static_cast<unsigned>(seg)) continue;
      if (p.as_prompt)
        s_count[c] = 0x80000000u;                        // every writer writes the same
      else
        atomicAdd(&s_count[c], 1u);
    }
  }
  if (bad && blockIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
  __syncthreads();
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.counts) + static_cast<size_t>(b) * p.vocab + seg0;
  for (int c = threadIdx.x; c < seg; c += kHistThreads) dst[c] = s_count[c];
}

}  // namespace

cudaError_t launch_process_logits(const LogitParams& p, bool bf16, cudaStream_t stream) {
  dim3 grid(p.segs, p.num_seqs, p.row_parts);
  // (each sequence has a row at least)
  const bool one = p.max_rows == p.num_seqs;
  if (bf16)
    return one ? launch_pdl(process_logits_kernel<true, true>, grid, dim3(kThreads), 0, stream, p)
               : launch_pdl(process_logits_kernel<true, false>, grid, dim3(kThreads), 0, stream, p);
  return one ? launch_pdl(process_logits_kernel<false, true>, grid, dim3(kThreads), 0, stream, p)
             : launch_pdl(process_logits_kernel<false, false>, grid, dim3(kThreads), 0, stream, p);
}

// (where rows are not aligned, up to 3 columns of the first CTA lie before the row)
int logit_segments(int vocab, bool even) { return (vocab + (even ? 0 : 3) + kSeg - 1) / kSeg; }

cudaError_t launch_count_tokens(const CountParams& p, cudaStream_t stream) {
  if (p.reset) {
    dim3 grid((p.vocab + p.seg - 1) / p.seg, p.num_seqs);
    return launch_pdl(rebuild_counts_kernel, grid, dim3(kHistThreads), static_cast<size_t>(p.seg) * 4, stream, p);
  }
  const unsigned grid = static_cast<unsigned>((p.max_tokens + kThreads - 1) / kThreads);
  return launch_pdl(count_tokens_kernel, dim3(grid), dim3(kThreads), 0, stream, p);
}

}  // namespace vfy
