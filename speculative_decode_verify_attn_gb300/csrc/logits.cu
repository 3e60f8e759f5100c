// Rules on the target's logits before the acceptance: penalties for tokens a sequence holds already,
// biases and grammar masks, for every row of the block; and the token counts behind the penalties.
//
// process_logits: with c = generated count of token v + how often v is drafted on the row's path,
//     x = seen ? (x > 0 ? x / r : x r) : x;  x -= f c + (c > 0 ? q : 0);  x += bias_v;  masked -> -inf
// A row reads V logits and V / 32 mask words and writes V floats; the counts and biases belong to
// the sequence. So a CTA takes one vocabulary segment of one sequence and runs over the block's rows:
// a thread keeps its columns' counts and biases in registers and reads them once for all rows. What
// differs between rows are the drafted tokens on their paths: the few columns of the segment that any
// node drafts carry the set of those nodes, and a row's extra count is the number of set nodes in its
// mask (popcounts). So a row needs no pass of its own and the call may work in place.
// Bound by the bytes of the logits in and out.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 4;                       // columns per thread
constexpr int kSeg = kThreads * kCols;         // columns per CTA
constexpr int kNodes = VFY_MAX_TREE_NODES;
constexpr int kWords = VFY_TREE_WORDS;
constexpr int kNone = 0x7fffffff;
constexpr int kRows = 4;                       // rows in flight

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* base, size_t at) {
  if constexpr (BF16)
    return __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16*>(base) + at));
  else
    return reinterpret_cast<const float*>(base)[at];     // may be the output: no read-only path
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) process_logits_kernel(const LogitParams p) {
  __shared__ int s_entry[kSeg];                // per column: lowest node (less one) that drafts it, or a bias entry's turn
  __shared__ float s_bias[kSeg];
  __shared__ uint32_t s_set[kNodes][kWords];   // per entry: the nodes that draft its token
  pdl_launch_dependents();
  pdl_wait();
  const vfy_logit_rules& r = p.rules;
  const int b = blockIdx.y;
  const int r0 = p.cu_rows[b];
  const int n = p.cu_rows[b + 1] - r0;
  const bool report = blockIdx.x == 0 && blockIdx.z == 0;
  // (r0 < b: an earlier sequence has no row, and the drafts of this one would start before the list)
  if (n < 1 || n > kNodes || r0 < b || r0 > p.max_rows - n) {
    if (report && threadIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const int seg0 = blockIdx.x * kSeg;
  const int i0 = static_cast<int>(static_cast<long long>(n) * blockIdx.z / gridDim.z);
  const int i1 = static_cast<int>(static_cast<long long>(n) * (blockIdx.z + 1) / gridDim.z);
  if (i0 >= i1 && !report) return;

  const bool penalties = r.counts != nullptr;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  int32_t count[kCols];
  float bias[kCols];
#pragma unroll
  for (int e = 0; e < kCols; ++e) {
    const int v = seg0 + e * kThreads + static_cast<int>(threadIdx.x);
    count[e] = penalties && v < p.vocab ? r.counts[static_cast<size_t>(b) * p.vocab + v] : 0;
    bias[e] = 0.f;
  }
  if (penalties) {
    if (r.repetition != nullptr) rep = r.repetition[b];
    if (r.frequency != nullptr) freq = r.frequency[b];
    if (r.presence != nullptr) pres = r.presence[b];
  }

  // ---- the sequence's biases of this segment, added up in list order ----
  bool have_bias = false;
  if (r.cu_bias != nullptr) {
    for (int c = threadIdx.x; c < kSeg; c += kThreads) {
      s_entry[c] = kNone;
      s_bias[c] = 0.f;
    }
    __syncthreads();
    const int e0 = r.cu_bias[b], e1 = r.cu_bias[b + 1];
    for (int base = e0; base < e1; base += kThreads) {
      const int e = base + static_cast<int>(threadIdx.x);
      int col = -1;
      float val = 0.f;
      if (e < e1) {
        const int tok = r.bias_token[e];
        if (tok < 0 || tok >= p.vocab) {
          if (report) atomicOr(p.err, kErrDeviceInput);
        } else if (tok >= seg0 && tok < seg0 + kSeg) {
          col = tok - seg0;
          val = r.bias_value[e];
        }
      }
      // of the entries with one token the lowest goes first: a round per repetition
      while (__syncthreads_or(col >= 0)) {
        have_bias = true;
        if (col >= 0) atomicMin(&s_entry[col], e);
        __syncthreads();
        const bool turn = col >= 0 && s_entry[col] == e;
        __syncthreads();
        if (turn) {
          s_bias[col] += val;
          s_entry[col] = kNone;
          col = -1;
        }
      }
    }
    if (have_bias) {
#pragma unroll
      for (int e = 0; e < kCols; ++e) bias[e] = s_bias[e * kThreads + threadIdx.x];
    }
  }

  // ---- the drafted tokens of this segment: for each, the set of nodes that draft it ----
  int entry[kCols];
#pragma unroll
  for (int e = 0; e < kCols; ++e) entry[e] = kNone;
  if (penalties && r.drafts != nullptr && n > 1) {
    const int node = static_cast<int>(threadIdx.x) + 1;      // node 0 is in the counts
    int col = -1;
    if (node < n) {
      const int tok = r.drafts[r0 - b + node - 1];
      if (tok < 0 || tok >= p.vocab) {
        if (report) atomicOr(p.err, kErrDeviceInput);
      } else if (tok >= seg0 && tok < seg0 + kSeg) {
        col = tok - seg0;
      }
    }
    if (__syncthreads_or(col >= 0)) {
      for (int c = threadIdx.x; c < kSeg; c += kThreads) s_entry[c] = kNone;
      for (int x = threadIdx.x; x < kNodes * kWords; x += kThreads) s_set[0][x] = 0u;
      __syncthreads();
      if (col >= 0) atomicMin(&s_entry[col], node - 1);
      __syncthreads();
      if (col >= 0) atomicOr(&s_set[s_entry[col]][node >> 5], 1u << (node & 31));
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kCols; ++e) entry[e] = s_entry[e * kThreads + threadIdx.x];
    }
  }

  // ---- the rows ----
  const size_t words_per_mask = (static_cast<size_t>(p.vocab) + 31) / 32;
  for (int ib = i0; ib < i1; ib += kRows) {
    float x[kRows][kCols];
    uint32_t lets[kRows][kCols];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = min(ib + u, i1 - 1);
      const size_t row = static_cast<size_t>(r0 + i);
      long long mask = -1;
      if (r.grammar != nullptr) {
        mask = r.mask_index != nullptr ? r.mask_index[row] : static_cast<long long>(row);
        if (mask < -1 || mask >= r.num_masks) {
          if (report && threadIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
          mask = -1;
        }
      }
#pragma unroll
      for (int e = 0; e < kCols; ++e) {
        const int v = seg0 + e * kThreads + static_cast<int>(threadIdx.x);
        const bool in = v < p.vocab;
        x[u][e] = in ? load_logit<BF16>(p.logits, row * p.stride + v) : 0.f;
        lets[u][e] = in && mask >= 0 ? __ldg(r.grammar + mask * words_per_mask + (v >> 5)) : 0xffffffffu;
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = ib + u;
      if (i >= i1) break;
      const size_t row = static_cast<size_t>(r0 + i);
#pragma unroll
      for (int e = 0; e < kCols; ++e) {
        const int v = seg0 + e * kThreads + static_cast<int>(threadIdx.x);
        if (v >= p.vocab) continue;
        int32_t word = count[e];
        if (entry[e] != kNone) {
          int extra = 0;
          for (int w = 0; w < kWords; ++w) {
            const uint32_t path = r.tree_mask != nullptr ? __ldg(r.tree_mask + row * kWords + w)
                                  : i >= 32 * w + 31     ? 0xffffffffu
                                  : i < 32 * w           ? 0u
                                                         : (2u << (i - 32 * w)) - 1u;
            extra += __popc(path & s_set[entry[e]][w]);
          }
          word += extra;                               // bit 31 stays: counts stay below 2^31
        }
        float y = x[u][e];
        if (word != 0) {
          const float c = static_cast<float>(word & 0x7fffffff);
          y = y > 0.f ? y / rep : y * rep;
          y -= freq * c;
          if (c > 0.f) y -= pres;
        }
        if (have_bias) y += bias[e];
        if (!((lets[u][e] >> (v & 31)) & 1u)) y = -INFINITY;
        p.out[row * p.vocab + v] = y;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) count_tokens_kernel(const CountParams p) {
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

}  // namespace

cudaError_t launch_process_logits(const LogitParams& p, bool bf16, cudaStream_t stream) {
  dim3 grid((p.vocab + kSeg - 1) / kSeg, p.num_seqs, p.row_parts);
  if (bf16) return launch_pdl(process_logits_kernel<true>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(process_logits_kernel<false>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_count_tokens(const CountParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.max_tokens + kThreads - 1) / kThreads);
  count_tokens_kernel<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vfy
