// Fused argmax + acceptance for a tree of drafted tokens.
// Source: "Laguna XS 2.1 33B on a RTX 3090" (lucebox), "The model, fast MoE with a drafter in the
// box" (commit only tokens the target itself would emit), for several drafted continuations.
//
// Phase 1: as in the chain's acceptance, every CTA reduces a vocabulary segment of one row to the
// row's key (argmax.cuh), combined with atomicMax. Rows start at any multiple of 4 bytes (an odd
// vocabulary), so a segment is scanned as 16-byte words between its aligned ends.
// Phase 2: the last CTA of a sequence (one ticket counter per sequence; no CTA waits for another)
// walks its tree. Node c > 0 is a match when its drafted token equals the argmax of its parent's row;
// the lowest matching child of every node is found for all nodes at once (atomicMin in shared
// memory), and the walk from node 0 follows those children. Sequences finish independently, so a
// batch's walks overlap the scan of the others.
// Bound by the logits' bytes from about 64 rows of 32K on, by latency below: 17 rows of 131072 in 5.7 us (1.6 TB/s;
// the chain's acceptance of the same logits 5.9), 496 rows of 32000 in 14.7 us (4.3 TB/s).
#include "argmax.cuh"
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;     // float4 loads in flight per thread
constexpr int kNodes = VFY_MAX_TREE_NODES;
static_assert(kNodes <= kThreads, "the walk takes one node per thread");

__global__ void __launch_bounds__(kThreads) accept_tree_kernel(const AcceptTreeParams p) {
  __shared__ unsigned long long warp_best[kThreads / 32];
  __shared__ int s_target[kNodes], s_child[kNodes], s_token[kNodes], s_path[kNodes];
  __shared__ bool s_last;
  __shared__ int s_len;
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int total = p.cu_rows[p.num_seqs];
  // A ticket counter returns to zero only if every row of its sequence is scanned by somebody, which
  // holds for ascending offsets: with any others every CTA leaves before it touches the workspace.
  // Sequences whose rows cannot be used are skipped by all their CTAs, and reported once.
  bool unordered = p.cu_rows[0] < 0;
  for (int x = threadIdx.x; x < p.num_seqs; x += kThreads) {
    const int c0 = p.cu_rows[x], c1 = p.cu_rows[x + 1];
    unordered = unordered || c1 < c0;
    if (row == 0 && blockIdx.x == 0 && (c0 < x || c1 - c0 < 1 || c1 - c0 > kNodes || c1 > p.max_rows))
      atomicOr(p.err, kErrDeviceInput);
  }
  if (__syncthreads_or(unordered) || row >= total) return;
  int lo = 0, hi = p.num_seqs - 1;               // the sequence owning this row (cu_rows ascending)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_rows[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  const int r0 = p.cu_rows[b], r1 = p.cu_rows[b + 1];
  const int n = r1 - r0;
  // (r0 < b: an earlier sequence has no row, and the drafts of this one would start before the list)
  if (n < 1 || n > kNodes || r0 < b || r1 > p.max_rows || row < r0 || row >= r1) return;

  // ---- phase 1: the best key of entries [v0, v1) of the row ----
  const int v0 = min(p.vocab, static_cast<int>(blockIdx.x) * p.seg);
  const int v1 = min(p.vocab, v0 + p.seg);
  const float* src = p.logits + static_cast<size_t>(row) * p.vocab;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(src + v0) >> 2) & 3);
  const int a0 = min(v1, v0 + ((4 - mis) & 3));    // first 16-byte aligned entry
  const int n4 = (v1 - a0) >> 2;
  unsigned long long best = scan_words<kThreads, kUnroll>(reinterpret_cast<const float4*>(src + a0), n4, a0);
  if (threadIdx.x < 8) {                           // at most 3 entries before and 3 after the words
    const int x = static_cast<int>(threadIdx.x), i = x < 4 ? v0 + x : a0 + 4 * n4 + x - 4;
    if (threadIdx.x < 4 ? i < a0 : i < v1) best = umax64(best, pack(src[i], i));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = umax64(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) warp_best[warp] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) best = umax64(best, warp_best[w]);
    atomicMax(p.keys + row, best);
    // Ticket of the sequence: the add releases this CTA's key, the last CTA acquires the others'.
    unsigned int ticket;
    asm volatile("atom.add.release.gpu.global.u32 %0, [%1], 1;" : "=r"(ticket) : "l"(p.counters + b) : "memory");
    s_last = ticket == static_cast<unsigned int>(n) * gridDim.x - 1u;
  }
  __syncthreads();
  if (!s_last) return;
  asm volatile("fence.acq_rel.gpu;" ::: "memory");

  // ---- phase 2: the walk (one node per thread) ----
  const int i = threadIdx.x;
  int parent = -1;
  if (i < n) {
    s_target[i] = unpack_index(__ldcg(p.keys + r0 + i));
    s_child[i] = kNodes;
    if (i > 0) {
      parent = p.parents[r0 + i];
      s_token[i] = p.drafts[r0 - b + i - 1];
      if (parent < -1 || parent >= i) {
        atomicOr(p.err, kErrDeviceInput);
        parent = -1;
      }
    }
  }
  __syncthreads();
  if (parent >= 0 && s_token[i] == s_target[parent]) atomicMin(&s_child[parent], i);
  __syncthreads();
  if (i == 0) {
    int len = 0, node = 0;
    s_path[0] = 0;
    while (s_child[node] < kNodes) {               // a child's index is above its parent's: it ends
      node = s_child[node];
      s_path[++len] = node;
    }
    s_len = len;
  }
  __syncthreads();
  const int len = s_len;
  if (i < n) {
    p.path[r0 + i] = i <= len ? s_path[i] : -1;
    p.committed[r0 + i] = i < len ? s_token[s_path[i + 1]] : i == len ? s_target[s_path[i]] : -1;
    p.keys[r0 + i] = 0ull;                         // leave the workspace as this call found it
  }
  if (i == 0) {
    p.accepted_len[b] = len;
    p.bonus[b] = s_target[s_path[len]];
    p.counters[b] = 0u;
  }
}

}  // namespace

cudaError_t launch_accept_tree(const AcceptTreeParams& p, cudaStream_t stream) {
  return launch_pdl(accept_tree_kernel, dim3(p.parts, p.max_rows), dim3(kThreads), 0, stream, p);
}

}  // namespace vfy
