// Trees of drafted tokens: the row masks of a block's nodes, and the compaction of an accepted path.
//
// tree_plan: node i attends itself and its ancestors, mask_i = {i} + mask_parent(i), and its depth is
// |mask_i| - 1. One CTA per sequence, one thread per node, all masks in shared memory. In round r a
// node takes over the mask of the node its jump pointer names and that node's jump pointer, so its
// mask covers 2^r generations: ceil(log2(depth + 1)) rounds. The call is bound by the latency of
// its two dependent loads and the rounds (a few bytes per node).
//
// compact: the row at position p0 + path[j] moves to p0 + j (j = 1 .. n) in every layer. path is
// ascending with path[j] >= j, so a row is read at or behind the place it is written to: a thread that
// owns one 16-byte word of the row and takes the rows in order, some loads ahead of their stores,
// never reads a word that it has overwritten, and no two threads share a word. One CTA covers one
// (sequence, layer, part of the words); the rows' places come from one pass over the path, kept in
// shared memory. The call moves a few KB per layer and is latency-bound: path -> chunk -> slot ->
// row, three dependent loads (two for rings), then the copy: 30 rings 2.7 us, 10 pools of 8 sequences 4.0 us (in a
// graph; the host needs 21 and 23 us to name that many layers from Python).
#include "ptx.cuh"
#include "vfy_internal.cuh"

namespace vfy {
namespace {

constexpr int kNodes = VFY_MAX_TREE_NODES;
constexpr int kWords = VFY_TREE_WORDS;

__global__ void __launch_bounds__(kNodes) tree_plan_kernel(const TreePlanParams p) {
  __shared__ uint32_t s_mask[kWords][kNodes];
  __shared__ int s_jump[kNodes];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x;
  const int r0 = p.cu_q[b];
  const int nq = p.cu_q[b + 1] - r0;
  const int i = threadIdx.x;
  if (nq < 0 || nq > p.max_q || r0 < 0 || r0 > p.token_cap - nq) {
    if (i == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const bool mine = i < nq;
  uint32_t m[kWords];
  int jump = -1;
  if (mine) {
    jump = p.parents[r0 + i];
    if (jump < -1 || jump >= i) {
      atomicOr(p.err, kErrDeviceInput);
      jump = -1;
    }
  }
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    m[w] = (i >> 5) == w ? 1u << (i & 31) : 0u;
    s_mask[w][i] = m[w];
  }
  s_jump[i] = jump;
  while (__syncthreads_or(jump >= 0)) {
    int next = -1;
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) m[w] |= s_mask[w][jump];
      next = s_jump[jump];
    }
    __syncthreads();
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) s_mask[w][i] = m[w];
      s_jump[i] = next;
    }
    jump = next;
  }
  if (!mine) return;
  int bits = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w) bits += __popc(m[w]);
  p.depth[r0 + i] = bits - 1;
  uint4* dst = reinterpret_cast<uint4*>(p.mask + static_cast<size_t>(r0 + i) * kWords);
  dst[0] = make_uint4(m[0], m[1], m[2], m[3]);
  dst[1] = make_uint4(m[4], m[5], m[6], m[7]);
}

constexpr int kCompactThreads = 128;
constexpr int kAhead = 8;       // rows loaded before the first of them is stored

template <bool RING>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
  // Places of row j in units of head rows (head 0); full layers: of the source in the pool or, where
  // the source's chunk has no slot, in the store; of the destination in the store and the pool (-1: none).
  __shared__ long long s_src[kNodes], s_dst[kNodes], s_store[kNodes];
  __shared__ bool s_from_store[kNodes];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.z, layer = blockIdx.y;
  const int q0 = p.cu_q[b];
  const int nq = p.cu_q[b + 1] - q0;
  const int L = p.seq_len[b];
  int n = p.accepted[b];
  const bool report = blockIdx.x == 0 && layer == 0;
  if (nq < 1 || nq > p.max_q || q0 < 0 || q0 > p.token_cap - nq || L < nq || n < 0 || n >= nq) {
    if (report && threadIdx.x == 0) atomicOr(p.err, kErrDeviceInput);
    return;
  }
  const long long p0 = static_cast<long long>(L) - nq;
  const int phi = RING ? ((p.ring_off[b] % p.ring_len) + p.ring_len) % p.ring_len : 0;
  for (int j = 1 + threadIdx.x; j <= n; j += kCompactThreads) {
    const int node = p.path[q0 + j];
    long long src = -1, dst = -1, store = -1;
    bool from_store = false;
    if (node < j || node >= nq) {
      if (report) atomicOr(p.err, kErrDeviceInput);
    } else if (node == j) {
      // in place already
    } else if (RING) {
      src = static_cast<long long>(b) * p.hkv * p.ring_len + (p0 + node + phi) % p.ring_len;
      dst = static_cast<long long>(b) * p.hkv * p.ring_len + (p0 + j + phi) % p.ring_len;
    } else {
      const long long c0 = p.cu_chunks[b];
      const long long cs = c0 + (p0 + node) / kChunk, cd = c0 + (p0 + j) / kChunk;
      if (c0 < 0 || cs >= p.num_host_chunks) {
        if (report) atomicOr(p.err, kErrDeviceInput);
      } else {
        const int ss = p.slot_of_chunk[cs], sd = p.slot_of_chunk[cd];
        from_store = ss < 0 || ss >= p.num_slots;
        src = (from_store ? cs : ss) * static_cast<long long>(p.hkv) * kChunk + (p0 + node) % kChunk;
        store = cd * p.hkv * kChunk + (p0 + j) % kChunk;
        dst = sd >= 0 && sd < p.num_slots ? static_cast<long long>(sd) * p.hkv * kChunk + (p0 + j) % kChunk : -1;
      }
    }
    s_src[j] = src;
    s_dst[j] = dst;
    s_store[j] = store;
    s_from_store[j] = from_store;
  }
  __syncthreads();
  const int w_head = p.head_dim / 8;                  // 16-byte words per head row
  const int words = p.hkv * w_head;                   // per K (or V) row of a token
  const int x = blockIdx.x * kCompactThreads + threadIdx.x;
  if (x >= 2 * words) return;
  const int kv = x >= words ? 1 : 0;
  const int h = (x - kv * words) / w_head, c = (x - kv * words) - h * w_head;
  const long long head = static_cast<long long>(h) * (RING ? p.ring_len : kChunk);
  uint4* dst = reinterpret_cast<uint4*>(p.dst[layer][kv]);
  uint4* store = RING ? nullptr : reinterpret_cast<uint4*>(p.store[layer][kv]);
  for (int j0 = 1; j0 <= n; j0 += kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (j <= n && s_src[j] >= 0) {
        const uint4* from = !RING && s_from_store[j] ? store : dst;
        v[u] = from[(s_src[j] + head) * w_head + c];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j > n || s_src[j] < 0) continue;
      if (s_dst[j] >= 0) dst[(s_dst[j] + head) * w_head + c] = v[u];
      if (!RING && s_store[j] >= 0) store[(s_store[j] + head) * w_head + c] = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream) {
  return launch_pdl(tree_plan_kernel, dim3(p.num_seqs), dim3(kNodes), 0, stream, p);
}

cudaError_t launch_compact(bool ring, const CompactParams& p, cudaStream_t stream) {
  const int words = 2 * p.hkv * (p.head_dim / 8);
  dim3 grid((words + kCompactThreads - 1) / kCompactThreads, p.num_layers, p.num_seqs);
  if (ring) return launch_pdl(compact_kernel<true>, grid, dim3(kCompactThreads), 0, stream, p);
  return launch_pdl(compact_kernel<false>, grid, dim3(kCompactThreads), 0, stream, p);
}

}  // namespace vfy
