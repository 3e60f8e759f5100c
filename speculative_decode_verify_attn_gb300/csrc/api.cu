// Host side of the C ABI: context and workspace, argument validation, tensor maps, launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "ptx.cuh"
#include "vfy_internal.cuh"

struct vfy_ctx {
  vfy_config cfg;
  int device;
  int num_sms;
  float scale;
  // split partials
  float* part_o;
  float* part_ml;
  // acceptance workspace
  unsigned long long* accept_keys;
  int accept_rows_cap;
  unsigned int* accept_counter;
  unsigned int* tree_counters;   // one per sequence (tree acceptance)
  vfy::TreePiece* tree_pieces;   // items cut between CTA pairs (tree attention)
  // sampled acceptance: row statistics, race keys, tickets
  float4* sample_stats;
  unsigned long long* sample_keys;
  unsigned int* sample_counters;
  // sticky device error word
  int* err;
  int full_splits;   // 0 = automatic
  int swa_splits;
  unsigned long long launches;   // kernels enqueued through this context
  int row_tiles;                 // ceil(max_queries_per_seq * G / 128)
  unsigned long long timeout_test_ns;   // see vfy_test_wait_timeout
  int stable_metadata;                // see vfy_set_stable_metadata
  int pagein_ctas;                    // see vfy_set_pagein_ctas (0 = 2)
};

namespace {

using vfy::kChunk;
using vfy::kMaxRows;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// 2-D view [rows][d] of a bf16 array; 64 x 64 boxes (128 bytes wide) with the 128-byte swizzle.
bool make_tmap(CUtensorMap* map, const void* base, uint64_t rows, int d) {
  EncodeTiledFn enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[2] = {64, 64};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Makes the context's device current for the duration of a call and restores the caller's.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      ok = false;
      prev = -1;
      return;
    }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

// Largest vocabulary of the calls that step over it in whole segments (32-bit indices do not wrap).
constexpr int kMaxVocab = 1 << 30;
constexpr long long kSampleCtas = 4;    // CTAs per SM of the sampled acceptance's row statistics

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Nodes of one sequence's tree that a context takes, and their row tiles.
int tree_capacity(const vfy_config& c) { return std::min(c.max_queries_per_seq, VFY_MAX_TREE_NODES); }
int tree_row_tiles(const vfy_config& c) {
  return ceil_div(static_cast<long long>(tree_capacity(c)) * (c.num_q_heads / c.num_kv_heads), kMaxRows);
}
// Can a context's trees go to CTA pairs at all (see tree_pairs)? Only then does it hold their partials (20 MB).
constexpr int kPairSeqs = 4;
bool pairs_possible(const vfy_config& c) {
  return c.head_dim == 128 && (tree_row_tiles(c) > 1 || c.max_seqs >= kPairSeqs);
}

}  // namespace

#define VFY_REQUIRE(c)           \
  do {                           \
    if (!(c)) return VFY_EINVAL; \
  } while (0)

#define VFY_CUDA(call)           \
  do {                           \
    if ((call) != cudaSuccess) { \
      (void)cudaGetLastError();  \
      return VFY_ECUDA;          \
    }                            \
  } while (0)

extern "C" {

unsigned long long vfy_launch_count(const vfy_ctx* ctx) { return ctx != nullptr ? ctx->launches : 0ull; }

const char* vfy_strerror(vfy_status s) {
  switch (s) {
    case VFY_OK: return "ok";
    case VFY_EINVAL: return "invalid argument";
    case VFY_ECUDA: return "CUDA runtime error";
    case VFY_ENOMEM: return "out of device memory";
    case VFY_EUNSUPPORTED: return "unsupported device or configuration";
    case VFY_EDEVICE_INPUT: return "a device-side list or length was out of range (element skipped)";
    case VFY_EDEVICE_TIMEOUT: return "a bounded device wait ran out";
  }
  return "unknown status";
}

vfy_status vfy_create(const vfy_config* cfg_in, int device, vfy_ctx** out) {
  VFY_REQUIRE(cfg_in != nullptr && out != nullptr);
  *out = nullptr;
  const vfy_config cfg = *cfg_in;
  VFY_REQUIRE(cfg.num_q_heads >= 1 && cfg.num_kv_heads >= 1 && cfg.num_q_heads % cfg.num_kv_heads == 0);
  VFY_REQUIRE(cfg.head_dim == 64 || cfg.head_dim == 128);
  VFY_REQUIRE(cfg.chunk_tokens == kChunk);
  VFY_REQUIRE(cfg.max_seqs >= 1 && cfg.max_queries_per_seq >= 1 && cfg.max_splits >= 1);
  VFY_REQUIRE(cfg.max_splits <= 64 && cfg.max_seqs <= 65535 && cfg.num_kv_heads <= 65535);
  const int group = cfg.num_q_heads / cfg.num_kv_heads;
  VFY_REQUIRE(static_cast<long long>(cfg.max_queries_per_seq) * group <= static_cast<long long>(kMaxRows) * vfy::kMaxRowTiles);
  VFY_REQUIRE(cfg.window >= 1 && cfg.ring_len >= kChunk && cfg.ring_len % kChunk == 0);
  // The ring must hold the union window of a block plus one tile of slack, so that the
  // slot-aligned tiles covering it are distinct.
  VFY_REQUIRE(static_cast<long long>(cfg.window) + cfg.max_queries_per_seq - 1 + kChunk <= cfg.ring_len);
  VFY_REQUIRE(cfg.softmax_scale >= 0.f && std::isfinite(cfg.softmax_scale));

  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) {
    (void)cudaGetLastError();
    return VFY_EINVAL;
  }
  cudaDeviceProp prop;
  VFY_CUDA(cudaGetDeviceProperties(&prop, device));
  if (!(prop.major == 10 && prop.minor == 3)) return VFY_EUNSUPPORTED;   // sm_103 only

  DeviceGuard guard(device);
  if (!guard.ok) return VFY_ECUDA;
  if (get_encode() == nullptr) return VFY_EUNSUPPORTED;
  vfy_ctx* ctx = new (std::nothrow) vfy_ctx();
  if (ctx == nullptr) return VFY_ENOMEM;
  ctx->cfg = cfg;
  ctx->device = device;
  ctx->num_sms = prop.multiProcessorCount;
  ctx->scale = cfg.softmax_scale > 0.f ? cfg.softmax_scale : 1.0f / std::sqrt(static_cast<float>(cfg.head_dim));

  ctx->row_tiles = ceil_div(static_cast<long long>(cfg.max_queries_per_seq) * group, kMaxRows);
  size_t parts = static_cast<size_t>(cfg.max_seqs) * ctx->row_tiles * cfg.num_kv_heads * cfg.max_splits * kMaxRows;
  // tree attention by CTA pairs: two partial segments of two row tiles for every two SMs
  if (pairs_possible(cfg)) parts = std::max(parts, static_cast<size_t>(ctx->num_sms) * 2 * kMaxRows);
  ctx->accept_rows_cap = cfg.max_seqs * cfg.max_queries_per_seq;
  bool ok = cudaMalloc(&ctx->part_o, parts * cfg.head_dim * sizeof(float)) == cudaSuccess &&
            cudaMalloc(&ctx->part_ml, parts * 2 * sizeof(float)) == cudaSuccess &&
            cudaMalloc(&ctx->accept_keys, ctx->accept_rows_cap * sizeof(unsigned long long)) == cudaSuccess &&
            cudaMalloc(&ctx->accept_counter, sizeof(unsigned int)) == cudaSuccess &&
            cudaMalloc(&ctx->tree_counters, cfg.max_seqs * sizeof(unsigned int)) == cudaSuccess &&
            cudaMalloc(&ctx->tree_pieces, ctx->num_sms * sizeof(vfy::TreePiece)) == cudaSuccess &&
            cudaMalloc(&ctx->sample_stats, (ctx->accept_rows_cap + kSampleCtas * ctx->num_sms) * sizeof(float4)) == cudaSuccess &&
            cudaMalloc(&ctx->sample_keys, cfg.max_seqs * sizeof(unsigned long long)) == cudaSuccess &&
            cudaMalloc(&ctx->sample_counters, cfg.max_seqs * sizeof(unsigned int)) == cudaSuccess &&
            cudaMalloc(&ctx->err, sizeof(int)) == cudaSuccess;
  if (ok)
    ok = cudaMemset(ctx->accept_keys, 0, ctx->accept_rows_cap * sizeof(unsigned long long)) == cudaSuccess &&
         cudaMemset(ctx->accept_counter, 0, sizeof(unsigned int)) == cudaSuccess &&
         cudaMemset(ctx->tree_counters, 0, cfg.max_seqs * sizeof(unsigned int)) == cudaSuccess &&
         cudaMemset(ctx->sample_keys, 0, cfg.max_seqs * sizeof(unsigned long long)) == cudaSuccess &&
         cudaMemset(ctx->sample_counters, 0, cfg.max_seqs * sizeof(unsigned int)) == cudaSuccess &&
         cudaMemset(ctx->err, 0, sizeof(int)) == cudaSuccess &&
         cudaMemset(ctx->part_ml, 0, parts * 2 * sizeof(float)) == cudaSuccess &&
         cudaDeviceSynchronize() == cudaSuccess;
  if (!ok) {
    (void)cudaGetLastError();
    vfy_destroy(ctx);
    return VFY_ENOMEM;
  }
  *out = ctx;
  return VFY_OK;
}

void vfy_destroy(vfy_ctx* ctx) {
  if (ctx == nullptr) return;
  {
    DeviceGuard guard(ctx->device);
    cudaDeviceSynchronize();
    cudaFree(ctx->part_o);
    cudaFree(ctx->part_ml);
    cudaFree(ctx->accept_keys);
    cudaFree(ctx->accept_counter);
    cudaFree(ctx->tree_counters);
    cudaFree(ctx->tree_pieces);
    cudaFree(ctx->sample_stats);
    cudaFree(ctx->sample_keys);
    cudaFree(ctx->sample_counters);
    cudaFree(ctx->err);
    (void)cudaGetLastError();
  }
  delete ctx;
}

vfy_status vfy_get_status(vfy_ctx* ctx, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int word = 0;
  VFY_CUDA(cudaStreamSynchronize(s));
  VFY_CUDA(cudaMemcpy(&word, ctx->err, sizeof(int), cudaMemcpyDeviceToHost));
  VFY_CUDA(cudaMemset(ctx->err, 0, sizeof(int)));
  VFY_CUDA(cudaDeviceSynchronize());
  if (word & vfy::kErrTimeout) return VFY_EDEVICE_TIMEOUT;
  if (word & vfy::kErrDeviceInput) return VFY_EDEVICE_INPUT;
  return VFY_OK;
}

vfy_status vfy_set_splits(vfy_ctx* ctx, int full_splits, int swa_splits) {
  VFY_REQUIRE(ctx != nullptr);
  VFY_REQUIRE(full_splits >= 0 && full_splits <= ctx->cfg.max_splits);
  VFY_REQUIRE(swa_splits >= 0 && swa_splits <= ctx->cfg.max_splits);
  ctx->full_splits = full_splits;
  ctx->swa_splits = swa_splits;
  return VFY_OK;
}

vfy_status vfy_set_pagein_ctas(vfy_ctx* ctx, int ctas_per_chunk) {
  VFY_REQUIRE(ctx != nullptr && ctas_per_chunk >= 0 && ctas_per_chunk <= vfy::kMaxPageInCtas);
  ctx->pagein_ctas = ctas_per_chunk;
  return VFY_OK;
}

vfy_status vfy_test_wait_timeout(vfy_ctx* ctx, uint64_t limit_ns) {
  VFY_REQUIRE(ctx != nullptr);
  ctx->timeout_test_ns = limit_ns;
  return VFY_OK;
}

vfy_status vfy_set_stable_metadata(vfy_ctx* ctx, int stable) {
  VFY_REQUIRE(ctx != nullptr && (stable == 0 || stable == 1));
  ctx->stable_metadata = stable;
  return VFY_OK;
}

vfy_status vfy_select_resident(vfy_ctx* ctx, const float* scores, const int32_t* cu_chunks, int num_seqs,
                               int max_chunks_per_seq, int k, int32_t* slot_of_chunk, int32_t* resident_ids,
                               int32_t* resident_slots, int32_t* cu_resident, int32_t* pagein_list,
                               int32_t* pagein_count, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && scores != nullptr && cu_chunks != nullptr && slot_of_chunk != nullptr);
  VFY_REQUIRE(resident_ids != nullptr && resident_slots != nullptr && cu_resident != nullptr);
  VFY_REQUIRE(pagein_list != nullptr && pagein_count != nullptr);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(k >= 1 && k <= vfy::kMaxSelectK);
  VFY_REQUIRE(max_chunks_per_seq >= 0 && max_chunks_per_seq <= vfy::kMaxSelectChunks);
  VFY_REQUIRE(static_cast<long long>(num_seqs) * k <= INT_MAX / 2);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::SelectParams p;
  p.scores = scores;
  p.cu_chunks = cu_chunks;
  p.num_seqs = num_seqs;
  p.max_n = max_chunks_per_seq;
  p.k = k;
  p.slot_of_chunk = slot_of_chunk;
  p.res_ids = resident_ids;
  p.res_slots = resident_slots;
  p.cu_res = cu_resident;
  p.pagein_list = pagein_list;
  p.pagein_count = pagein_count;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_select(p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

// Outside stream capture: check that a caller's "host" buffers are addressable by the device
// (pinned, managed or device memory) and translate pinned host pointers to their device
// addresses. During capture the check is skipped (the pointers are used as given).
static vfy_status device_view(cudaStream_t s, void** ptrs, int n) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) return VFY_ECUDA;
  if (cap != cudaStreamCaptureStatusNone) return VFY_OK;
  for (int i = 0; i < n; ++i) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, ptrs[i]) != cudaSuccess) {
      (void)cudaGetLastError();
      return VFY_EINVAL;
    }
    if (a.type == cudaMemoryTypeUnregistered) return VFY_EINVAL;
    if (a.type == cudaMemoryTypeHost && a.devicePointer != nullptr) ptrs[i] = a.devicePointer;
  }
  return VFY_OK;
}

vfy_status vfy_page_in(vfy_ctx* ctx, const uint16_t* host_k, const uint16_t* host_v, int64_t num_host_chunks,
                       uint16_t* k_pool, uint16_t* v_pool, int num_slots, const int32_t* pagein_list,
                       const int32_t* pagein_count, int num_seqs, int k, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && host_k != nullptr && host_v != nullptr && k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(pagein_list != nullptr && pagein_count != nullptr);
  VFY_REQUIRE(aligned16(host_k) && aligned16(host_v) && aligned16(k_pool) && aligned16(v_pool));
  VFY_REQUIRE(num_host_chunks >= 1 && num_host_chunks <= INT_MAX && num_slots >= 1);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs && k >= 1 && k <= vfy::kMaxSelectK);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* dev_ptr[2] = {const_cast<uint16_t*>(host_k), const_cast<uint16_t*>(host_v)};
  const vfy_status st = device_view(s, dev_ptr, 2);
  if (st != VFY_OK) return st;
  vfy::PageInParams p;
  p.host_k = static_cast<const uint16_t*>(dev_ptr[0]);
  p.host_v = static_cast<const uint16_t*>(dev_ptr[1]);
  p.num_host_chunks = num_host_chunks;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.num_slots = num_slots;
  p.list = pagein_list;
  p.count = pagein_count;
  p.num_seqs = num_seqs;
  p.k = k;
  p.chunk_elems = static_cast<long long>(ctx->cfg.num_kv_heads) * kChunk * ctx->cfg.head_dim;
  p.err = ctx->err;
  p.parts = ctx->pagein_ctas > 0 ? ctx->pagein_ctas : 2;
  VFY_CUDA(vfy::launch_page_in(p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_append_full(vfy_ctx* ctx, const uint16_t* k_new, const uint16_t* v_new, const int32_t* cu_q,
                           const int32_t* seq_len, const int32_t* cu_chunks, const int32_t* slot_of_chunk,
                           uint16_t* host_k, uint16_t* host_v, int64_t num_host_chunks, uint16_t* k_pool,
                           uint16_t* v_pool, int num_slots, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && k_new != nullptr && v_new != nullptr && cu_q != nullptr && seq_len != nullptr);
  VFY_REQUIRE(cu_chunks != nullptr && slot_of_chunk != nullptr && host_k != nullptr && host_v != nullptr);
  VFY_REQUIRE(k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(aligned16(k_new) && aligned16(v_new) && aligned16(host_k) && aligned16(host_v) &&
              aligned16(k_pool) && aligned16(v_pool));
  VFY_REQUIRE(num_host_chunks >= 1 && num_host_chunks <= INT_MAX && num_slots >= 1);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* store[2] = {host_k, host_v};
  const vfy_status st = device_view(s, store, 2);
  if (st != VFY_OK) return st;
  vfy::AppendParams p = {};
  p.k_new = k_new;
  p.v_new = v_new;
  p.cu_q = cu_q;
  p.seq_len = seq_len;
  p.num_seqs = num_seqs;
  p.max_q = ctx->cfg.max_queries_per_seq;
  p.token_cap = num_seqs * ctx->cfg.max_queries_per_seq;
  p.hkv = ctx->cfg.num_kv_heads;
  p.head_dim = ctx->cfg.head_dim;
  p.cu_chunks = cu_chunks;
  p.slot_of_chunk = slot_of_chunk;
  p.host_k = static_cast<uint16_t*>(store[0]);
  p.host_v = static_cast<uint16_t*>(store[1]);
  p.num_host_chunks = num_host_chunks;
  p.num_slots = num_slots;
  p.k_dst = k_pool;
  p.v_dst = v_pool;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_append(false, p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_append_swa(vfy_ctx* ctx, const uint16_t* k_new, const uint16_t* v_new, const int32_t* cu_q,
                          const int32_t* seq_len, const int32_t* ring_offset, uint16_t* k_ring, uint16_t* v_ring,
                          int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && k_new != nullptr && v_new != nullptr && cu_q != nullptr && seq_len != nullptr);
  VFY_REQUIRE(ring_offset != nullptr && k_ring != nullptr && v_ring != nullptr);
  VFY_REQUIRE(aligned16(k_new) && aligned16(v_new) && aligned16(k_ring) && aligned16(v_ring));
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::AppendParams p = {};
  p.k_new = k_new;
  p.v_new = v_new;
  p.cu_q = cu_q;
  p.seq_len = seq_len;
  p.num_seqs = num_seqs;
  p.max_q = ctx->cfg.max_queries_per_seq;
  p.token_cap = num_seqs * ctx->cfg.max_queries_per_seq;
  p.hkv = ctx->cfg.num_kv_heads;
  p.head_dim = ctx->cfg.head_dim;
  p.ring_off = ring_offset;
  p.ring_len = ctx->cfg.ring_len;
  p.k_dst = k_ring;
  p.v_dst = v_ring;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_append(true, p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

// Does a tree's full layer go to CTA pairs of 256 rows (and how many), or to the linear block's kernel (0)?
// Pairs balance whatever the lengths, and halve the K/V traffic of two row tiles; each run pays about 8 us for its
// start and the merge. us of one layer, 4 KV heads, the linear kernel with its best splits against pairs:
//   two row tiles (64 nodes, G = 4), 32 chunks: 8 sequences 28.0 / 27.9, 12: 28.2 / 32.4; 64 chunks: 1: 14.9 / 17.8,
//   2: 19.5 / 23.4, 4: 26.9 / 26.3, 8: 43.8 / 32.4, 16: 46.8 / 48.5, 16 ragged: 46.3 / 41.3; 128 chunks: 1: 18.5 / 19.7;
//   256 chunks: 1: 22.5 / 22.1, 4: 55 / 41, 16: 160 / 99; 1024 chunks: 8: 264 / 162;
//   one row tile (17 nodes), 256 chunks: 2 sequences 19.6 / 25.9, 4: 31.6 / 35.5, 8: 54 / 54, 16: 97 / 83;
//   1024 chunks: 2: 57 / 64, 8: 168 / 157, 8 ragged (750 chunks at most): 105 / 98, and 130 with one wave of splits,
//   which is the best for equal lengths.
// The rule is coarser than the table and takes pairs at three of its points where they are slower: one sequence, two
// row tiles, 128 chunks (1.2 us); four sequences, one row tile, 256 chunks (3.9); 16 equal sequences, two row tiles,
// 64 chunks (1.7, where ragged ones gain 5.0). Row tiles are those of the context's capacity, not of the block. The
// table is for 4 KV heads; the pair kernel is written for d = 128.
static int tree_pairs(const vfy_ctx* ctx, int row_tiles, int num_seqs, int max_res) {
  if (ctx->full_splits != 0 || !pairs_possible(ctx->cfg)) return 0;
  const long long items = static_cast<long long>(ctx->cfg.num_kv_heads) * num_seqs * row_tiles;
  // (pairs_possible names what this rule asks of a context)
  const bool take = row_tiles > 1 ? max_res >= 128 || (max_res >= 48 && items >= 32)
                                  : num_seqs >= kPairSeqs && max_res >= 256;
  return take ? std::min(vfy::attend_tree_pairs(), ctx->num_sms / 2) : 0;
}

static vfy_status attend_common(vfy_ctx* ctx, bool ring, const uint16_t* q, const int32_t* cu_q,
                                const uint16_t* k_src, const uint16_t* v_src, uint64_t src_rows,
                                const int32_t* ids, const int32_t* slots, const int32_t* cu_res, int num_slots,
                                int max_res, const int32_t* ring_offset, const int32_t* seq_len, uint16_t* out,
                                float* lse, int num_seqs, vfy_stream_t stream,
                                const uint32_t* tree_mask = nullptr, const int32_t* tree_depth = nullptr) {
  const vfy_config& c = ctx->cfg;
  const bool tree = tree_mask != nullptr;
  const int max_q = tree ? tree_capacity(c) : c.max_queries_per_seq;
  const int row_tiles = tree ? tree_row_tiles(c) : ctx->row_tiles;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  CUtensorMap tk, tv;
  if (!make_tmap(&tk, k_src, src_rows, c.head_dim) || !make_tmap(&tv, v_src, src_rows, c.head_dim))
    return VFY_EINVAL;
  const int hkv = c.num_kv_heads;
  int splits;
  if (!ring) {
    splits = ctx->full_splits;
    if (splits == 0) {
      if (tree && (row_tiles > 1 || num_seqs > 1)) {   // (else as the linear block: a chain has its bits)
        // One wave of CTAs: us with one wave against four of 17 nodes over 64 chunks, 4 sequences 15.3 / 31.9, 8
        // 22.3 / 36.4, 16 35.3 / 47.1. Long contexts of a batch (here with d = 64; with d = 128 CTA pairs take them)
        // get two waves, for sequences of different lengths: 8 of equal lengths over 256 chunks 25.0 / 27.3.
        const long long items = static_cast<long long>(hkv) * num_seqs * row_tiles;
        splits = static_cast<int>(ctx->num_sms * (num_seqs >= 4 && max_res >= 256 ? 2 : 1) / items);
        // Short contexts: as many as one cluster merges in the attention kernel, which with 16 splits finds too few
        // GPCs (64 chunks, 8 items: 12 splits 11.9 us, 16 20.6, 19 and the combine 13.5).
        if (max_res <= 64) splits = std::min(splits, 12);
      } else if (row_tiles > 1) {
        // Blocks of several row tiles (prefill-shaped) have (KV head, row tile) items enough to
        // fill the SMs with few splits, and a long split keeps the tensor pipe busier: at most one
        // wave. Measured with 1024 queries over 128 chunks (128 items): 1 split 121 us, 2 splits
        // 130, 3 138, 4 146, 5 (four waves) 155.
        splits = ctx->num_sms / (hkv * num_seqs * row_tiles);
      } else {
        // One wave of CTAs for one sequence; several waves for a batch, so that the hardware
        // scheduler can balance sequences of different lengths.
        const int target = ctx->num_sms * (num_seqs > 1 ? 4 : 1);
        splits = ceil_div(target, static_cast<long long>(hkv) * num_seqs);
      }
      splits = clampi(splits, 1, max_res > 0 ? max_res : 1);
    }
  } else {
    splits = ctx->swa_splits;
    if (splits == 0) {
      // a row tile's queries: at most 128 / G of them
      // (a tree's row tiles all take the whole block's span)
      const int tile_q = tree ? max_q : std::min(max_q, ceil_div(kMaxRows, c.num_q_heads / hkv));
      const int max_tiles = ceil_div(static_cast<long long>(kChunk - 1) + c.window + tile_q - 1, kChunk);
      // Trees take at most one wave of CTAs: a batch's (8 sequences of 64 nodes) 17.2 us with 2 splits,
      // 22.1 with 3 (192 CTAs); of 17 nodes 10.1 us with 4, 14.5 with 5 (160 CTAs).
      const long long items = static_cast<long long>(hkv) * num_seqs * row_tiles;
      const int by_sms = tree ? static_cast<int>(ctx->num_sms / items) : ceil_div(ctx->num_sms, items);
      splits = clampi(by_sms, 1, max_tiles);
      // With SMs to spare (one tile per split), two more splits than tiles: the splits without a
      // tile only take their share of the cluster merge. Measured on the 40-layer pass (10
      // tiles: 12 splits 10.27-10.29 us/layer against 10.40-10.51 for 10, 11, 13, 14 and 16).
      if (by_sms > max_tiles && max_tiles + 2 <= vfy::kMaxClusterSplits) splits = std::min(max_tiles + 2, by_sms);

    }
  }
  splits = clampi(splits, 1, c.max_splits);

  vfy::AttnParams p;
  p.q = q;
  p.cu_q = cu_q;
  p.seq_len = seq_len;
  p.res_ids = ids;
  p.res_slots = slots;
  p.cu_res = cu_res;
  p.num_slots = num_slots;
  p.ring_off = ring_offset;
  p.ring_len = c.ring_len;
  p.window = c.window;
  p.hq = c.num_q_heads;
  p.hkv = hkv;
  p.group = c.num_q_heads / hkv;
  p.num_splits = splits;
  p.max_q = max_q;
  p.row_tiles = row_tiles;
  p.scale_log2 = ctx->scale * 1.4426950408889634f;
  p.part_o = ctx->part_o;
  p.part_ml = ctx->part_ml;
  p.timeout_test_ns = ctx->timeout_test_ns;
  p.stable_metadata = ctx->stable_metadata;
  p.err = ctx->err;
  p.tree_mask = tree_mask;
  p.tree_depth = tree_depth;
  p.num_seqs = num_seqs;
  p.tree_pieces = ctx->tree_pieces;
  p.token_cap = num_seqs * c.max_queries_per_seq;      // (a tree may lie behind a longer sequence, which is left out)
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int pairs = tree && !ring ? tree_pairs(ctx, row_tiles, num_seqs, max_res) : 0;
  if (pairs > 0) {
    p.out = out;
    p.lse = lse;
    VFY_CUDA(vfy::launch_attend_tree(p, tk, tv, pairs, s));
    ctx->launches += 2;
    return VFY_OK;
  }
  // Full-layer splits over many resident chunks take wide tiles (their combine is a small part
  // of a long split). Otherwise up to kMaxClusterSplits splits (and no more than one GPC holds)
  // merge inside the attention kernel, as one thread-block cluster per (sequence, KV head, row
  // tile); more go through the combine.
  const bool wide = !ring && ceil_div(max_res > 0 ? max_res : 1, splits) >= vfy::kWideMinChunks;
  // A single split of a long block writes O itself (no combine launch).
  const bool direct = wide && splits == 1;
  const bool merge = !direct && !wide && splits <= vfy::kMaxClusterSplits &&
                     splits <= vfy::attend_merge_limit(ring, c.head_dim, tree);
  const vfy::AttnTiles tiles = merge    ? vfy::AttnTiles::kMerge
                              : direct ? vfy::AttnTiles::kWideDirect
                              : wide   ? vfy::AttnTiles::kWide
                                       : vfy::AttnTiles::kNarrow;
  p.out = merge || direct ? out : nullptr;
  p.lse = merge || direct ? lse : nullptr;
  VFY_CUDA(vfy::launch_attend(ring, c.head_dim, tiles, p, tk, tv, num_seqs, s));
  ++ctx->launches;
  if (merge || direct) return VFY_OK;

  vfy::CombineParams cp;
  cp.cu_q = cu_q;
  cp.seq_len = seq_len;
  cp.num_seqs = num_seqs;
  cp.hq = c.num_q_heads;
  cp.hkv = hkv;
  cp.group = p.group;
  cp.num_splits = splits;
  cp.max_q = max_q;
  cp.row_tiles = row_tiles;
  cp.token_cap = p.token_cap;
  cp.by_seq = max_q < c.max_queries_per_seq;
  cp.stable_metadata = ctx->stable_metadata;
  cp.part_o = ctx->part_o;
  cp.part_ml = ctx->part_ml;
  cp.out = out;
  cp.lse = lse;
  cp.err = ctx->err;
  VFY_CUDA(vfy::launch_combine(c.head_dim, cp, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_attend_full(vfy_ctx* ctx, const uint16_t* q, const int32_t* cu_q, const uint16_t* k_pool,
                           const uint16_t* v_pool, int num_slots, const int32_t* resident_ids,
                           const int32_t* resident_slots, const int32_t* cu_resident, int max_resident_per_seq,
                           const int32_t* seq_len, uint16_t* out, float* lse, int num_seqs,
                           vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && q != nullptr && cu_q != nullptr && k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(resident_ids != nullptr && resident_slots != nullptr && cu_resident != nullptr);
  VFY_REQUIRE(seq_len != nullptr && out != nullptr);
  VFY_REQUIRE(aligned16(q) && aligned16(k_pool) && aligned16(v_pool) && aligned16(out));
  VFY_REQUIRE(lse == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(num_slots >= 1 && max_resident_per_seq >= 0);
  const uint64_t rows = static_cast<uint64_t>(num_slots) * ctx->cfg.num_kv_heads * kChunk;
  VFY_REQUIRE(rows <= static_cast<uint64_t>(INT_MAX));
  return attend_common(ctx, false, q, cu_q, k_pool, v_pool, rows, resident_ids, resident_slots, cu_resident,
                       num_slots, max_resident_per_seq, nullptr, seq_len, out, lse, num_seqs, stream);
}

vfy_status vfy_attend_swa(vfy_ctx* ctx, const uint16_t* q, const int32_t* cu_q, const uint16_t* k_ring,
                          const uint16_t* v_ring, const int32_t* ring_offset, const int32_t* seq_len,
                          uint16_t* out, float* lse, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && q != nullptr && cu_q != nullptr && k_ring != nullptr && v_ring != nullptr);
  VFY_REQUIRE(ring_offset != nullptr && seq_len != nullptr && out != nullptr);
  VFY_REQUIRE(aligned16(q) && aligned16(k_ring) && aligned16(v_ring) && aligned16(out));
  VFY_REQUIRE(lse == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  const uint64_t rows = static_cast<uint64_t>(num_seqs) * ctx->cfg.num_kv_heads * ctx->cfg.ring_len;
  VFY_REQUIRE(rows <= static_cast<uint64_t>(INT_MAX));
  return attend_common(ctx, true, q, cu_q, k_ring, v_ring, rows, nullptr, nullptr, nullptr, 0, 0, ring_offset,
                       seq_len, out, lse, num_seqs, stream);
}

vfy_status vfy_accept(vfy_ctx* ctx, const float* logits, int vocab, const int32_t* drafts, const int32_t* cu_rows,
                      int max_rows, int32_t* accepted_len, int32_t* bonus, int32_t* committed, int num_seqs,
                      vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && logits != nullptr && drafts != nullptr && cu_rows != nullptr);
  VFY_REQUIRE(accepted_len != nullptr && bonus != nullptr && committed != nullptr);
  VFY_REQUIRE(vocab >= 1 && num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(max_rows >= 1 && max_rows <= ctx->accept_rows_cap && max_rows <= 65535);
  VFY_REQUIRE((reinterpret_cast<uintptr_t>(logits) & 3u) == 0);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::AcceptParams p;
  p.logits = logits;
  p.vocab = vocab;
  p.drafts = drafts;
  p.cu_rows = cu_rows;
  p.num_seqs = num_seqs;
  p.max_rows = max_rows;
  // About two CTAs per SM over all rows; each CTA scans a whole number of 16-byte words.
  int parts = ceil_div(2LL * ctx->num_sms, max_rows);
  parts = clampi(parts, 1, ceil_div(vocab, 1024));
  int seg = ceil_div(vocab, parts);
  seg = (seg + 3) & ~3;
  p.parts = ceil_div(vocab, seg);
  p.seg = seg;
  p.accepted_len = accepted_len;
  p.bonus = bonus;
  p.committed = committed;
  p.keys = ctx->accept_keys;
  p.counter = ctx->accept_counter;
  p.stable_metadata = ctx->stable_metadata;
  p.err = ctx->err;
  const bool vec4 = (vocab % 4 == 0) && aligned16(logits);
  VFY_CUDA(vfy::launch_accept(p, vec4, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_tree_plan(vfy_ctx* ctx, const int32_t* parents, const int32_t* cu_q, int32_t* depth,
                         uint32_t* tree_mask, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && parents != nullptr && cu_q != nullptr && depth != nullptr && tree_mask != nullptr);
  VFY_REQUIRE(aligned16(tree_mask));
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::TreePlanParams p;
  p.parents = parents;
  p.cu_q = cu_q;
  p.num_seqs = num_seqs;
  p.max_q = tree_capacity(ctx->cfg);
  p.token_cap = num_seqs * ctx->cfg.max_queries_per_seq;
  p.depth = depth;
  p.mask = tree_mask;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_tree_plan(p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_attend_full_tree(vfy_ctx* ctx, const uint16_t* q, const int32_t* cu_q, const uint32_t* tree_mask,
                                const uint16_t* k_pool, const uint16_t* v_pool, int num_slots,
                                const int32_t* resident_ids, const int32_t* resident_slots,
                                const int32_t* cu_resident, int max_resident_per_seq, const int32_t* seq_len,
                                uint16_t* out, float* lse, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && q != nullptr && cu_q != nullptr && tree_mask != nullptr);
  VFY_REQUIRE(k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(resident_ids != nullptr && resident_slots != nullptr && cu_resident != nullptr);
  VFY_REQUIRE(seq_len != nullptr && out != nullptr);
  VFY_REQUIRE(aligned16(q) && aligned16(tree_mask) && aligned16(k_pool) && aligned16(v_pool) && aligned16(out));
  VFY_REQUIRE(lse == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(num_slots >= 1 && max_resident_per_seq >= 0);
  const uint64_t rows = static_cast<uint64_t>(num_slots) * ctx->cfg.num_kv_heads * kChunk;
  VFY_REQUIRE(rows <= static_cast<uint64_t>(INT_MAX));
  return attend_common(ctx, false, q, cu_q, k_pool, v_pool, rows, resident_ids, resident_slots, cu_resident,
                       num_slots, max_resident_per_seq, nullptr, seq_len, out, lse, num_seqs, stream, tree_mask);
}

vfy_status vfy_attend_swa_tree(vfy_ctx* ctx, const uint16_t* q, const int32_t* cu_q, const uint32_t* tree_mask,
                               const int32_t* depth, const uint16_t* k_ring, const uint16_t* v_ring,
                               const int32_t* ring_offset, const int32_t* seq_len, uint16_t* out, float* lse,
                               int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && q != nullptr && cu_q != nullptr && tree_mask != nullptr && depth != nullptr);
  VFY_REQUIRE(k_ring != nullptr && v_ring != nullptr && ring_offset != nullptr && seq_len != nullptr);
  VFY_REQUIRE(out != nullptr);
  VFY_REQUIRE(aligned16(q) && aligned16(tree_mask) && aligned16(k_ring) && aligned16(v_ring) && aligned16(out));
  VFY_REQUIRE(lse == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(ctx->cfg.window >= tree_capacity(ctx->cfg));
  const uint64_t rows = static_cast<uint64_t>(num_seqs) * ctx->cfg.num_kv_heads * ctx->cfg.ring_len;
  VFY_REQUIRE(rows <= static_cast<uint64_t>(INT_MAX));
  return attend_common(ctx, true, q, cu_q, k_ring, v_ring, rows, nullptr, nullptr, nullptr, 0, 0, ring_offset,
                       seq_len, out, lse, num_seqs, stream, tree_mask, depth);
}

vfy_status vfy_process_logits(vfy_ctx* ctx, const void* logits, int logits_type, int64_t row_stride, int vocab,
                              const int32_t* cu_rows, int max_rows, const vfy_logit_rules* rules, float* out,
                              int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && logits != nullptr && cu_rows != nullptr && rules != nullptr && out != nullptr);
  VFY_REQUIRE(logits_type == VFY_LOGITS_F32 || logits_type == VFY_LOGITS_BF16);
  const bool bf16 = logits_type == VFY_LOGITS_BF16;
  VFY_REQUIRE(vocab >= 1 && vocab <= kMaxVocab && row_stride >= vocab);
  VFY_REQUIRE((reinterpret_cast<uintptr_t>(logits) & (bf16 ? 1u : 3u)) == 0);
  VFY_REQUIRE((reinterpret_cast<uintptr_t>(out) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(max_rows >= 1 && max_rows <= ctx->accept_rows_cap);
  VFY_REQUIRE(row_stride <= (INT64_MAX / 8) / max_rows);
  const vfy_logit_rules& r = *rules;
  VFY_REQUIRE(r.cu_bias == nullptr || (r.bias_token != nullptr && r.bias_value != nullptr));
  VFY_REQUIRE(r.grammar == nullptr || r.num_masks >= 1);
  VFY_REQUIRE(r.tree_mask == nullptr || aligned16(r.tree_mask));
  // In place (the same rows) or apart: the kernel reads other rows' logits after it wrote some.
  const bool same = !bf16 && static_cast<const void*>(out) == logits && row_stride == vocab;
  const uintptr_t l0 = reinterpret_cast<uintptr_t>(logits), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t l1 = l0 + (static_cast<uintptr_t>(max_rows - 1) * row_stride + vocab) * (bf16 ? 2u : 4u);
  const uintptr_t o1 = o0 + static_cast<uintptr_t>(max_rows) * vocab * 4u;
  VFY_REQUIRE(same || l1 <= o0 || o1 <= l0);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::LogitParams p;
  p.logits = logits;
  p.stride = row_stride;
  p.vocab = vocab;
  p.cu_rows = cu_rows;
  p.num_seqs = num_seqs;
  p.max_rows = max_rows;
  // About four CTAs per SM where the rows allow it, else one for all rows of a segment: each reads the
  // segment's counts and biases. (Where rows start at different places of a 16-byte word, parts that are
  // a multiple of 4 hold rows that start alike.)
  const bool even = vocab % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && row_stride % 4 == 0;
  p.segs = vfy::logit_segments(vocab, even);
  const long long ctas = static_cast<long long>(p.segs) * num_seqs;
  const int rows_per_seq = std::min(ceil_div(max_rows, num_seqs), VFY_MAX_TREE_NODES);
  p.row_parts = clampi(ceil_div(4LL * ctx->num_sms, ctas), 1, rows_per_seq);
  if (!even && p.row_parts > 1) p.row_parts = (p.row_parts + 3) & ~3;
  p.rules = r;
  p.out = out;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_process_logits(p, bf16, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_count_tokens(vfy_ctx* ctx, const int32_t* tokens, const int32_t* cu_tokens, int64_t max_tokens,
                            int as_prompt, int reset, int32_t* counts, int vocab, int num_seqs,
                            vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && tokens != nullptr && cu_tokens != nullptr && counts != nullptr);
  VFY_REQUIRE(max_tokens >= 1 && max_tokens <= INT_MAX && vocab >= 1 && vocab <= kMaxVocab);
  VFY_REQUIRE((as_prompt == 0 || as_prompt == 1) && (reset == 0 || reset == 1));
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  vfy::CountParams p;
  p.tokens = tokens;
  p.cu_tokens = cu_tokens;
  p.max_tokens = max_tokens;
  p.num_seqs = num_seqs;
  p.vocab = vocab;
  p.as_prompt = as_prompt;
  p.reset = reset;
  // A reset takes segments for about one wave of CTAs, of 1K to 8K counts (32 KB of shared memory).
  p.seg = clampi(ceil_div(static_cast<long long>(vocab) * num_seqs, ctx->num_sms), 1024, 8192);
  p.counts = counts;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_count_tokens(p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_accept_tree(vfy_ctx* ctx, const float* logits, int vocab, const int32_t* drafts,
                           const int32_t* parents, const int32_t* cu_rows, int max_rows, int32_t* accepted_len,
                           int32_t* path, int32_t* bonus, int32_t* committed, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && logits != nullptr && drafts != nullptr && parents != nullptr && cu_rows != nullptr);
  VFY_REQUIRE(accepted_len != nullptr && path != nullptr && bonus != nullptr && committed != nullptr);
  VFY_REQUIRE(vocab >= 1 && vocab <= kMaxVocab && num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(max_rows >= 1 && max_rows <= ctx->accept_rows_cap && max_rows <= 65535);
  VFY_REQUIRE((reinterpret_cast<uintptr_t>(logits) & 3u) == 0);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::AcceptTreeParams p;
  p.logits = logits;
  p.vocab = vocab;
  p.drafts = drafts;
  p.parents = parents;
  p.cu_rows = cu_rows;
  p.num_seqs = num_seqs;
  p.max_rows = max_rows;
  // As in vfy_accept: about two CTAs per SM over all rows, segments of at least 1024 entries.
  int parts = ceil_div(2LL * ctx->num_sms, max_rows);
  parts = clampi(parts, 1, ceil_div(vocab, 1024));
  int seg = ceil_div(vocab, parts);
  seg = (seg + 3) & ~3;
  p.parts = ceil_div(vocab, seg);
  p.seg = seg;
  p.accepted_len = accepted_len;
  p.path = path;
  p.bonus = bonus;
  p.committed = committed;
  p.keys = ctx->accept_keys;
  p.counters = ctx->tree_counters;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_accept_tree(p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

// Do buffers of `bytes` bytes from these addresses on lie apart? (The layers of a call move their rows at the same time.)
static bool apart(uintptr_t* at, int n, uint64_t bytes) {
  std::sort(at, at + n);
  for (int i = 1; i < n; ++i)
    if (at[i] - at[i - 1] < bytes) return false;
  return true;
}

// The arguments that both compactions share.
static void compact_params(const vfy_ctx* ctx, const int32_t* path, const int32_t* accepted_len,
                           const int32_t* cu_q, const int32_t* seq_len, int num_layers, int num_seqs,
                           vfy::CompactParams* p) {
  p->path = path;
  p->accepted = accepted_len;
  p->cu_q = cu_q;
  p->seq_len = seq_len;
  p->num_seqs = num_seqs;
  p->max_q = tree_capacity(ctx->cfg);
  p->token_cap = num_seqs * ctx->cfg.max_queries_per_seq;
  p->hkv = ctx->cfg.num_kv_heads;
  p->head_dim = ctx->cfg.head_dim;
  p->num_layers = num_layers;
  p->err = ctx->err;
}

vfy_status vfy_compact_full(vfy_ctx* ctx, const int32_t* path, const int32_t* accepted_len, const int32_t* cu_q,
                            const int32_t* seq_len, const int32_t* cu_chunks, const int32_t* slot_of_chunk,
                            int num_layers, uint16_t* const* host_k, uint16_t* const* host_v,
                            int64_t num_host_chunks, uint16_t* const* k_pool, uint16_t* const* v_pool,
                            int num_slots, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && path != nullptr && accepted_len != nullptr && cu_q != nullptr && seq_len != nullptr);
  VFY_REQUIRE(cu_chunks != nullptr && slot_of_chunk != nullptr);
  VFY_REQUIRE(host_k != nullptr && host_v != nullptr && k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(num_layers >= 1 && num_layers <= VFY_MAX_COMPACT_LAYERS);
  VFY_REQUIRE(num_host_chunks >= 1 && num_host_chunks <= INT_MAX && num_slots >= 1);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  uintptr_t pools[2 * VFY_MAX_COMPACT_LAYERS], stores[2 * VFY_MAX_COMPACT_LAYERS];
  for (int l = 0; l < num_layers; ++l) {
    VFY_REQUIRE(host_k[l] != nullptr && host_v[l] != nullptr && k_pool[l] != nullptr && v_pool[l] != nullptr);
    VFY_REQUIRE(aligned16(host_k[l]) && aligned16(host_v[l]) && aligned16(k_pool[l]) && aligned16(v_pool[l]));
    pools[2 * l] = reinterpret_cast<uintptr_t>(k_pool[l]);
    pools[2 * l + 1] = reinterpret_cast<uintptr_t>(v_pool[l]);
    stores[2 * l] = reinterpret_cast<uintptr_t>(host_k[l]);
    stores[2 * l + 1] = reinterpret_cast<uintptr_t>(host_v[l]);
  }
  const uint64_t chunk_bytes = 2ull * ctx->cfg.num_kv_heads * kChunk * ctx->cfg.head_dim;
  VFY_REQUIRE(apart(pools, 2 * num_layers, chunk_bytes * num_slots));
  VFY_REQUIRE(apart(stores, 2 * num_layers, chunk_bytes * static_cast<uint64_t>(num_host_chunks)));
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  vfy::CompactParams p = {};
  compact_params(ctx, path, accepted_len, cu_q, seq_len, num_layers, num_seqs, &p);
  p.cu_chunks = cu_chunks;
  p.slot_of_chunk = slot_of_chunk;
  p.num_host_chunks = num_host_chunks;
  p.num_slots = num_slots;
  for (int l = 0; l < num_layers; ++l) {
    void* store[2] = {host_k[l], host_v[l]};
    const vfy_status st = device_view(s, store, 2);
    if (st != VFY_OK) return st;
    p.store[l][0] = static_cast<uint16_t*>(store[0]);
    p.store[l][1] = static_cast<uint16_t*>(store[1]);
    p.dst[l][0] = k_pool[l];
    p.dst[l][1] = v_pool[l];
  }
  VFY_CUDA(vfy::launch_compact(false, p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_compact_swa(vfy_ctx* ctx, const int32_t* path, const int32_t* accepted_len, const int32_t* cu_q,
                           const int32_t* seq_len, const int32_t* ring_offset, int num_layers,
                           uint16_t* const* k_ring, uint16_t* const* v_ring, int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && path != nullptr && accepted_len != nullptr && cu_q != nullptr && seq_len != nullptr);
  VFY_REQUIRE(ring_offset != nullptr && k_ring != nullptr && v_ring != nullptr);
  VFY_REQUIRE(num_layers >= 1 && num_layers <= VFY_MAX_COMPACT_LAYERS);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  uintptr_t rings[2 * VFY_MAX_COMPACT_LAYERS];
  for (int l = 0; l < num_layers; ++l) {
    VFY_REQUIRE(k_ring[l] != nullptr && v_ring[l] != nullptr && aligned16(k_ring[l]) && aligned16(v_ring[l]));
    rings[2 * l] = reinterpret_cast<uintptr_t>(k_ring[l]);
    rings[2 * l + 1] = reinterpret_cast<uintptr_t>(v_ring[l]);
  }
  const uint64_t ring_bytes = 2ull * ctx->cfg.num_kv_heads * ctx->cfg.ring_len * ctx->cfg.head_dim;
  VFY_REQUIRE(apart(rings, 2 * num_layers, ring_bytes * num_seqs));
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::CompactParams p = {};
  compact_params(ctx, path, accepted_len, cu_q, seq_len, num_layers, num_seqs, &p);
  p.ring_off = ring_offset;
  p.ring_len = ctx->cfg.ring_len;
  for (int l = 0; l < num_layers; ++l) {
    p.dst[l][0] = k_ring[l];
    p.dst[l][1] = v_ring[l];
  }
  VFY_CUDA(vfy::launch_compact(true, p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

// ------------------------------ rotation and append ------------------------------------------
// Rows of `width` values, `stride` apart: 16-byte words of every row are aligned.
static bool row_stride_ok(int64_t stride, int64_t width) {
  return stride >= width && stride % 8 == 0 && stride <= (int64_t{1} << 32);
}
// Arguments that the three calls share (q and k may be absent in vfy_rope; the output rows of a call may be its input rows).
static bool rope_params(const vfy_ctx* ctx, const vfy_rotary* r, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                        int64_t k_stride, const int32_t* cu_q, const int32_t* seq_len, const int32_t* depth,
                        uint16_t* q_out, int num_seqs, vfy::RopeParams* p) {
  if (ctx == nullptr || r == nullptr || cu_q == nullptr || seq_len == nullptr) return false;
  if (num_seqs < 1 || num_seqs > ctx->cfg.max_seqs) return false;
  const vfy_config& c = ctx->cfg;
  if (r->rot_dim < 0 || r->rot_dim > c.head_dim || r->rot_dim % 8 != 0) return false;
  if ((r->rot_dim > 0) != (r->inv_freq != nullptr)) return false;
  if ((reinterpret_cast<uintptr_t>(r->inv_freq) & 3u) != 0) return false;
  if (r->interleaved != 0 && r->interleaved != 1) return false;
  if (!std::isfinite(r->attention_factor) || !(r->eps >= 0.f) || !std::isfinite(r->eps)) return false;
  if (!aligned16(r->q_norm) || !aligned16(r->k_norm)) return false;
  const int64_t q_width = static_cast<int64_t>(c.num_q_heads) * c.head_dim;
  if ((q != nullptr) != (q_out != nullptr)) return false;
  if (q != nullptr && (!aligned16(q) || !aligned16(q_out) || !row_stride_ok(q_stride, q_width))) return false;
  if (q != nullptr && q == q_out && q_stride != q_width) return false;
  if (k != nullptr && (!aligned16(k) || !row_stride_ok(k_stride, static_cast<int64_t>(c.num_kv_heads) * c.head_dim)))
    return false;
  *p = {};
  p->q = q;
  p->k = k;
  p->q_stride = q_stride;
  p->k_stride = k_stride;
  p->inv_freq = r->inv_freq;
  p->rot = r->rot_dim;
  p->interleaved = r->interleaved;
  p->factor = r->attention_factor == 0.f ? 1.f : r->attention_factor;
  p->q_norm = r->q_norm;
  p->k_norm = r->k_norm;
  p->eps = r->eps;
  p->cu_q = cu_q;
  p->seq_len = seq_len;
  p->depth = depth;
  p->num_seqs = num_seqs;
  p->max_q = c.max_queries_per_seq;
  p->token_cap = num_seqs * c.max_queries_per_seq;
  // One token a CTA while all of them run at once (eight CTAs per SM), else one a warp: 17 tokens 2.8 us against 4.5, 608 3.4
  // against 4.8, 1216 4.5 against 5.1; 2432 8.1 against 6.2.
  p->tokens_per_cta = p->token_cap <= 8 * ctx->num_sms ? 1 : vfy::rope_cta_tokens();
  p->hq = c.num_q_heads;
  p->hkv = c.num_kv_heads;
  p->head_dim = c.head_dim;
  p->q_out = q_out;
  p->err = ctx->err;
  return true;
}

vfy_status vfy_rope(vfy_ctx* ctx, const vfy_rotary* rotary, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                    int64_t k_stride, const int32_t* cu_q, const int32_t* seq_len, const int32_t* depth, uint16_t* q_out,
                    uint16_t* k_out, int num_seqs, vfy_stream_t stream) {
  vfy::RopeParams p;
  VFY_REQUIRE(rope_params(ctx, rotary, q, q_stride, k, k_stride, cu_q, seq_len, depth, q_out, num_seqs, &p));
  VFY_REQUIRE((k != nullptr) == (k_out != nullptr) && (q != nullptr || k != nullptr));
  VFY_REQUIRE(aligned16(k_out));
  VFY_REQUIRE(k == nullptr || k != k_out || k_stride == static_cast<int64_t>(p.hkv) * p.head_dim);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  p.k_dst = k_out;
  VFY_CUDA(vfy::launch_rope(p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_rope_append_full(vfy_ctx* ctx, const vfy_rotary* rotary, const uint16_t* q, int64_t q_stride,
                                const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                const int32_t* cu_q, const int32_t* seq_len, const int32_t* depth,
                                const int32_t* cu_chunks, const int32_t* slot_of_chunk, uint16_t* host_k,
                                uint16_t* host_v, int64_t num_host_chunks, uint16_t* k_pool, uint16_t* v_pool,
                                int num_slots, uint16_t* q_out, int num_seqs, vfy_stream_t stream) {
  vfy::RopeParams p;
  VFY_REQUIRE(rope_params(ctx, rotary, q, q_stride, k, k_stride, cu_q, seq_len, depth, q_out, num_seqs, &p));
  VFY_REQUIRE(k != nullptr && v != nullptr && cu_chunks != nullptr && slot_of_chunk != nullptr);
  VFY_REQUIRE(host_k != nullptr && host_v != nullptr && k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(aligned16(v) && aligned16(host_k) && aligned16(host_v) && aligned16(k_pool) && aligned16(v_pool));
  VFY_REQUIRE(row_stride_ok(v_stride, static_cast<int64_t>(p.hkv) * p.head_dim));
  VFY_REQUIRE(num_host_chunks >= 1 && num_host_chunks <= INT_MAX && num_slots >= 1);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* store[2] = {host_k, host_v};
  const vfy_status st = device_view(s, store, 2);
  if (st != VFY_OK) return st;
  p.v = v;
  p.v_stride = v_stride;
  p.cu_chunks = cu_chunks;
  p.slot_of_chunk = slot_of_chunk;
  p.host_k = static_cast<uint16_t*>(store[0]);
  p.host_v = static_cast<uint16_t*>(store[1]);
  p.num_host_chunks = num_host_chunks;
  p.num_slots = num_slots;
  p.k_dst = k_pool;
  p.v_dst = v_pool;
  VFY_CUDA(vfy::launch_rope(p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_rope_append_swa(vfy_ctx* ctx, const vfy_rotary* rotary, const uint16_t* q, int64_t q_stride,
                               const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                               const int32_t* cu_q, const int32_t* seq_len, const int32_t* depth,
                               const int32_t* ring_offset, uint16_t* k_ring, uint16_t* v_ring, uint16_t* q_out,
                               int num_seqs, vfy_stream_t stream) {
  vfy::RopeParams p;
  VFY_REQUIRE(rope_params(ctx, rotary, q, q_stride, k, k_stride, cu_q, seq_len, depth, q_out, num_seqs, &p));
  VFY_REQUIRE(k != nullptr && v != nullptr && ring_offset != nullptr && k_ring != nullptr && v_ring != nullptr);
  VFY_REQUIRE(aligned16(v) && aligned16(k_ring) && aligned16(v_ring));
  VFY_REQUIRE(row_stride_ok(v_stride, static_cast<int64_t>(p.hkv) * p.head_dim));
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  p.v = v;
  p.v_stride = v_stride;
  p.ring_off = ring_offset;
  p.ring_len = ctx->cfg.ring_len;
  p.k_dst = k_ring;
  p.v_dst = v_ring;
  VFY_CUDA(vfy::launch_rope(p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

// ------------------------------ 4-bit chunks -------------------------------------------------
static bool tensor_scale_ok(float g) { return g > 0.f && std::isfinite(g); }

vfy_status vfy_append_full_packed(vfy_ctx* ctx, const uint16_t* k_new, const uint16_t* v_new, const int32_t* cu_q,
                                  const int32_t* seq_len, const int32_t* cu_chunks, const int32_t* slot_of_chunk,
                                  uint8_t* host_k, uint8_t* host_v, int64_t num_host_chunks, uint8_t* k_pool,
                                  uint8_t* v_pool, int num_slots, float k_scale, float v_scale, int num_seqs,
                                  vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && k_new != nullptr && v_new != nullptr && cu_q != nullptr && seq_len != nullptr);
  VFY_REQUIRE(cu_chunks != nullptr && slot_of_chunk != nullptr && host_k != nullptr && host_v != nullptr);
  VFY_REQUIRE(k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(aligned16(k_new) && aligned16(v_new) && aligned16(host_k) && aligned16(host_v) && aligned16(k_pool) &&
              aligned16(v_pool));
  VFY_REQUIRE(num_host_chunks >= 1 && num_host_chunks <= INT_MAX && num_slots >= 1);
  VFY_REQUIRE(tensor_scale_ok(k_scale) && tensor_scale_ok(v_scale));
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* store[2] = {host_k, host_v};
  const vfy_status st = device_view(s, store, 2);
  if (st != VFY_OK) return st;
  vfy::PackedAppendParams p = {};
  p.k_new = k_new;
  p.v_new = v_new;
  p.cu_q = cu_q;
  p.seq_len = seq_len;
  p.num_seqs = num_seqs;
  p.max_q = ctx->cfg.max_queries_per_seq;
  p.token_cap = num_seqs * ctx->cfg.max_queries_per_seq;
  p.hkv = ctx->cfg.num_kv_heads;
  p.head_dim = ctx->cfg.head_dim;
  p.cu_chunks = cu_chunks;
  p.slot_of_chunk = slot_of_chunk;
  p.host_k = static_cast<uint8_t*>(store[0]);
  p.host_v = static_cast<uint8_t*>(store[1]);
  p.num_host_chunks = num_host_chunks;
  p.num_slots = num_slots;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.num_sms = ctx->num_sms;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  auto reciprocal = [](float g) { return g > 7.9e-31f && g < 1.2e30f ? 1.f / g : 0.f; };   // 2^-100 .. 2^100
  p.k_inv = reciprocal(k_scale);
  p.v_inv = reciprocal(v_scale);
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_append_packed(p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_page_in_packed(vfy_ctx* ctx, const uint8_t* host_k, const uint8_t* host_v, int64_t num_host_chunks,
                              uint8_t* k_pool, uint8_t* v_pool, int num_slots, const int32_t* pagein_list,
                              const int32_t* pagein_count, int num_seqs, int k, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && host_k != nullptr && host_v != nullptr && k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(pagein_list != nullptr && pagein_count != nullptr);
  VFY_REQUIRE(aligned16(host_k) && aligned16(host_v) && aligned16(k_pool) && aligned16(v_pool));
  VFY_REQUIRE(num_host_chunks >= 1 && num_host_chunks <= INT_MAX && num_slots >= 1);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs && k >= 1 && k <= vfy::kMaxSelectK);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* store[2] = {const_cast<uint8_t*>(host_k), const_cast<uint8_t*>(host_v)};
  const vfy_status st = device_view(s, store, 2);
  if (st != VFY_OK) return st;
  // The same copy as vfy_page_in, of chunks of another size (a multiple of 16 bytes too).
  vfy::PageInParams p;
  p.host_k = static_cast<const uint16_t*>(store[0]);
  p.host_v = static_cast<const uint16_t*>(store[1]);
  p.num_host_chunks = num_host_chunks;
  p.k_pool = reinterpret_cast<uint16_t*>(k_pool);
  p.v_pool = reinterpret_cast<uint16_t*>(v_pool);
  p.num_slots = num_slots;
  p.list = pagein_list;
  p.count = pagein_count;
  p.num_seqs = num_seqs;
  p.k = k;
  p.chunk_elems = static_cast<long long>(ctx->cfg.num_kv_heads) * VFY_PACKED_BYTES(ctx->cfg.head_dim) / 2;
  p.err = ctx->err;
  p.parts = ctx->pagein_ctas > 0 ? ctx->pagein_ctas : 2;
  VFY_CUDA(vfy::launch_page_in(p, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_unpack_chunks(vfy_ctx* ctx, const uint8_t* k_pool, const uint8_t* v_pool, int num_slots,
                             const int32_t* slots, int num_chunks, float k_scale, float v_scale, uint16_t* k_out,
                             uint16_t* v_out, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && k_pool != nullptr && v_pool != nullptr && num_slots >= 1 && num_chunks >= 0);
  VFY_REQUIRE(tensor_scale_ok(k_scale) && tensor_scale_ok(v_scale));
  if (num_chunks == 0) return VFY_OK;
  VFY_REQUIRE(slots != nullptr && k_out != nullptr && v_out != nullptr);
  VFY_REQUIRE(aligned16(k_pool) && aligned16(v_pool) && aligned16(k_out) && aligned16(v_out));
  VFY_REQUIRE(static_cast<long long>(num_chunks) * ctx->cfg.num_kv_heads <= INT_MAX);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::UnpackParams p;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.num_slots = num_slots;
  p.slots = slots;
  p.n = num_chunks;
  p.hkv = ctx->cfg.num_kv_heads;
  p.head_dim = ctx->cfg.head_dim;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_out = k_out;
  p.v_out = v_out;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_unpack(p, reinterpret_cast<cudaStream_t>(stream)));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_attend_full_packed(vfy_ctx* ctx, const uint16_t* q, const int32_t* cu_q, const uint8_t* k_pool,
                                  const uint8_t* v_pool, int num_slots, const int32_t* resident_ids,
                                  const int32_t* resident_slots, const int32_t* cu_resident, int max_resident_per_seq,
                                  const int32_t* seq_len, float k_scale, float v_scale, uint16_t* out, float* lse,
                                  int num_seqs, vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && q != nullptr && cu_q != nullptr && k_pool != nullptr && v_pool != nullptr);
  VFY_REQUIRE(resident_ids != nullptr && resident_slots != nullptr && cu_resident != nullptr);
  VFY_REQUIRE(seq_len != nullptr && out != nullptr);
  VFY_REQUIRE(aligned16(q) && aligned16(k_pool) && aligned16(v_pool) && aligned16(out));
  VFY_REQUIRE(lse == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(num_slots >= 1 && max_resident_per_seq >= 0);
  VFY_REQUIRE(tensor_scale_ok(k_scale) && tensor_scale_ok(v_scale));
  const vfy_config& c = ctx->cfg;
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  vfy::PackedAttnParams p;
  p.q = q;
  p.cu_q = cu_q;
  p.seq_len = seq_len;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.num_slots = num_slots;
  p.res_ids = resident_ids;
  p.res_slots = resident_slots;
  p.cu_res = cu_resident;
  p.hq = c.num_q_heads;
  p.hkv = c.num_kv_heads;
  p.group = p.hq / p.hkv;
  p.head_dim = c.head_dim;
  p.max_q = c.max_queries_per_seq;
  p.row_tiles = ctx->row_tiles;
  const int block_rows = c.max_queries_per_seq * p.group;
  const bool few = block_rows <= vfy::kPackedFewRows;
  // Row tiles of equal size (in whole groups of eight rows).
  p.n_tiles = ceil_div(block_rows, vfy::packed_tile_rows());
  p.tile_rows = (ceil_div(block_rows, p.n_tiles) + 7) & ~7;
  p.n_tiles = ceil_div(block_rows, p.tile_rows);
  VFY_REQUIRE(static_cast<long long>(num_seqs) * p.n_tiles <= 65535);
  int splits = ctx->full_splits;
  if (splits == 0) {
    const long long items = static_cast<long long>(p.hkv) * num_seqs * p.n_tiles;
    if (few) {
      // One CTA an SM (for a batch twice as many, which even out), each with five chunks: half a chunk for ten of its
      // sixteen warps (128 chunks: 8 splits 10.9 us, 24 8.3, 38 10.3).
      splits = static_cast<int>(ctx->num_sms * (num_seqs > 1 ? 2 : 1) / items);
      splits = clampi(splits, 1, std::max(1, ceil_div(max_resident_per_seq, 5)));
    } else {
      // One CTA an SM, for a batch twice as many, which even out sequences of different lengths (8 ragged ones: 9 splits
      // 67.5 us, 5 74, 12 73; 16: 4 splits 38.2, 5 43.6), and no fewer than three tiles each: what a CTA begins and ends with
      // is as long (64 tiles: 22 splits 13.4 us, 38 15.5).
      splits = static_cast<int>(ctx->num_sms * (num_seqs > 1 ? 2 : 1) / items);
      splits = clampi(splits, 1, std::max(1, ceil_div(max_resident_per_seq, 6)));
    }
  }
  p.num_splits = clampi(splits, 1, c.max_splits);
  p.token_cap = num_seqs * c.max_queries_per_seq;
  int scale_exp = 0, k_exp = 0;
  const float scale = std::frexp(ctx->scale, &scale_exp), k_part = std::frexp(k_scale, &k_exp);
  p.scale_log2 = scale * 1.4426950408889634f * k_part;
  p.scale_exp = scale_exp + k_exp;
  p.v_scale = v_scale;
  p.part_o = ctx->part_o;
  p.part_ml = ctx->part_ml;
  p.num_seqs = num_seqs;
  p.timeout_test_ns = ctx->timeout_test_ns;
  p.stable_metadata = ctx->stable_metadata;
  p.err = ctx->err;
  p.out = out;
  p.lse = lse;
  VFY_CUDA(few ? vfy::launch_attend_packed_few(p, num_seqs, s) : vfy::launch_attend_packed(p, num_seqs, s));
  ++ctx->launches;
  if (few && p.num_splits == 1) return VFY_OK;
  vfy::CombineParams cp;
  cp.cu_q = cu_q;
  cp.seq_len = seq_len;
  cp.num_seqs = num_seqs;
  cp.hq = p.hq;
  cp.hkv = p.hkv;
  cp.group = p.group;
  cp.num_splits = p.num_splits;
  cp.max_q = p.max_q;
  cp.row_tiles = p.row_tiles;
  cp.token_cap = p.token_cap;
  cp.by_seq = false;
  cp.stable_metadata = ctx->stable_metadata;
  cp.part_o = ctx->part_o;
  cp.part_ml = ctx->part_ml;
  cp.out = out;
  cp.lse = lse;
  cp.err = ctx->err;
  VFY_CUDA(vfy::launch_combine(c.head_dim, cp, s));
  ++ctx->launches;
  return VFY_OK;
}

vfy_status vfy_accept_sampled(vfy_ctx* ctx, const void* logits, int logits_type, int64_t row_stride, int vocab,
                              const float* temperature, const int32_t* drafts, const float* draft_probs,
                              const float* uniform, const float* noise, const int32_t* cu_rows, int max_rows,
                              int32_t* accepted_len, int32_t* bonus, int32_t* committed, int num_seqs,
                              vfy_stream_t stream) {
  VFY_REQUIRE(ctx != nullptr && logits != nullptr && temperature != nullptr && noise != nullptr && cu_rows != nullptr);
  VFY_REQUIRE(accepted_len != nullptr && bonus != nullptr && committed != nullptr);
  VFY_REQUIRE(logits_type == VFY_LOGITS_F32 || logits_type == VFY_LOGITS_BF16);
  const bool bf16 = logits_type == VFY_LOGITS_BF16;
  VFY_REQUIRE(vocab >= 1 && vocab <= kMaxVocab && row_stride >= vocab);
  VFY_REQUIRE((reinterpret_cast<uintptr_t>(logits) & (bf16 ? 1u : 3u)) == 0);
  VFY_REQUIRE(((reinterpret_cast<uintptr_t>(draft_probs) | reinterpret_cast<uintptr_t>(noise)) & 3u) == 0);
  VFY_REQUIRE(num_seqs >= 1 && num_seqs <= ctx->cfg.max_seqs);
  VFY_REQUIRE(max_rows >= 1 && max_rows <= ctx->accept_rows_cap && max_rows <= 65535);
  VFY_REQUIRE((drafts != nullptr && uniform != nullptr) || max_rows <= num_seqs);
  VFY_REQUIRE(row_stride <= (INT64_MAX / 8) / max_rows);
  DeviceGuard guard(ctx->device);
  if (!guard.ok) return VFY_ECUDA;
  vfy::SampleParams p;
  p.logits = logits;
  p.stride = row_stride;
  p.vocab = vocab;
  p.temperature = temperature;
  p.drafts = drafts;
  p.probs = draft_probs;
  p.uniform = uniform;
  p.noise = noise;
  p.cu_rows = cu_rows;
  p.num_seqs = num_seqs;
  p.max_rows = max_rows;
  // Segments of whole 16-byte words, at least 4096 entries (one round of loads of a CTA), at most 32 of a row (a warp merges
  // them), and no more than run at once, four CTAs per SM, over all rows.
  p.parts = clampi(static_cast<int>(kSampleCtas * ctx->num_sms / max_rows), 1, std::min(32, ceil_div(vocab, 4096)));
  p.seg = (ceil_div(vocab, p.parts) + 7) & ~7;
  p.parts = ceil_div(vocab, p.seg);
  // The draw: at least one round of loads of a CTA, and no more than run at once, two CTAs per SM over the sequences.
  p.draw_parts = clampi(static_cast<int>(2LL * ctx->num_sms / num_seqs), 1, ceil_div(vocab, 2048));
  p.draw_seg = ceil_div(vocab, p.draw_parts);
  p.draw_parts = ceil_div(vocab, p.draw_seg);
  p.accepted_len = accepted_len;
  p.bonus = bonus;
  p.committed = committed;
  p.stats = ctx->sample_stats;
  p.keys = ctx->sample_keys;
  p.counters = ctx->sample_counters;
  p.err = ctx->err;
  VFY_CUDA(vfy::launch_accept_sampled(p, bf16, reinterpret_cast<cudaStream_t>(stream)));
  ctx->launches += 2;
  return VFY_OK;
}

}  // extern "C"
