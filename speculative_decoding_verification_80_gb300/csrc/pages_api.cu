// pages_api.cu — the C ABI of the paged cache's forks, moves and copies: argument
// checks, launch shapes and launches.  The declarations, with the meaning of every
// argument, are in include/specdec_step.h.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "specdec_step.h"

#include "host_checks.cuh"
#include "page_kernels.cuh"

namespace specdec {
namespace {

specdec_status_t check_workspace(const void* workspace, size_t bytes, int64_t N) {
  return workspace == nullptr || !aligned(workspace, 16) || bytes < page_words(N) * 4 ? SPECDEC_ERR_WORKSPACE : SPECDEC_OK;
}

// CTAs' work that a cluster of 8 does, whose barriers are shorter than a grid's.  (Forks
// of 4, 7 and 9 CTAs' work take 10.4, 12.4 and 12.6 us in a cluster and 12.6, 15.2 and
// 16.4 in a grid; a compaction of 22 takes 14.4 and 12.4, a fork of 40 18.5 and 14.4.)
constexpr int kPageClusterWork = 16;

// As many CTAs as `items` threads' work needs: one cluster of up to 8, or a
// cooperative launch of at most one an SM.
template <typename Args>
specdec_status_t launch_page(void (*in_cluster)(Args), void (*in_grid)(Args), Args& a, int64_t items, cudaStream_t st) {
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPECDEC_ERR_CUDA;
  const int64_t wanted = (items + kPageThreads - 1) / kPageThreads;
  const bool cluster = wanted <= kPageClusterWork;
  unsigned ctas = 1;
  if (cluster)
    while (ctas < kPageCluster && ctas < wanted) ctas *= 2;
  else
    ctas = static_cast<unsigned>(wanted > sms ? sms : wanted);
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(ctas);
  config.blockDim = dim3(kPageThreads);
  config.stream = st;
  cudaLaunchAttribute attr;
  if (cluster) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  } else {
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
  }
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, cluster ? in_cluster : in_grid, a) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" size_t specdec_page_workspace_bytes(int32_t num_blocks) { return num_blocks > 0 ? page_words(num_blocks) * 4 : 0; }

extern "C" specdec_status_t kv_fork(int32_t P, int32_t B, int32_t block_size, int32_t max_blocks, int32_t num_blocks,
                                    const int32_t* block_table, const int32_t* kv_len, const int32_t* accepted_len,
                                    const int32_t* held, const int32_t* parent, const int32_t* keep,
                                    const int32_t* shares, int32_t* free_ring, const int32_t* ring_state,
                                    int32_t* table_out, int32_t* kv_len_out, int32_t* held_out, int32_t* shares_out,
                                    int32_t* ring_state_out, int32_t* copies, int32_t* count, void* workspace,
                                    size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (P < 0 || B < 0 || block_size <= 0 || max_blocks <= 0 || num_blocks <= 0) return SPECDEC_ERR_INVALID_ARG;
  if (!block_size_ok(block_size) || P > SPECDEC_MAX_BATCH || B > SPECDEC_MAX_BATCH) return SPECDEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX || static_cast<int64_t>(max_blocks) * block_size > INT32_MAX)
    return SPECDEC_ERR_UNSUPPORTED;
  if (shares == nullptr || free_ring == nullptr || ring_state == nullptr || shares_out == nullptr || ring_state_out == nullptr ||
      count == nullptr)
    return SPECDEC_ERR_INVALID_ARG;
  if (P > 0 && (block_table == nullptr || kv_len == nullptr || held == nullptr)) return SPECDEC_ERR_INVALID_ARG;
  if (B > 0 && (parent == nullptr || table_out == nullptr || kv_len_out == nullptr || held_out == nullptr || copies == nullptr))
    return SPECDEC_ERR_INVALID_ARG;
  // a request reads its parent's numbers, which another may replace
  if ((P > 0 && B > 0 && (table_out == block_table || kv_len_out == kv_len || held_out == held)) || (B > 0 && kv_len_out == accepted_len))
    return SPECDEC_ERR_INVALID_ARG;
  const specdec_status_t ws = check_workspace(workspace, workspace_bytes, num_blocks);
  if (ws != SPECDEC_OK) return ws;
  const size_t p4 = 4 * static_cast<size_t>(P), b4 = 4 * static_cast<size_t>(B), n4 = 4 * static_cast<size_t>(num_blocks);
  const Span in[] = {{block_table, p4 * max_blocks}, {kv_len, p4}, {accepted_len, p4}, {held, p4}, {parent, b4}, {keep, b4}, {shares, n4}, {ring_state, 8}};
  const Span out[] = {{table_out, b4 * max_blocks}, {kv_len_out, b4}, {held_out, b4}, {shares_out, n4, shares}, {ring_state_out, 8, ring_state},
                      {free_ring, n4}, {copies, 2 * b4}, {count, 4}, {workspace, workspace_bytes}, {error_word, 4}};
  if (outputs_collide(in, out)) return SPECDEC_ERR_INVALID_ARG;
  ForkArgs a;
  memset(&a, 0, sizeof a);
  a.P = P;
  a.B = B;
  a.bs_log2 = block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.table = block_table;
  a.kv_len = kv_len;
  a.accepted_len = accepted_len;
  a.held = held;
  a.parent = parent;
  a.keep = keep;
  a.shares = shares;
  a.ring = free_ring;
  a.ring_state = ring_state;
  a.table_out = table_out;
  a.kv_len_out = kv_len_out;
  a.held_out = held_out;
  a.shares_out = shares_out;
  a.ring_state_out = ring_state_out;
  a.copies = copies;
  a.count = count;
  a.err = error_word;
  a.work = page_work(workspace, workspace_bytes, num_blocks);
  // a thread for each entry of the tables or block
  const int64_t entries = (static_cast<int64_t>(P) + B) * max_blocks;
  return launch_page(fork_kernel<true>, fork_kernel<false>, a, entries > num_blocks ? entries : num_blocks, static_cast<cudaStream_t>(stream));
}

extern "C" specdec_status_t kv_compact(int32_t B, int32_t max_blocks, int32_t num_blocks, const int32_t* block_table,
                                       const int32_t* held, const int32_t* shares, const int32_t* free_ring,
                                       const int32_t* ring_state, int32_t* table_out, int32_t* shares_out,
                                       int32_t* ring_out, int32_t* ring_state_out, int32_t* renamed, int32_t* copies,
                                       int32_t* count, void* workspace, size_t workspace_bytes, uint32_t* error_word,
                                       void* stream) {
  if (B < 0 || max_blocks <= 0 || num_blocks <= 0) return SPECDEC_ERR_INVALID_ARG;
  if (B > SPECDEC_MAX_BATCH || num_blocks > (1 << 27)) return SPECDEC_ERR_UNSUPPORTED;
  if (shares == nullptr || free_ring == nullptr || ring_state == nullptr || shares_out == nullptr || ring_out == nullptr ||
      ring_state_out == nullptr || renamed == nullptr || (copies == nullptr && num_blocks > 1) || count == nullptr)
    return SPECDEC_ERR_INVALID_ARG;
  if (B > 0 && (block_table == nullptr || held == nullptr || table_out == nullptr)) return SPECDEC_ERR_INVALID_ARG;
  const specdec_status_t ws = check_workspace(workspace, workspace_bytes, num_blocks);
  if (ws != SPECDEC_OK) return ws;
  const size_t b4 = 4 * static_cast<size_t>(B), n4 = 4 * static_cast<size_t>(num_blocks);
  const Span in[] = {{block_table, b4 * max_blocks}, {held, b4}, {shares, n4}, {free_ring, n4}, {ring_state, 8}};
  const Span out[] = {{table_out, b4 * max_blocks, block_table}, {shares_out, n4, shares}, {ring_out, n4, free_ring}, {ring_state_out, 8, ring_state},
                      {renamed, n4}, {copies, 8 * static_cast<size_t>(num_blocks / 2)}, {count, 4}, {workspace, workspace_bytes}, {error_word, 4}};
  if (outputs_collide(in, out)) return SPECDEC_ERR_INVALID_ARG;
  CompactArgs a;
  memset(&a, 0, sizeof a);
  a.B = B;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.table = block_table;
  a.held = held;
  a.shares = shares;
  a.ring = free_ring;
  a.ring_state = ring_state;
  a.table_out = table_out;
  a.shares_out = shares_out;
  a.ring_out = ring_out;
  a.ring_state_out = ring_state_out;
  a.renamed = renamed;
  a.copies = copies;
  a.count = count;
  a.err = error_word;
  a.work = page_work(workspace, workspace_bytes, num_blocks);
  const int64_t entries = static_cast<int64_t>(B) * max_blocks;
  return launch_page(compact_kernel<true>, compact_kernel<false>, a, entries > num_blocks ? entries : num_blocks, static_cast<cudaStream_t>(stream));
}

extern "C" specdec_status_t kv_copy(const int32_t* copies, const int32_t* count, int32_t capacity, int32_t layers,
                                    void* const* caches, int32_t num_blocks, int32_t block_size, int32_t H, int32_t D,
                                    void* stream) {
  if (capacity < 0 || layers < 0 || num_blocks <= 0 || block_size <= 0 || H <= 0 || D <= 0) return SPECDEC_ERR_INVALID_ARG;
  if (!block_size_ok(block_size) || (D != 64 && D != 128) || H > 65535 || static_cast<int64_t>(num_blocks) * block_size > INT32_MAX)
    return SPECDEC_ERR_UNSUPPORTED;
  if (capacity == 0 || layers == 0) return SPECDEC_OK;
  if (copies == nullptr || count == nullptr || caches == nullptr) return SPECDEC_ERR_INVALID_ARG;
  for (int64_t i = 0; i < 4LL * layers; ++i)
    if (caches[i] == nullptr || !aligned(caches[i], i % 4 < 2 ? 16 : 4)) return SPECDEC_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPECDEC_ERR_CUDA;
  CopyArgs a;
  a.capacity = capacity;
  a.num_blocks = num_blocks;
  a.H = H;
  a.bytes = static_cast<int64_t>(H) * block_size * D;
  a.chunk = static_cast<int32_t>(a.bytes < 8192 ? a.bytes : 8192);
  a.chunks = static_cast<int32_t>((a.bytes + a.chunk - 1) / a.chunk);
  a.pairs = copies;
  a.count = count;
  for (int32_t l0 = 0; l0 < layers; l0 += kCopyLayers) {
    a.layers = layers - l0 < kCopyLayers ? layers - l0 : kCopyLayers;
    for (int l = 0; l < a.layers; ++l) {
      void* const* c = caches + 4LL * (l0 + l);
      a.layer[l] = {c[0], c[1], static_cast<float*>(c[2]), static_cast<float*>(c[3])};
    }
    // as many warps as there can be parts, at most 32 CTAs an SM: four are there at a
    // time, and the others level what they take (616 MB of blocks in 4, 8, 16 and 32
    // CTAs an SM: 105, 98, 96 and 95 us; in parts of 4 KB, which have more to look
    // up, 107, 100 and, with 32, 95)
    const int64_t parts = static_cast<int64_t>(capacity) * a.layers * 2 * a.chunks;
    const int64_t ctas = (parts + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    copy_kernel<<<static_cast<unsigned>(ctas < 32 * sms ? ctas : 32 * sms), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SPECDEC_ERR_CUDA;
  }
  return SPECDEC_OK;
}
