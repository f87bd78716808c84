// step_api.cu — the C ABI of the operators around the verify step: argument
// checks, launch shapes and launches.  The declarations, with the meaning of
// every argument, are in include/specdec_step.h.
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>
#include <string.h>

#include "specdec_step.h"

#include "attention_kernel.cuh"
#include "kv_kernels.cuh"
#include "logits_kernel.cuh"

namespace specdec {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

specdec_status_t launched() { return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA; }

bool block_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

// Whether p is memory that the CUDA runtime gave out (false without a device).
bool on_device(const void* p) {
  cudaPointerAttributes at;
  if (p == nullptr) return false;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

// The cache's shape: INVALID_ARG, UNSUPPORTED or OK.
specdec_status_t check_cache(int32_t num_blocks, int32_t block_size, int32_t H, int32_t D) {
  if (num_blocks <= 0 || block_size <= 0 || H <= 0 || D <= 0) return SPECDEC_ERR_INVALID_ARG;
  if (!block_size_ok(block_size) || (D != 64 && D != 128)) return SPECDEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX || H > 65535) return SPECDEC_ERR_UNSUPPORTED;
  return SPECDEC_OK;
}

// SMs of the current device, which is asked once.
cudaError_t device_sms(int* dev, int* sms) {
  static int known[64] = {0};
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= 64) return cudaErrorInvalidDevice;
  if (known[*dev] == 0) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev);
    if (e != cudaSuccess) return e;
    known[*dev] = n;
  }
  *sms = known[*dev];
  return cudaSuccess;
}

template <typename Elt>
cudaError_t launch_logits(LogitArgs a, cudaStream_t st) {
  using L = LogitLayout<Elt>;
  constexpr int kElt = sizeof(Elt);
  static bool ready[64] = {false};
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(process_logits_kernel<Elt>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(kLogitRowBytes / kElt));
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  // Few requests are cut finer, until every SM has two items.  (Eight would
  // double the history's reading: 64 requests take 50 us instead of 35.)
  a.share = kLogitRowBytes / kElt;
  while (a.share * kElt > kLogitLeastBytes && static_cast<int64_t>(a.B) * ((a.V + a.share - 1) / a.share) < 2 * sms) a.share /= 2;
  a.chunks = (a.V + a.share - 1) / a.share;
  const int items = a.B * a.chunks;
  process_logits_kernel<Elt><<<static_cast<unsigned>(items < sms ? items : sms), kLogitThreads, L::bytes(a.share), st>>>(a);
  return cudaGetLastError();
}

// Map of a cache [num_blocks, H, bs, D]: a box is one head of one block, its
// rows swizzled as the matrix descriptors read them.
cudaError_t cache_map(CUtensorMap* map, const void* cache, int D, int bs, int H, int num_blocks) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode encode = nullptr;
  if (encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    encode = reinterpret_cast<Encode>(fn);
  }
  const cuuint64_t row = static_cast<cuuint64_t>(D);
  const cuuint64_t dims[4] = {row, static_cast<cuuint64_t>(bs), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[3] = {row, row * bs, row * bs * H};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(bs), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr size_t kPartialAt = 64 * 1024;  // of the workspace; the counters are before it
constexpr int kAttnMaxCtas = 1000;        // two records each fit the workspace
static_assert(kPartialAt + static_cast<size_t>(kAttnMaxCtas) * 2 * kPartialFloats * 4 <= SPECDEC_ATTENTION_WORKSPACE_BYTES,
              "the workspace holds every CTA's records");
constexpr int kAttnSmem = 227 * 1024;     // one CTA an SM

template <int D>
cudaError_t launch_attention(AttnArgs a, const void* k_cache, const void* v_cache, cudaStream_t st) {
  CUtensorMap km, vm;
  cudaError_t e = cache_map(&km, k_cache, D, a.bs, a.H, a.num_blocks);
  if (e == cudaSuccess) e = cache_map(&vm, v_cache, D, a.bs, a.H, a.num_blocks);
  if (e != cudaSuccess) return e;
  static bool ready[64] = {false};
  int dev = 0, sms = 0;
  e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  using L = AttnLayout<D>;
  // As many tiles as there is room for: they are what is on its way from HBM.
  int tiles = (kAttnSmem - L::bytes(0, a.rows)) / L::kTileBytes;
  tiles = tiles < 2 * kMaxRing ? tiles : 2 * kMaxRing;
  a.v_ring = tiles / 2;
  a.k_ring = tiles - a.v_ring;
  const int grid = sms < kAttnMaxCtas ? sms : kAttnMaxCtas;
  attention_kernel<D><<<grid, kAttnThreads, L::bytes(tiles, a.rows), st>>>(a, km, vm);
  return cudaGetLastError();
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" specdec_status_t spec_process_logits(
    const void* logits, void* out, specdec_dtype_t dtype, int32_t B, int32_t n_max, int32_t V, const int32_t* history,
    int32_t history_stride, const int32_t* prompt_len, const int32_t* history_len, const int32_t* draft_tokens,
    const int32_t* draft_len, const float* repetition, const float* presence, const float* frequency,
    const int32_t* bias_offsets, const int32_t* bias_ids, const float* bias_values, int32_t num_bias,
    const uint32_t* mask, int32_t mask_count, const int32_t* mask_rows, uint32_t* error_word, void* stream) {
  if (dtype != SPECDEC_F32 && dtype != SPECDEC_BF16) return SPECDEC_ERR_INVALID_ARG;
  if (B < 0 || n_max < 0 || V <= 0 || history_stride < 0 || num_bias < 0 || mask_count < 0) return SPECDEC_ERR_INVALID_ARG;
  if (V > SPECDEC_MAX_VOCAB || n_max > SPECDEC_MAX_DRAFT || B > SPECDEC_MAX_BATCH ||
      history_stride > static_cast<int32_t>(kCountMask))
    return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (logits == nullptr || out == nullptr) return SPECDEC_ERR_INVALID_ARG;
  const uintptr_t elt = dtype == SPECDEC_F32 ? 4 : 2;
  if (!aligned(logits, elt) || !aligned(out, elt)) return SPECDEC_ERR_INVALID_ARG;
  if (history_stride > 0 && (history == nullptr || prompt_len == nullptr || history_len == nullptr))
    return SPECDEC_ERR_INVALID_ARG;
  if (n_max > 0 && draft_tokens == nullptr) return SPECDEC_ERR_INVALID_ARG;
  if (bias_offsets != nullptr && num_bias > 0 && (bias_ids == nullptr || bias_values == nullptr))
    return SPECDEC_ERR_INVALID_ARG;
  if ((mask == nullptr || mask_count == 0) != (mask_rows == nullptr)) return SPECDEC_ERR_INVALID_ARG;

  LogitArgs a;
  memset(&a, 0, sizeof a);
  a.logits = logits;
  a.out = out;
  a.B = B;
  a.n_max = n_max;
  a.V = V;
  a.history_stride = history_stride;
  a.history = history;
  a.prompt_len = prompt_len;
  a.history_len = history_len;
  a.draft_tokens = draft_tokens;
  a.draft_len = draft_len;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_offsets = num_bias > 0 ? bias_offsets : nullptr;
  a.bias_ids = bias_ids;
  a.bias_values = bias_values;
  a.num_bias = num_bias;
  a.mask = mask;
  a.mask_count = mask_count;
  a.mask_words = (V + 31) / 32;
  a.mask_rows = mask_rows;
  a.err = error_word;
  a.same_phase = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0 ? 1 : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SPECDEC_F32 ? launch_logits<float>(a, st) : launch_logits<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

extern "C" specdec_status_t kv_block_step(int32_t B, int32_t block_size, int32_t max_blocks, int32_t num_blocks,
                                          const int32_t* kv_len, const int32_t* accepted_len,
                                          const int32_t* new_tokens, const int32_t* held, int32_t* block_table,
                                          int32_t* free_ring, const int32_t* ring_state, int32_t* kv_len_out,
                                          int32_t* held_out, int32_t* ring_state_out, int32_t* cu_tokens,
                                          int32_t* cu_blocks, int32_t* slot_map, int32_t* positions,
                                          int32_t capacity, uint32_t* error_word, void* stream) {
  if (B < 0 || block_size <= 0 || max_blocks <= 0 || num_blocks <= 0 || capacity < 0) return SPECDEC_ERR_INVALID_ARG;
  if (!block_size_ok(block_size) || B > SPECDEC_MAX_BATCH) return SPECDEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX ||
      static_cast<int64_t>(max_blocks) * block_size > INT32_MAX)
    return SPECDEC_ERR_UNSUPPORTED;
  // A step without requests has no arrays of them, but leaves its other outputs
  // as any step does, unless there is no ring on a device.
  if (B == 0 && !on_device(ring_state)) return SPECDEC_OK;
  if (B > 0 && (kv_len == nullptr || new_tokens == nullptr || held == nullptr || block_table == nullptr ||
                kv_len_out == nullptr || held_out == nullptr))
    return SPECDEC_ERR_INVALID_ARG;
  if (free_ring == nullptr || ring_state == nullptr || ring_state_out == nullptr || cu_tokens == nullptr || cu_blocks == nullptr)
    return SPECDEC_ERR_INVALID_ARG;
  if (capacity > 0 && (slot_map == nullptr || positions == nullptr)) return SPECDEC_ERR_INVALID_ARG;
  BlockArgs a;
  memset(&a, 0, sizeof a);
  a.B = B;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.capacity = capacity;
  a.kv_len = kv_len;
  a.accepted_len = accepted_len;
  a.new_tokens = new_tokens;
  a.held = held;
  a.table = block_table;
  a.ring = free_ring;
  a.ring_state = ring_state;
  a.kv_len_out = kv_len_out;
  a.held_out = held_out;
  a.ring_state_out = ring_state_out;
  a.cu_tokens = cu_tokens;
  a.cu_blocks = cu_blocks;
  a.slot_map = slot_map;
  a.positions = positions;
  a.err = error_word;
  a.slots_vec = aligned(slot_map, 16) ? 1 : 0;
  a.positions_vec = aligned(positions, 16) ? 1 : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One launch spares the host the second; on the device both forms take as long
  // (12.3 and 9.1 us for 1024 requests and 512 prompts in one, 11.1 and 9.5 in two).
  const bool apart = kv_len_out != kv_len && held_out != held && ring_state_out != ring_state;
  if (apart && B <= kBlockShared) {
    const int bytes = 4 * (B + 1) * static_cast<int>(sizeof(int32_t));
    if (bytes > 40 * 1024 && cudaFuncSetAttribute(block_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  4 * (kBlockShared + 1) * static_cast<int>(sizeof(int32_t))) != cudaSuccess)
      return SPECDEC_ERR_CUDA;
    const int64_t ctas = (static_cast<int64_t>(capacity) + 4 * kBlockThreads - 1) / (4 * kBlockThreads);
    block_step_kernel<<<static_cast<unsigned>(ctas < 1 ? 1 : (ctas > 128 ? 128 : ctas)), kBlockThreads, bytes, st>>>(a);
  } else {
    block_plan_kernel<<<1, kBlockThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SPECDEC_ERR_CUDA;
    const int64_t threads = (static_cast<int64_t>(capacity) + 3) / 4;
    block_fill_kernel<<<static_cast<unsigned>(threads < 256 ? 1 : (threads + 255) / 256), 256, 0, st>>>(a);
  }
  return launched();
}

extern "C" specdec_status_t kv_append(const void* k, const void* v, specdec_dtype_t dtype, int32_t T, int32_t H,
                                      int32_t D, int64_t k_token_stride, int64_t k_head_stride,
                                      int64_t v_token_stride, int64_t v_head_stride, const int32_t* slot_map,
                                      int32_t num_blocks, int32_t block_size, void* k_cache, void* v_cache,
                                      float* k_scale, float* v_scale, void* stream) {
  if (dtype != SPECDEC_F32 && dtype != SPECDEC_BF16) return SPECDEC_ERR_INVALID_ARG;
  if (T < 0) return SPECDEC_ERR_INVALID_ARG;
  const specdec_status_t chk = check_cache(num_blocks, block_size, H, D);
  if (chk != SPECDEC_OK) return chk;
  if (T == 0) return SPECDEC_OK;
  if (k == nullptr || v == nullptr || slot_map == nullptr || k_cache == nullptr || v_cache == nullptr ||
      k_scale == nullptr || v_scale == nullptr)
    return SPECDEC_ERR_INVALID_ARG;
  const int64_t elt = dtype == SPECDEC_F32 ? 4 : 2;
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  for (int64_t s : strides)
    if (s < 0 || s > (INT64_MAX >> 4) || s * elt % 16 != 0) return SPECDEC_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return SPECDEC_ERR_INVALID_ARG;
  AppendArgs a;
  memset(&a, 0, sizeof a);
  a.x[0] = k;
  a.x[1] = v;
  for (int i = 0; i < 2; ++i) {
    a.token_stride[i] = strides[2 * i] * elt;
    a.head_stride[i] = strides[2 * i + 1] * elt;
  }
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.slot_map = slot_map;
  a.T = T;
  a.H = H;
  a.bs = block_size;
  a.num_blocks = num_blocks;
  // A team holds a block's rows: 8 loads of 16 bytes a thread, or 16.
  const int64_t loads = static_cast<int64_t>(block_size) * D * elt / 16;
  const int vecs = loads <= 8 * kAppendThreads ? 8 : 16;
  a.team = 32;
  while (a.team * vecs < loads) a.team *= 2;
  a.pairs = 2 * H < 4 ? 2 * H : 4;  // (8 take 57 us where 4 take 54, 16 more)
  const unsigned splits = static_cast<unsigned>((2 * H + a.pairs - 1) / a.pairs);
  // Windows of a block's tokens, or fewer while that leaves SMs without work.
  int dev = 0, sms = 0;
  if (device_sms(&dev, &sms) != cudaSuccess) return SPECDEC_ERR_CUDA;
  a.window = block_size;
  while (a.window > 1 && static_cast<int64_t>(T) * splits < static_cast<int64_t>(a.window) * 2 * sms) a.window /= 2;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + a.window - 1) / a.window), splits);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPECDEC_F32) {
    if (D == 64)
      append_kernel<float, 64, 8><<<grid, kAppendThreads, 0, st>>>(a);
    else if (vecs == 8)
      append_kernel<float, 128, 8><<<grid, kAppendThreads, 0, st>>>(a);
    else
      append_kernel<float, 128, 16><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    if (D == 64)
      append_kernel<__nv_bfloat16, 64, 8><<<grid, kAppendThreads, 0, st>>>(a);
    else
      append_kernel<__nv_bfloat16, 128, 8><<<grid, kAppendThreads, 0, st>>>(a);
  }
  return launched();
}

extern "C" specdec_status_t spec_attention(const void* q, int64_t q_token_stride, int32_t T, int32_t Hq, int32_t H,
                                           int32_t D, int32_t B, const int32_t* cu_tokens, const int32_t* kv_len,
                                           const int32_t* block_table, int32_t max_blocks, int32_t num_blocks,
                                           int32_t block_size, const void* k_cache, const void* v_cache,
                                           const float* k_scale, const float* v_scale, float scale, void* out,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || B < 0 || Hq <= 0 || max_blocks <= 0) return SPECDEC_ERR_INVALID_ARG;
  const specdec_status_t chk = check_cache(num_blocks, block_size, H, D);
  if (chk != SPECDEC_OK) return chk;
  constexpr float kLog2e = 1.4426950408889634f;
  if (Hq % H != 0 || !(scale >= 0.f) || !(scale * kLog2e <= FLT_MAX)) return SPECDEC_ERR_INVALID_ARG;
  if (B > SPECDEC_MAX_BATCH || static_cast<int64_t>(max_blocks) * block_size + T > INT32_MAX) return SPECDEC_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return SPECDEC_OK;
  if (q == nullptr || cu_tokens == nullptr || kv_len == nullptr || block_table == nullptr || k_cache == nullptr ||
      v_cache == nullptr || k_scale == nullptr || v_scale == nullptr || out == nullptr)
    return SPECDEC_ERR_INVALID_ARG;
  if (q_token_stride < static_cast<int64_t>(Hq) * D || q_token_stride % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return SPECDEC_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < SPECDEC_ATTENTION_WORKSPACE_BYTES)
    return SPECDEC_ERR_WORKSPACE;
  AttnArgs a;
  memset(&a, 0, sizeof a);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_token_stride;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.T = T;
  a.Hq = Hq;
  a.H = H;
  a.B = B;
  a.cu_tokens = cu_tokens;
  a.kv_len = kv_len;
  a.table = block_table;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.bs = block_size;
  a.bs_log2 = block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : 7;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.scale_log2e = (scale > 0.f ? scale : (D == 64 ? 0.125f : 0.08838834764831845f)) * kLog2e;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + 256);
  a.partial = reinterpret_cast<float*>(ws + kPartialAt);
  // Rows of a group.  Few leave shared memory to the tiles on their way (8
  // tiles of K and V of D = 128 with 16 rows, 7 with 32, 6 with 64); a request
  // of more rows is read once for each of its groups.  How the tokens lie is
  // known on the device only, and this guess is about speed alone: as many for
  // each request where that is possible (which may still not be so), else evenly
  // spread, with the longest near twice the mean.  (128 requests of
  // one token over 4500: 141 us with 16 rows, 147 with 64; 256 of up to 32 rows:
  // 285 with 32, 287 with 64.)
  const int64_t rows = static_cast<int64_t>(T) * (Hq / H), likely = T % B == 0 ? rows / B : 7 * rows / (4 * B);
  a.rows = likely <= 16 ? 16 : likely <= 32 ? 32 : kAttnRows;
  // The kernel counts the cost of tiles of positions, over row groups and
  // heads, in 31 bits.
  const int64_t groups = rows / a.rows + (T < B ? T : B) + 1;
  const int64_t most_cost = (static_cast<int64_t>(max_blocks) * block_size + kTile - 1) / kTile * tile_cost(a.rows) + kItemCost;
  if (groups > INT32_MAX / H || groups * H > INT32_MAX / most_cost) return SPECDEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64 ? launch_attention<64>(a, k_cache, v_cache, st) : launch_attention<128>(a, k_cache, v_cache, st);
  return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}
