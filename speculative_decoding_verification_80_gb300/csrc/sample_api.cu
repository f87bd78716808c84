// sample_api.cu — the C ABI of sampling and rotary positions: argument checks,
// launch shapes and launches.  The declarations, with the meaning of every
// argument, are in include/specdec_step.h.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "specdec_step.h"

#include "host_checks.cuh"
#include "rotary_kernel.cuh"
#include "sample_kernel.cuh"

namespace specdec {
namespace {

template <typename Elt>
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  static bool ready[64] = {false};
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  // (bf16: a byte for each vector of a CTA's part behind the rest)
  constexpr size_t kFixed = sizeof(SampleSmem<Elt>);
  auto bytes = [](int32_t V, int ctas) { return kFixed + (sizeof(Elt) == 2 ? static_cast<size_t>((V / 8 + 2 + ctas - 1) / ctas + 1) : 0); };
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(sample_kernel<Elt>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes(SPECDEC_MAX_VOCAB, 1)));
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int64_t rows = static_cast<int64_t>(a.B) * (a.n_max + 1);
  // A row's parts: as many as half of the SMs have room for, or two on all of them.
  // (One row of 128256 bf16 logits in 1, 2, 4 and 8 parts: 26.8, 24.7, 20.6 and 18.5
  // us; 19 rows 28.7, 24.7, 20.6, 21.7; 38 rows 28.7, 24.7, 25.4, 37.0; 76 rows 28.8,
  // 26.0, 41, 58; 152 rows 28.8, 32.9.  Of 32003 all take 18.5.)
  int ctas = 1;
  if (static_cast<int64_t>(a.V) * sizeof(Elt) >= 65536)
    while (ctas < kSampleClusterMax && (4 * ctas * rows <= sms || (ctas == 1 && 2 * rows <= sms))) ctas *= 2;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(static_cast<unsigned>(rows * ctas));
  config.blockDim = dim3(kSampleThreads);
  config.dynamicSmemBytes = bytes(a.V, ctas);
  config.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, sample_kernel<Elt>, a, ctas);
}

// The widest load that a call's addresses, strides and parts allow, in values.
template <typename Elt>
cudaError_t launch_rotary(RotaryArgs a, int D, bool half, cudaStream_t st) {
  uintptr_t low = 0;
  bool apart = false;
  for (int w = 0; w < 2; ++w) {
    if (a.heads[w] == 0) continue;
    low |= reinterpret_cast<uintptr_t>(a.x[w]) | reinterpret_cast<uintptr_t>(a.y[w]) | static_cast<uintptr_t>(a.x_token[w]) |
           static_cast<uintptr_t>(a.x_head[w]) | static_cast<uintptr_t>(a.y_token[w]) | static_cast<uintptr_t>(a.y_head[w]);
    apart |= a.x[w] != a.y[w];
  }
  low |= static_cast<uintptr_t>(half ? a.pairs : 2 * a.pairs) * sizeof(Elt);
  if (apart) low |= static_cast<uintptr_t>(D - 2 * a.pairs) * sizeof(Elt);
  const int bytes = (low & 15) == 0 ? 16 : ((low & 7) == 0 ? 8 : static_cast<int>(sizeof(Elt)));
  int N = bytes / static_cast<int>(sizeof(Elt));
  if (!half && N > 1 && a.pairs % N != 0) N = a.pairs % (8 / static_cast<int>(sizeof(Elt))) == 0 ? 8 / static_cast<int>(sizeof(Elt)) : 1;
  a.turned = a.pairs / N;
  a.units = a.turned + (apart ? (D - 2 * a.pairs) / N : 0);
  a.group = 1;
  int dev = 0, sms = 0;
  const cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  while (2 * a.group * a.pairs <= kRotaryPairs && 2 * a.group <= kRotaryTokens && a.T > 8 * sms * a.group) a.group *= 2;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.T) + a.group - 1) / a.group);
  constexpr int kWide = 16 / static_cast<int>(sizeof(Elt));
  if (half) {
    if (N == kWide)
      rotary_kernel<Elt, kWide, true><<<grid, kRotaryThreads, 0, st>>>(a);
    else if (N == kWide / 2)
      rotary_kernel<Elt, kWide / 2, true><<<grid, kRotaryThreads, 0, st>>>(a);
    else
      rotary_kernel<Elt, 1, true><<<grid, kRotaryThreads, 0, st>>>(a);
  } else {
    if (N == kWide)
      rotary_kernel<Elt, kWide, false><<<grid, kRotaryThreads, 0, st>>>(a);
    else if (N == kWide / 2)
      rotary_kernel<Elt, kWide / 2, false><<<grid, kRotaryThreads, 0, st>>>(a);
    else
      rotary_kernel<Elt, 1, false><<<grid, kRotaryThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" specdec_status_t spec_sample(const void* logits, void* out, specdec_dtype_t dtype, int32_t B, int32_t n_max,
                                        int32_t V, const int32_t* draft_len, const float* temperature,
                                        const int32_t* top_k, const float* top_p, const float* min_p,
                                        const float* uniform, int32_t* tokens, uint32_t* error_word, void* stream) {
  if (dtype != SPECDEC_F32 && dtype != SPECDEC_BF16) return SPECDEC_ERR_INVALID_ARG;
  if (B < 0 || n_max < 0 || V <= 0) return SPECDEC_ERR_INVALID_ARG;
  if (V > SPECDEC_MAX_VOCAB || n_max > SPECDEC_MAX_DRAFT || B > SPECDEC_MAX_BATCH) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (logits == nullptr || (out == nullptr && tokens == nullptr) || (tokens == nullptr) != (uniform == nullptr))
    return SPECDEC_ERR_INVALID_ARG;
  const uintptr_t elt = dtype == SPECDEC_F32 ? 4 : 2;
  if (!aligned(logits, elt) || !aligned(out, elt)) return SPECDEC_ERR_INVALID_ARG;
  const size_t b4 = 4 * static_cast<size_t>(B), r4 = b4 * (static_cast<size_t>(n_max) + 1), bytes = r4 / 4 * V * elt;
  const Span in[] = {{logits, bytes}, {draft_len, b4}, {temperature, b4}, {top_k, b4}, {top_p, b4}, {min_p, b4}, {uniform, r4}};
  const Span outs[] = {{out, bytes, logits}, {tokens, r4}, {error_word, 4}};
  if (outputs_collide(in, outs)) return SPECDEC_ERR_INVALID_ARG;
  SampleArgs a;
  memset(&a, 0, sizeof a);
  a.logits = logits;
  a.out = out;
  a.B = B;
  a.n_max = n_max;
  a.V = V;
  a.draft_len = draft_len;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniform = uniform;
  a.tokens = tokens;
  a.err = error_word;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SPECDEC_F32 ? launch_sample<float>(a, st) : launch_sample<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

extern "C" specdec_status_t spec_rotary(const void* q, const void* k, specdec_dtype_t dtype, int32_t T, int32_t Hq,
                                        int32_t H, int32_t D, int64_t q_token_stride, int64_t q_head_stride,
                                        int64_t k_token_stride, int64_t k_head_stride, const int32_t* positions,
                                        const uint64_t* turns, int32_t rotary_dim, int32_t interleaved, float factor,
                                        void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                                        int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream) {
  if (dtype != SPECDEC_F32 && dtype != SPECDEC_BF16) return SPECDEC_ERR_INVALID_ARG;
  if (T < 0 || Hq < 0 || H < 0 || Hq + static_cast<int64_t>(H) <= 0 || D <= 0 || rotary_dim <= 0 || rotary_dim % 2 != 0 ||
      rotary_dim > D || (interleaved != 0 && interleaved != 1) || !(factor > 0.f) || !(factor <= 3e38f))
    return SPECDEC_ERR_INVALID_ARG;
  if (Hq > 65535 || H > 65535 || D > 1024) return SPECDEC_ERR_UNSUPPORTED;
  if (T == 0) return SPECDEC_OK;
  if ((Hq > 0 && (q == nullptr || q_out == nullptr)) || (H > 0 && (k == nullptr || k_out == nullptr)) || positions == nullptr ||
      turns == nullptr || !aligned(turns, 8))
    return SPECDEC_ERR_INVALID_ARG;
  const int64_t elt = dtype == SPECDEC_F32 ? 4 : 2;
  const int64_t strides[8] = {q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride,
                              k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride};
  RotaryArgs a;
  memset(&a, 0, sizeof a);
  const void* x[2] = {q, k};
  void* y[2] = {q_out, k_out};
  a.heads[0] = Hq;
  a.heads[1] = H;
  for (int w = 0; w < 2; ++w) {
    if (a.heads[w] == 0) continue;
    // (of one token, or one head, there is no next)
    const int64_t s[4] = {T > 1 ? strides[4 * w] : 0, a.heads[w] > 1 ? strides[4 * w + 1] : 0, T > 1 ? strides[4 * w + 2] : 0,
                          a.heads[w] > 1 ? strides[4 * w + 3] : 0};
    // (the last row's start stays within 64 bits)
    const int64_t most[2] = {(INT64_MAX >> 4) / (T > 1 ? T - 1 : 1), (INT64_MAX >> 4) / (a.heads[w] > 1 ? a.heads[w] - 1 : 1)};
    for (int i = 0; i < 4; ++i)
      if (s[i] < 0 || s[i] > most[i % 2]) return SPECDEC_ERR_INVALID_ARG;
    if (!aligned(x[w], elt) || !aligned(y[w], elt)) return SPECDEC_ERR_INVALID_ARG;
    // in place means in every place
    if (x[w] == y[w] && (s[0] != s[2] || s[1] != s[3])) return SPECDEC_ERR_INVALID_ARG;
    // rows of an output lie apart
    if ((T > 1 && s[2] < D) || (a.heads[w] > 1 && s[3] < D)) return SPECDEC_ERR_INVALID_ARG;
    if (T > 1 && a.heads[w] > 1 && s[2] < (a.heads[w] - 1) * s[3] + D && (s[3] - D) / (T - 1) < s[2]) return SPECDEC_ERR_INVALID_ARG;
    a.x[w] = static_cast<const char*>(x[w]);
    a.y[w] = static_cast<char*>(y[w]);
    a.x_token[w] = s[0] * elt;
    a.x_head[w] = s[1] * elt;
    a.y_token[w] = s[2] * elt;
    a.y_head[w] = s[3] * elt;
  }
  a.T = T;
  a.positions = positions;
  a.turns = reinterpret_cast<const unsigned long long*>(turns);
  a.factor = factor;
  a.pairs = rotary_dim / 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SPECDEC_F32 ? launch_rotary<float>(a, D, interleaved == 0, st)
                                             : launch_rotary<__nv_bfloat16>(a, D, interleaved == 0, st);
  return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}
