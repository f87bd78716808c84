// attention_kernel.cuh — attention of new tokens over the 8-bit paged cache
// (spec_attention).
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "kv_kernels.cuh"

namespace specdec {

struct AttnArgs {
  const __nv_bfloat16* q;
  long long q_stride;  // elements
  __nv_bfloat16* out;
  int32_t T, Hq, H, B;
  const int32_t* cu_tokens;
  const int32_t* kv_len;
  const int32_t* table;
  int32_t max_blocks, num_blocks, bs;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  float scale;
};

// Simple form: a warp per query row, one position at a time.
template <int D>
__global__ void __launch_bounds__(128) attention_simple_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (row >= static_cast<long long>(a.T) * a.Hq) return;
  const int t = static_cast<int>(row / a.Hq), hq = static_cast<int>(row % a.Hq);
  const int total = min(a.cu_tokens[a.B], a.T);
  if (t >= total || t < a.cu_tokens[0]) return;
  const int b = owner_of(a.cu_tokens, a.B, t);
  const long long last = min(static_cast<long long>(a.kv_len[b]) + (t - a.cu_tokens[b]),
                             static_cast<long long>(a.max_blocks) * a.bs - 1);
  const int h = hq / (a.Hq / a.H);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[t * a.q_stride + hq * D + lane * E + e]) * a.scale;
    o[e] = 0.f;
  }
  for (long long p = 0; p <= last; ++p) {
    const int block = a.table[static_cast<long long>(b) * a.max_blocks + p / a.bs];
    const bool there = block >= 0 && block < a.num_blocks;
    const long long tile = there ? static_cast<long long>(block) * a.H + h : 0;
    const long long at = (tile * a.bs + p % a.bs) * D + lane * E;
    const float ks = there ? a.k_scale[tile] : 0.f, vs = there ? a.v_scale[tile] : 0.f;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 f = there ? e4m3_values(*reinterpret_cast<const uint16_t*>(a.k_cache + at + e)) : make_float2(0.f, 0.f);
      s += q[e] * f.x + q[e + 1] * f.y;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= ks;
    const float m2 = fmaxf(m, s);
    const float f = expf(m - m2), w = expf(s - m2);
    m = m2;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = there ? e4m3_values(*reinterpret_cast<const uint16_t*>(a.v_cache + at + e)) : make_float2(0.f, 0.f);
      o[e] = o[e] * f + w * (x.x * vs);
      o[e + 1] = o[e + 1] * f + w * (x.y * vs);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[row * D + lane * E + e] = __float2bfloat16_rn(last >= 0 ? o[e] / l : 0.f);
}

}  // namespace specdec
