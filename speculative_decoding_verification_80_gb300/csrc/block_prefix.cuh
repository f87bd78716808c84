// block_prefix.cuh — prefix sums over a CTA, for what is planned a request or
// a block at a time (kv_block_step, kv_fork).
#pragma once
#include <stdint.h>

namespace specdec {

constexpr int kBlockThreads = 1024;

// Sums that stay at the largest int: what they are compared with is no larger.
__device__ __forceinline__ uint32_t capped_sum(uint32_t x, uint32_t y) { return min(x + y, 0x7FFFFFFFu); }

// Exclusive prefix sums over the block of N values a thread (each at most the
// largest int); `total` are the sums.  `part` holds a warp's sums each, and
// then those before it.
template <int N>
__device__ __forceinline__ void block_prefix(const uint32_t (&x)[N], uint32_t (*part)[N], uint32_t (&before)[N], uint32_t (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = x[i];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, s[i], d);
      if (lane >= d) s[i] = capped_sum(s[i], o);
    }
  }
  __syncthreads();  // the last use of `part` is over
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[warp + 1][i] = s[i];
  }
  __syncthreads();
  if (warp < N) {
    uint32_t w = part[lane + 1][warp];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if (lane >= d) w = capped_sum(w, o);
    }
    part[lane + 1][warp] = w;
    if (lane == 0) part[0][warp] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = part[32][i];
    const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, s[i], 1);
    before[i] = capped_sum(part[warp][i], lane > 0 ? up : 0);
  }
}
static_assert(kBlockThreads / 32 == 32, "a lane for each warp");

}  // namespace specdec
