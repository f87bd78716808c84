// sample_row.cuh — what spec_sample's kernels share: arguments, a row, keys.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "sample_weight.cuh"

namespace specdec {

struct SampleArgs {
  const void* logits;
  void* out;              // or NULL
  int32_t B, n_max, V;
  const int32_t* draft_len;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniform;   // or NULL
  int32_t* tokens;        // or NULL
  uint32_t* err;
};

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr uint32_t kKeyFloor = 0x007FFFFFu;  // -infinity's

// What is asked of a row, after the checks of its numbers.
struct SampleAsk {
  float u;
  float p;
  int k;                      // 1 .. V
  unsigned long long least;   // weight that min-p asks for, 0: none
  WeightScale scale;
  float unit;                 // sample_any: a power of two that logits are taken times, for that scale
};

// Larger for a larger number; finite x, or an infinity.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) != 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}

// NaN counts as -infinity, and -0 as 0.
__device__ __forceinline__ float plain_logit(float x) { return x == x ? x + 0.f : -INFINITY; }

template <typename Elt>
struct SampleRow {
  static constexpr int E = 16 / sizeof(Elt);
  const Elt* p;  // on 16 bytes: the row starts `phase` elements later
  int phase, V, vecs;

  __device__ __forceinline__ SampleRow(const Elt* row, int V_) : V(V_) {
    phase = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(Elt));
    p = row - phase;
    vecs = (phase + V + E - 1) / E;
  }
  // Logits of the ids E j - phase and on; -infinity where there are none.
  __device__ __forceinline__ void load(int j, float (&x)[E]) const {
    const int first = E * j - phase;
    if (first >= 0 && first + E <= V) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[j];  // (the row may be cut in place)
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(Elt) == 2) {
          x[(2 * i) % E] = plain_logit(__uint_as_float(w[i] << 16));
          x[(2 * i + 1) % E] = plain_logit(__uint_as_float(w[i] & 0xFFFF0000u));
        } else {
          x[i % E] = plain_logit(__uint_as_float(w[i]));
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        x[e] = first + e >= 0 && first + e < V ? plain_logit(static_cast<float>(p[static_cast<long long>(E) * j + e])) : -INFINITY;
    }
  }
};

}  // namespace specdec
