// rotary_kernel.cuh — rotary positions of queries and keys (spec_rotary).
//
// A pair (a, b) of a head's values at position p becomes
//   factor * (a cos - b sin, a sin + b cos),  angle = 2 pi p turns_i / 2^64,
// where turns_i is the pair's frequency as a 64-bit fraction of a turn: the low
// half of p * turns_i is the angle without its whole turns, exactly, at any
// position (a float angle at position 131072 is off by 2^-8).
//
// Bytes bound it: a token's heads share its sines, which a CTA makes once into shared
// memory, factor and all, and then has its 256 threads turn 16 bytes of pairs each, two
// loads and two stores.  Few pairs a token and many tokens: a CTA has several.  50000
// tokens of 40 heads of 128 in bf16 (1.02 GB) take 155 us, 6.6 TB/s; 512 in fp32 (21
// MB) 8.3 us and one 4.2, which are a launch, a position, the sines and the rows one
// after another.  Products and sums are in 32 bits, and rounded once to bf16.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace specdec {

struct RotaryArgs {
  const char* x[2];  // q, k
  char* y[2];
  long long x_token[2], x_head[2], y_token[2], y_head[2];  // strides in bytes
  int32_t T, heads[2];
  const int32_t* positions;
  const unsigned long long* turns;
  float factor;
  int32_t pairs;      // of a head
  int32_t units;      // of a head: vectors of pairs, then (to other memory) of values that are not turned
  int32_t turned;     // units of pairs among them
  int32_t group;      // tokens of a CTA
};

constexpr int kRotaryThreads = 256;
constexpr int kRotaryPairs = 2048;  // of a CTA's tokens, in shared memory
constexpr int kRotaryTokens = 8;    // of a CTA, at most

template <typename Elt, int N>
struct RotaryVec {
  __align__(N * sizeof(Elt)) Elt v[N];
};
__device__ __forceinline__ float rotary_value(float x) { return x; }
__device__ __forceinline__ float rotary_value(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename Elt>
__device__ __forceinline__ Elt rotary_round(float x);
template <>
__device__ __forceinline__ float rotary_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rotary_round<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N values a load; kHalf: value i is paired with value i + pairs, else 2 i with
// 2 i + 1.  A unit is N pairs of a head (two loads).
template <typename Elt, int N, bool kHalf>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a) {
  using Vec = RotaryVec<Elt, N>;
  __shared__ float2 turn[kRotaryPairs];
  __shared__ int32_t position[kRotaryTokens];
  const int tid = threadIdx.x, t0 = blockIdx.x * a.group, tokens = min(a.group, a.T - t0);
  for (int i = tid; i < tokens * a.pairs; i += kRotaryThreads) {
    const int t = i / a.pairs, c = i - t * a.pairs, p = a.positions[t0 + t];
    const int32_t angle = static_cast<int32_t>((static_cast<unsigned long long>(static_cast<uint32_t>(p)) * a.turns[c]) >> 32);
    float sn, cs;
    sincospif(static_cast<float>(angle) * 0x1p-31f, &sn, &cs);
    // (a unit's pairs lie `turned` apart, so that neighbouring lanes read neighbours)
    turn[t * a.pairs + (c % N) * a.turned + c / N] = make_float2(cs * a.factor, sn * a.factor);
    if (c == 0) position[t] = p;
  }
  __syncthreads();
  const int per_token = (a.heads[0] + a.heads[1]) * a.units;
  for (int i = tid; i < tokens * per_token; i += kRotaryThreads) {
    const int t = i / per_token, rest = i - t * per_token, head = rest / a.units, unit = rest - head * a.units;
    if (position[t] < 0) continue;
    const int w = head >= a.heads[0] ? 1 : 0, h = head - (w ? a.heads[0] : 0);
    const char* x = a.x[w] + (t0 + t) * a.x_token[w] + h * a.x_head[w];
    char* y = a.y[w] + (t0 + t) * a.y_token[w] + h * a.y_head[w];
    if (unit >= a.turned) {
      const long long at = (2LL * a.pairs + static_cast<long long>(unit - a.turned) * N) * sizeof(Elt);
      *reinterpret_cast<Vec*>(y + at) = *reinterpret_cast<const Vec*>(x + at);
      continue;
    }
    const float2* r = turn + t * a.pairs + unit;
    if (kHalf) {
      const int at = unit * N * sizeof(Elt), far = at + a.pairs * sizeof(Elt);
      Vec lo = *reinterpret_cast<const Vec*>(x + at), hi = *reinterpret_cast<const Vec*>(x + far);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 cs = r[e * a.turned];
        const float u = rotary_value(lo.v[e]), v = rotary_value(hi.v[e]);
        lo.v[e] = rotary_round<Elt>(u * cs.x - v * cs.y);
        hi.v[e] = rotary_round<Elt>(u * cs.y + v * cs.x);
      }
      *reinterpret_cast<Vec*>(y + at) = lo;
      *reinterpret_cast<Vec*>(y + far) = hi;
    } else {
      Elt z[2 * N];
      const int at = unit * 2 * N * sizeof(Elt);
      if (N == 1) {
        z[0] = reinterpret_cast<const Elt*>(x + at)[0];
        z[1] = reinterpret_cast<const Elt*>(x + at)[1];
      } else {
        const Vec l = reinterpret_cast<const Vec*>(x + at)[0], g = reinterpret_cast<const Vec*>(x + at)[1];
#pragma unroll
        for (int e = 0; e < N; ++e) z[e] = l.v[e], z[N + e] = g.v[e];
      }
      Vec o[2];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 cs = r[e * a.turned];
        const float u = rotary_value(z[2 * e]), v = rotary_value(z[2 * e + 1]);
        o[2 * e / N].v[2 * e % N] = rotary_round<Elt>(u * cs.x - v * cs.y);
        o[(2 * e + 1) / N].v[(2 * e + 1) % N] = rotary_round<Elt>(u * cs.y + v * cs.x);
      }
      reinterpret_cast<Vec*>(y + at)[0] = o[0];
      reinterpret_cast<Vec*>(y + at)[1] = o[1];
    }
  }
}

}  // namespace specdec
