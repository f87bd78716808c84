// logits_kernel.cuh — penalties, biases and grammar masks on the rows that the
// verify step reads (spec_process_logits).
//
// A cluster of kLogitCtas CTAs holds one request's token counts in its shared
// memory, a 32-bit word for each vocabulary entry: CTA r owns entries
// [r * share, (r + 1) * share).  Every CTA reads its part of the history once
// and adds to the owner's words through distributed shared memory, so the
// history is read once a request, whatever its length.  Then each CTA streams
// its entries of all rows: a thread keeps the words of its 16 bytes in
// registers while it goes through the rows, whose loads do not depend on one
// another.  Bound by the rows' bytes, read and written once.
#pragma once
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace specdec {

constexpr int kLogitCtas = 8;        // CTAs of a cluster (the portable most)
constexpr int kLogitThreads = 512;
constexpr int kLogitRows = 4;        // rows in flight per thread
constexpr int kBiasList = 512;       // biases of a CTA's entries kept in shared memory
constexpr uint32_t kInPrompt = 1u << 31;
constexpr uint32_t kHasBias = 1u << 30;
constexpr uint32_t kCountMask = kHasBias - 1;

struct LogitArgs {
  const void* logits;
  void* out;
  int32_t B, n_max, V, history_stride;
  const int32_t* history;
  const int32_t* prompt_len;
  const int32_t* history_len;
  const int32_t* draft_tokens;
  const int32_t* draft_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_offsets;
  const int32_t* bias_ids;
  const float* bias_values;
  int32_t num_bias;
  const uint32_t* mask;
  int32_t mask_count, mask_words;
  const int32_t* mask_rows;
  uint32_t* err;
  int32_t share;     // vocabulary entries of a CTA, a multiple of 32
  int32_t row_step;  // row groups: cluster y takes rows y, y + row_step, ...
};

struct LogitParams {  // one request's penalties
  float rep, pres, freq;
};

// l after penalties; c is the token's word with the drafts before the row
// added.
__device__ __forceinline__ float penalised(float l, uint32_t word, float bias, const LogitParams& p) {
  const uint32_t c = word & kCountMask;
  if (c != 0 || (word & kInPrompt)) l = l > 0.f ? l / p.rep : l * p.rep;
  l -= p.freq * static_cast<float>(c);
  if (c != 0) l -= p.pres;
  return l + bias;
}

struct BiasList {
  int32_t id[kBiasList];
  float value[kBiasList];
  int32_t n;
};

// Sum of the biases of token v, in the order they are listed.
__device__ inline float bias_of(int v, const BiasList& list, const LogitArgs& a, int lo, int hi) {
  float s = 0.f;
  if (list.n <= kBiasList) {
    for (int i = 0; i < list.n; ++i)
      if (list.id[i] == v) s += list.value[i];
  } else {  // more than the list holds: all of the request's
    for (int i = lo; i < hi; ++i)
      if (__ldg(a.bias_ids + i) == v) s += __ldg(a.bias_values + i);
  }
  return s;
}

__device__ __forceinline__ float elt_to_float(float x) { return x; }
__device__ __forceinline__ float elt_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void float_to_elt(float x, float& y) { y = x; }
__device__ __forceinline__ void float_to_elt(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

template <typename Elt>
struct alignas(16) EltVec {
  static constexpr int N = 16 / sizeof(Elt);
  Elt e[N];
};

// kVec: rows are 16-byte aligned and whole vectors long; otherwise a thread
// takes one entry at a time.
template <typename Elt, bool kVec>
__global__ void __cluster_dims__(kLogitCtas, 1, 1) __launch_bounds__(kLogitThreads)
    process_logits_kernel(const LogitArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t words[];
  __shared__ BiasList bl;
  constexpr int N = kVec ? EltVec<Elt>::N : 1;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = static_cast<int>(blockIdx.x) / kLogitCtas;
  const int tid = threadIdx.x;
  const int v0 = rank * a.share;
  const int v1 = min(a.V, v0 + a.share);  // may be <= v0

  uint32_t bad = 0;
  int n_b = a.n_max;
  if (a.draft_len != nullptr) {
    n_b = __ldg(a.draft_len + b);
    if (n_b < 0 || n_b > a.n_max) {
      bad = 1;
      n_b = max(0, min(n_b, a.n_max));
    }
  }
  LogitParams p;
  p.rep = a.repetition != nullptr ? __ldg(a.repetition + b) : 1.f;
  p.pres = a.presence != nullptr ? __ldg(a.presence + b) : 0.f;
  p.freq = a.frequency != nullptr ? __ldg(a.frequency + b) : 0.f;
  if (!(p.rep > 0.f) || isinf(p.rep)) bad = 1, p.rep = 1.f;
  if (!isfinite(p.pres)) bad = 1, p.pres = 0.f;
  if (!isfinite(p.freq)) bad = 1, p.freq = 0.f;
  int hist = 0, prompt = 0;
  if (a.history_stride > 0) {
    hist = __ldg(a.history_len + b);
    prompt = __ldg(a.prompt_len + b);
    if (hist < 0 || hist > a.history_stride || prompt < 0 || prompt > hist) bad = 1;
    hist = max(0, min(hist, a.history_stride));
    prompt = max(0, min(prompt, hist));
  }
  int lo = 0, hi = 0;
  if (a.bias_offsets != nullptr) {
    lo = __ldg(a.bias_offsets + b);
    hi = __ldg(a.bias_offsets + b + 1);
    if (lo < 0 || hi < lo || hi > a.num_bias) {
      bad = 1;
      lo = max(0, min(lo, a.num_bias));
      hi = max(lo, min(hi, a.num_bias));
    }
  }
  if (bad && a.err != nullptr && rank == 0 && blockIdx.y == 0 && tid == 0)
    atomicOr(a.err, SPECDEC_DEV_ERR_PENALTY);

  for (int i = tid; i < a.share / 4; i += kLogitThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) bl.n = 0;
  cluster.sync();

  // The history, once per cluster.
  const int32_t* h = a.history + static_cast<long long>(b) * a.history_stride;
  for (int i = rank * kLogitThreads + tid; i < hist; i += kLogitCtas * kLogitThreads) {
    const int v = __ldg(h + i);
    if (v < 0 || v >= a.V) continue;
    const int owner = v / a.share;
    uint32_t* w = cluster.map_shared_rank(words, owner) + (v - owner * a.share);
    if (i < prompt)
      atomicOr(w, kInPrompt);
    else
      atomicAdd(w, 1u);
  }
  // This CTA's biases, in their order (the first warp).
  if (tid < 32) {
    int n = 0;
    for (int i = lo + tid; i - tid < hi; i += 32) {
      const int v = i < hi ? __ldg(a.bias_ids + i) : -1;
      const bool mine = v >= v0 && v < v1;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
      if (mine) {
        const int at = n + __popc(m & ((1u << tid) - 1));
        if (at < kBiasList) {
          bl.id[at] = v;
          bl.value[at] = __ldg(a.bias_values + i);
        }
        atomicOr(words + (v - v0), kHasBias);
      }
      n += __popc(m);
    }
    if (tid == 0) bl.n = n;
  }
  cluster.sync();

  const Elt* in = static_cast<const Elt*>(a.logits) + static_cast<long long>(b) * (a.n_max + 1) * a.V;
  Elt* out = static_cast<Elt*>(a.out) + static_cast<long long>(b) * (a.n_max + 1) * a.V;
  const int32_t* x = a.draft_tokens + static_cast<long long>(b) * a.n_max;
  const int32_t* mr = a.mask_rows + static_cast<long long>(b) * (a.n_max + 1);
  const bool in_place = a.out == a.logits;

  for (int v = v0 + tid * N; v < v1; v += kLogitThreads * N) {
    uint32_t w[N];
    uint32_t any = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) any |= w[e] = words[v - v0 + e];
    float bias[N];
#pragma unroll
    for (int e = 0; e < N; ++e) bias[e] = 0.f;
    if (any & kHasBias) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (w[e] & kHasBias) bias[e] = bias_of(v + e, bl, a, lo, hi);
    }
    int counted = 0;  // drafts already in w
    for (int j0 = blockIdx.y; j0 <= n_b; j0 += kLogitRows * a.row_step) {
      EltVec<Elt> r[kLogitRows];
      uint32_t allow[kLogitRows];
#pragma unroll
      for (int k = 0; k < kLogitRows; ++k) {
        const int j = j0 + k * a.row_step;
        allow[k] = 0xFFFFFFFFu;
        if (j <= n_b) {
          if (kVec)
            r[k] = *reinterpret_cast<const EltVec<Elt>*>(in + static_cast<long long>(j) * a.V + v);
          else
            r[k].e[0] = in[static_cast<long long>(j) * a.V + v];
          if (a.mask_rows != nullptr) {
            const int m = __ldg(mr + j);
            if (m >= 0 && m < a.mask_count)
              allow[k] = __ldg(a.mask + static_cast<long long>(m) * a.mask_words + (v >> 5)) >> (v & 31);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kLogitRows; ++k) {
        const int j = j0 + k * a.row_step;
        if (j > n_b) break;
        for (; counted < j; ++counted) {
          const uint32_t d = static_cast<uint32_t>(__ldg(x + counted) - v);
          if (d < static_cast<uint32_t>(N)) {
            any |= 1;
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (d == static_cast<uint32_t>(e)) ++w[e];
          }
        }
        const uint32_t all = N == 32 ? 0xFFFFFFFFu : (1u << N) - 1;
        const bool masked = (allow[k] & all) != all;
        if (any) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (w[e]) float_to_elt(penalised(elt_to_float(r[k].e[e]), w[e], bias[e], p), r[k].e[e]);
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (!((allow[k] >> e) & 1)) float_to_elt(-INFINITY, r[k].e[e]);
        }
        if (in_place && !any && !masked) continue;
        if (kVec)
          *reinterpret_cast<EltVec<Elt>*>(out + static_cast<long long>(j) * a.V + v) = r[k];
        else
          out[static_cast<long long>(j) * a.V + v] = r[k].e[0];
      }
    }
  }
}

}  // namespace specdec
