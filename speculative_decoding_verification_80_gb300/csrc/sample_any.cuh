// sample_any.cuh — a row of spec_sample, whatever is in it, by one CTA.  Right for
// every row and slow: several passes and many barriers.  One row of 128256 logits takes
// 0.10 to 0.14 ms where some are infinite, 0.15 to 0.3 in most other cases (the rows of
// logits less their largest, in bf16; flat fp32 rows away from 0) and 0.5 to 0.94 where
// one or two values are most of the row, whose additions in shared memory wait for one
// another.  (sample_kernel.cuh has the usual rows, in 0.02 to 0.06, and gives those to
// this that its bins cannot tell apart.)
//
// A histogram over the weights' exponent gives the bin in which a border lies, then
// one over the keys of that bin's ids, in three steps of 11, 11 and 10 bits, the
// logit; ids of that logit are counted in their order.
#pragma once
#include "sample_row.cuh"

namespace specdec {

constexpr int kSampleBins = 2048;  // 1/32 of a power of two each
constexpr int kSampleList = 4096;  // ids of a bin that are kept in shared memory

struct SampleShared {
  uint32_t count[kSampleBins];
  uint32_t lo[kSampleBins], hi[kSampleBins];  // halves of the sums
  uint32_t list[kSampleList];
  ExpPair table[256];
  unsigned long long warp_sum[kSampleWarps + 1];
  uint32_t warp_count[kSampleWarps + 1];
  // answers
  unsigned long long sum_before;
  uint32_t count_before, bin, ids, listed;
  float best[kSampleWarps];
};

__device__ __forceinline__ void add_weight(SampleShared& s, int bin, unsigned long long w) {
  const uint32_t lo = static_cast<uint32_t>(w);
  uint32_t hi = static_cast<uint32_t>(w >> 32);
  if (lo != 0) {
    const uint32_t old = atomicAdd(&s.lo[bin], lo);
    hi += old + lo < old ? 1 : 0;
  }
  if (hi != 0) atomicAdd(&s.hi[bin], hi);
}

// Sums over the CTA of a count and a weight before each thread's own, and the
// whole.  All threads call it.
__device__ __forceinline__ void sample_prefix(SampleShared& s, uint32_t c, unsigned long long w, uint32_t* c_before,
                                              unsigned long long* w_before, uint32_t* c_all, unsigned long long* w_all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t cs = c;
  unsigned long long ws = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t co = __shfl_up_sync(0xFFFFFFFFu, cs, d);
    const unsigned long long wo = __shfl_up_sync(0xFFFFFFFFu, ws, d);
    if (lane >= d) cs += co, ws += wo;
  }
  __syncthreads();
  if (lane == 31) s.warp_count[warp] = cs, s.warp_sum[warp] = ws;
  __syncthreads();
  uint32_t cb = 0, ca = 0;
  unsigned long long wb = 0, wa = 0;
#pragma unroll
  for (int i = 0; i < kSampleWarps; ++i) {
    if (i == warp) cb = ca, wb = wa;
    ca += s.warp_count[i];
    wa += s.warp_sum[i];
  }
  *c_before = cb + cs - c;
  *w_before = wb + ws - w;
  *c_all = ca;
  *w_all = wa;
}

// The bins in shared memory with the sums before each, in registers.
constexpr int kBinsOfThread = kSampleBins / kSampleThreads;
struct BinSums {
  uint32_t c[kBinsOfThread + 1];
  unsigned long long w[kBinsOfThread + 1];
  uint32_t c_all;
  unsigned long long w_all;
};
__device__ __forceinline__ void sum_bins(SampleShared& s, BinSums& b) {
  const int first = threadIdx.x * kBinsOfThread;
  uint32_t c[kBinsOfThread], ct = 0;
  unsigned long long w[kBinsOfThread], wt = 0;
#pragma unroll
  for (int i = 0; i < kBinsOfThread; ++i) {
    c[i] = s.count[first + i];
    w[i] = (static_cast<unsigned long long>(s.hi[first + i]) << 32) + s.lo[first + i];
    ct += c[i];
    wt += w[i];
  }
  sample_prefix(s, ct, wt, &b.c[0], &b.w[0], &b.c_all, &b.w_all);
#pragma unroll
  for (int i = 0; i < kBinsOfThread; ++i) b.c[i + 1] = b.c[i] + c[i], b.w[i + 1] = b.w[i] + w[i];
}
__device__ __forceinline__ void clear_bins(SampleShared& s) {
  for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads) s.count[i] = s.lo[i] = s.hi[i] = 0;
}

// What a border is counted in: ids up to `target` of them (1 and on), or weight
// up to `target` of it, or more than `target` of it; or the logits from the key
// `target` on.
enum SampleBorder { kByCount, kBySumTo, kBySumPast, kByKey };

// Whether a running value passes the border between `before` and `after`.
__device__ __forceinline__ bool crosses(SampleBorder by, uint32_t c0, uint32_t c1, unsigned long long w0,
                                        unsigned long long w1, unsigned long long target) {
  if (by == kByCount) return c0 < target && target <= c1;
  if (by == kBySumTo) return w0 < target && target <= w1;
  return w0 <= target && target < w1;
}

// The bin in which the border lies, for all threads; the sums before it are in s.
// One bin has to be the answer.
__device__ __forceinline__ int find_bin(SampleShared& s, const BinSums& b, SampleBorder by, unsigned long long target) {
#pragma unroll
  for (int i = 0; i < kBinsOfThread; ++i)
    if (crosses(by, b.c[i], b.c[i + 1], b.w[i], b.w[i + 1], target)) {
      s.bin = threadIdx.x * kBinsOfThread + i;
      s.count_before = b.c[i];
      s.sum_before = b.w[i];
      s.ids = b.c[i + 1] - b.c[i];
    }
  __syncthreads();
  return s.bin;
}

// A place in the order: ids of larger keys, then the first `ids` of those of `key`.
struct SamplePlace {
  uint32_t key, ids, all;        // all: ids of that key
  unsigned long long sum;        // weight before the key's ids
};
// All ids: as many of the least finite logit as there may be.
constexpr uint32_t kAnyIds = 0xFFFFFFFFu;

template <typename Elt>
struct Sampler {
  static constexpr int E = SampleRow<Elt>::E;
  SampleShared& s;
  const SampleRow<Elt> row;
  float top;       // the largest logit in the unit, 0 if it is infinite
  bool infinite;   // it is infinite: the others have no weight
  WeightScale scale;
  float unit;      // what logits are taken times

  __device__ __forceinline__ float relative(float x) const { return infinite ? (x == INFINITY ? 0.f : -INFINITY) : x; }
  __device__ __forceinline__ unsigned long long weight(float x) const { return sample_weight(x * unit, top, scale, s.table); }
  // (monotone: each step rounds a monotone function)
  __device__ __forceinline__ int bin_of(float x) const {
    const float t = (x * unit - top) * (scale.hi * -32.f);
    return t < static_cast<float>(kSampleBins - 1) ? static_cast<int>(t) : kSampleBins - 1;
  }

  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
    for (int j = threadIdx.x; j < row.vecs; j += kSampleThreads) {
      float x[E];
      row.load(j, x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(relative(x[e]), E * j + e - row.phase);
    }
  }

  // Within the bin that find_bin gave: the key at which the border lies.
  __device__ __forceinline__ SamplePlace refine(SampleBorder by, unsigned long long target) {
    const int bin = s.bin;
    const uint32_t ids = s.ids;
    uint32_t c0 = s.count_before;
    unsigned long long w0 = s.sum_before;
    const bool in_list = ids <= kSampleList;
    __syncthreads();
    if (in_list) {
      if (threadIdx.x == 0) s.listed = 0;
      __syncthreads();
      each([&](float x, int) {
        if (x != -INFINITY && bin_of(x) == bin) s.list[atomicAdd(&s.listed, 1)] = key_of(x);
      });
    }
    uint32_t key = 0, all = 0;
    int shift = 32;
#pragma unroll 1
    for (int bits = 11; shift > 0; bits = shift < 11 ? shift : 11) {
      const uint32_t above = key;  // the bits found so far
      const int was = shift;
      shift -= bits;
      __syncthreads();
      clear_bins(s);
      __syncthreads();
      auto one = [&](uint32_t k) {
        if (was < 32 && (k >> was) != (above >> was)) return;
        // the largest first
        const int at = ((1 << bits) - 1) - static_cast<int>((k >> shift) & ((1u << bits) - 1));
        atomicAdd(&s.count[at], 1u);
        if (by != kByCount) add_weight(s, at, weight(of_key(k)));
      };
      if (in_list) {
        for (uint32_t i = threadIdx.x; i < ids; i += kSampleThreads) one(s.list[i]);
      } else {
        each([&](float x, int) {
          if (x != -INFINITY && bin_of(x) == bin) one(key_of(x));
        });
      }
      __syncthreads();
      BinSums b;
      sum_bins(s, b);
      int at;
      if (by == kByKey) {
        // the bin that the key itself is in, whether it has ids or not
        at = ((1 << bits) - 1) - static_cast<int>((static_cast<uint32_t>(target) >> shift) & ((1u << bits) - 1));
        if (at / kBinsOfThread == threadIdx.x) {
#pragma unroll
          for (int i = 0; i < kBinsOfThread; ++i)
            if (i == at % kBinsOfThread) s.count_before = b.c[i], s.sum_before = b.w[i], s.ids = b.c[i + 1] - b.c[i];
        }
        __syncthreads();
      } else {
        unsigned long long rest = target - (by == kByCount ? c0 : w0);
        at = find_bin(s, b, by, rest);
      }
      c0 += s.count_before;
      w0 += s.sum_before;
      all = s.ids;
      key = above | (static_cast<uint32_t>(((1 << bits) - 1) - at) << shift);
    }
    __syncthreads();
    SamplePlace p;
    p.key = key;
    p.all = all;
    p.sum = w0;
    if (by == kByCount) {
      p.ids = static_cast<uint32_t>(target) - c0;
    } else if (by == kByKey) {
      p.ids = all;
    } else {
      const unsigned long long w = weight(of_key(key)), rest = target - w0;
      p.ids = static_cast<uint32_t>(by == kBySumTo ? (rest + w - 1) / w : rest / w + 1);
    }
    return p;
  }

  // The id of the nth (1 and on) of the ids with this key, in their order.
  __device__ __forceinline__ int nth(uint32_t key, uint32_t n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = (row.vecs + kSampleWarps - 1) / kSampleWarps, j0 = min(warp * share, row.vecs), j1 = min(j0 + share, row.vecs);
    uint32_t mine = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      float x[E];
      row.load(j, x);
#pragma unroll
      for (int e = 0; e < E; ++e) mine += x[e] != -INFINITY && key_of(relative(x[e])) == key ? 1 : 0;
    }
    mine = __reduce_add_sync(0xFFFFFFFFu, mine);
    __syncthreads();
    if (lane == 0) s.warp_count[warp] = mine;
    if (threadIdx.x == 0) s.bin = 0;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < warp; ++i) before += s.warp_count[i];
    if (before < n && n <= before + mine) {
      uint32_t left = n - before;
      for (int j = j0; j < j1; j += 32) {
        float x[E];
        uint32_t here = 0;
        if (j + lane < j1) {
          row.load(j + lane, x);
#pragma unroll
          for (int e = 0; e < E; ++e) here += x[e] != -INFINITY && key_of(relative(x[e])) == key ? 1 : 0;
        }
        uint32_t upto = here;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= d) upto += o;
        }
        if (here != 0 && upto - here < left && left <= upto) {
          uint32_t k = upto - here;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (x[e] != -INFINITY && key_of(relative(x[e])) == key && ++k == left) s.bin = E * (j + lane) + e - row.phase;
        }
        const uint32_t sum = __shfl_sync(0xFFFFFFFFu, upto, 31);
        if (left <= sum) break;
        left -= sum;
      }
    }
    __syncthreads();
    const int id = s.bin;
    __syncthreads();
    return id;
  }
};

// The row with -infinity for the ids that are not kept: keys above `key`, and ids up
// to `last` of those that have it, keep their bits (-0 is 0 in the order alone).
template <typename Elt>
__device__ __forceinline__ void write_cut_row(const SampleRow<Elt>& row, Elt* out, uint32_t key, int last, bool infinite) {
  constexpr int E = SampleRow<Elt>::E;
  const Elt none = static_cast<Elt>(-INFINITY);
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == row.phase * sizeof(Elt);
  for (int j = threadIdx.x; j < row.vecs; j += kSampleThreads) {
    const int first = E * j - row.phase;
    const bool whole = first >= 0 && first + E <= row.V;
    __align__(16) Elt y[E];
    if (whole) {
      *reinterpret_cast<uint4*>(y) = reinterpret_cast<const uint4*>(row.p)[j];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = first + e >= 0 && first + e < row.V ? row.p[static_cast<long long>(E) * j + e] : none;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = plain_logit(static_cast<float>(y[e])), r = infinite ? (x == INFINITY ? 0.f : -INFINITY) : x;
      const uint32_t k = key_of(r);
      if (!(r != -INFINITY && (k > key || (k == key && first + e <= last)))) y[e] = none;
    }
    if (same && whole) {
      *reinterpret_cast<uint4*>(out + first) = *reinterpret_cast<const uint4*>(y);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (first + e >= 0 && first + e < row.V) out[first + e] = y[e];
    }
  }
}

// For a top-k of 2 and more and a temperature above 0.  Returns false for a row
// without a number above -infinity.
template <typename Elt>
__device__ __noinline__ bool sample_any(SampleShared& s, const SampleRow<Elt> row, const SampleAsk ask, Elt* out, int32_t* token) {
  constexpr int E = SampleRow<Elt>::E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();
  if (tid < 256) s.table[tid] = kExp2Table[tid];
  float best = -INFINITY;
#pragma unroll 4
  for (int v = tid; v < row.vecs; v += kSampleThreads) {
    float x[E];
    row.load(v, x);
#pragma unroll
    for (int e = 0; e < E; ++e) best = fmaxf(best, x[e]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, d));
  if (lane == 0) s.best[warp] = best;
  clear_bins(s);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < kSampleWarps; ++i) best = fmaxf(best, s.best[i]);
  const bool infinite = best == INFINITY;
  if (best == -INFINITY) {
    if (tid == 0 && token != nullptr) *token = -1;
    if (out != nullptr) write_cut_row(row, out, kKeyFloor, -1, false);
    return false;
  }

  Sampler<Elt> f = {s, row, infinite ? 0.f : best * ask.unit, infinite, ask.scale, ask.unit};
  f.each([&](float x, int) {
    if (x == -INFINITY) return;
    const int bin = f.bin_of(x);
    atomicAdd(&s.count[bin], 1u);
    add_weight(s, bin, f.weight(x));
  });
  __syncthreads();
  BinSums sums;
  sum_bins(s, sums);
  // what is kept: larger keys, and the first ids of this one; its weight
  SamplePlace kept = {kKeyFloor + 1, kAnyIds, 0, 0};
  unsigned long long weight = sums.w_all;
  if (static_cast<uint32_t>(ask.k) < sums.c_all) {
    find_bin(s, sums, kByCount, ask.k);
    // (the sums before the key are needed as well: by key, once it is known)
    kept = f.refine(kByCount, ask.k);
    const uint32_t ids = kept.ids;
    const int bin = f.bin_of(of_key(kept.key));
    __syncthreads();
    if (bin / kBinsOfThread == tid) {
#pragma unroll
      for (int i = 0; i < kBinsOfThread; ++i)
        if (i == bin % kBinsOfThread) s.bin = bin, s.count_before = sums.c[i], s.sum_before = sums.w[i], s.ids = sums.c[i + 1] - sums.c[i];
    }
    __syncthreads();
    kept = f.refine(kByKey, kept.key);
    kept.ids = ids;
    weight = kept.sum + ids * f.weight(of_key(kept.key));
  }
  if (ask.p < 1.f) {
    const double goal = ceil(static_cast<double>(ask.p) * static_cast<double>(weight));
    unsigned long long target = static_cast<unsigned long long>(goal);
    target = target < 1 ? 1 : (target > weight ? weight : target);
    __syncthreads();
    find_bin(s, sums, kBySumTo, target);
    const SamplePlace at = f.refine(kBySumTo, target);
    // (a beginning of what top-k left)
    if (at.key > kept.key || (at.key == kept.key && at.ids < kept.ids)) {
      kept = at;
      weight = kept.sum + kept.ids * f.weight(of_key(kept.key));
    }
  }
  if (ask.least > 0 && f.weight(of_key(kept.key)) < ask.least) {
    // the least key with enough weight: 32 of them are looked at a time
    __syncthreads();
    if (warp == 0) {
      uint32_t no = kept.key, yes = key_of(infinite ? 0.f : best);  // no < yes; yes has enough
      while (yes - no > 1) {
        const uint32_t step = (yes - no + 31) / 32, at = no + step * (lane + 1);
        const bool enough = at >= yes || f.weight(of_key(at)) >= ask.least;
        const int first = __ffs(__ballot_sync(0xFFFFFFFFu, enough)) - 1;
        const uint32_t up = min(no + step * (first + 1), yes);
        no = no + step * first;
        yes = up;
      }
      if (lane == 0) s.listed = yes;
    }
    __syncthreads();
    const uint32_t key = s.listed;
    const int bin = f.bin_of(of_key(key));
    __syncthreads();
    if (bin / kBinsOfThread == tid) {
#pragma unroll
      for (int i = 0; i < kBinsOfThread; ++i)
        if (i == bin % kBinsOfThread) s.bin = bin, s.count_before = sums.c[i], s.sum_before = sums.w[i], s.ids = sums.c[i + 1] - sums.c[i];
    }
    __syncthreads();
    kept = f.refine(kByKey, key);
    weight = kept.sum + kept.ids * f.weight(of_key(kept.key));
  }
  if (token != nullptr) {
    unsigned long long target = static_cast<unsigned long long>(static_cast<double>(ask.u) * static_cast<double>(weight));
    if (target >= weight) target = weight - 1;
    __syncthreads();
    find_bin(s, sums, kBySumPast, target);
    const SamplePlace at = f.refine(kBySumPast, target);
    const int id = f.nth(at.key, at.ids);
    if (tid == 0) *token = id;
  }
  if (out != nullptr) {
    const int last = kept.ids < kept.all ? f.nth(kept.key, kept.ids) : row.V;
    write_cut_row(row, out, kept.key, last, infinite);
  }
  return true;
}

}  // namespace specdec
