// sample_kernel.cuh — tokens drawn with temperature, top-k, top-p and min-p from
// given random numbers, and the rows cut to what may be drawn (spec_sample).
//
// What a row keeps is a beginning of its ids in order of their logits (equal ones
// in order of the ids), and the token drawn is where that order's running sum of
// weights passes a share of the whole.  So everything is one question, asked up to
// four times: at which id of the order does a running count or sum pass a border?
// It is answered without sorting, from a histogram of the logits' first 16 bits
// (a bf16 logit whole) in shared memory, largest first:
//
//   - bf16: ids of a bin have one logit and so one weight, which is made once a bin
//     and not once an id; a border's bin is its logit.
//   - fp32: a second pass adds every id's weight to its bin, or lists the ids that
//     top-k or min-p can keep and adds theirs; the ids of a border's bin are listed
//     and looked at one by one.
//
// Groups of 16 bins have their sums in shared memory too, so that a warp finds a
// border by itself, in three looks of its lanes, without a barrier.  The row is
// written in a last pass, which marks where ids of the borders' logits are: those
// past a border in the order of the ids are taken back, and one is the token (fp32
// tokens mostly come from the list of a bin's ids).
//
// A row is one cluster's of 1 to 8 CTAs (the rule is where it is launched); each has
// a part of the row, a histogram of it, and a share of the bins to add up.  Two CTAs
// an SM, with 64 registers a thread (28 bytes of bf16's and 16 of fp32's are spilt):
// three with 40 spilt more and were slower (58 us instead of 48 on the 256 rows below),
// four had no room for the bins.
//
// Measured on one GB300, cut rows written back: one row of 128256 bf16 logits 18.5 us,
// 256 rows 48 (131 MB, 2.8 TB/s), 832 of 152064 141 (506 MB, 3.6 TB/s).  A row's chain
// of barriers and looks takes 12 to 14 us of its 34 to 45; the histogram takes 20 (a
// warp's 32 additions in shared memory some 4 cycles), the pass that writes 11 to 30.
// Tokens alone of 300 fp32 rows of 50001 (60 MB) take 80 us from L2 and 93 from HBM; a
// row that top-p alone cuts takes 67 of them, 38 for all its weights (some 75
// instructions each), and 15 for two lists of a bin's ids, each a pass over the row.
// What was no faster: 16384 bins, lists of the bins that have ids, shorter weights for
// small ones, clusters of two for many rows (300 fp32 rows: 115 us), ids looked at by
// several lanes each.
#pragma once
#include <cooperative_groups.h>

#include "sample_any.cuh"

namespace specdec {

constexpr int kSampleClusterMax = 8;
constexpr int kNear = 512;    // ids of a border's bin that are listed (fp32)
constexpr int kSampleGroups = kSampleThreads;  // of neighbouring bins, whose sums are kept

// Of the halves of two words.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bins of a logit's first 16 bits, the largest first: magnitudes from 2^12 down
// have one for each 7 bits of mantissa; what is above is in the outermost bins and
// what is below in the two of zero.
template <typename Elt>
struct SampleBinsOf {
  static constexpr int kBins = 8192;
  static constexpr int kHalf = kBins / 2;
  static constexpr uint32_t kTop = (127 + 12) << 7;          // 2^12 and above
  static constexpr uint32_t kBase = kTop - (kHalf - 1);      // about 2^-20 and below

  // A bin in 8 bits: a 16th of a power of two each, and all below 2^-4 in one.
  static __device__ __forceinline__ uint32_t coarse(uint32_t bin) { return min(bin >> 3, 255u); }

  // of two logits' bits at once, a half each
  static __device__ __forceinline__ uint32_t two(uint32_t w) {
    const uint32_t m = min_u16x2(max_u16x2(w & 0x7FFF7FFFu, kBase * 0x10001u), kTop * 0x10001u) - (kBase - kHalf) * 0x10001u;
    uint32_t negative;  // a mask in each half
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(negative) : "r"(w));
    return m ^ (~negative & (kBins - 1) * 0x10001u);
  }
  static __device__ __forceinline__ int one(float x) {
    const uint32_t b = __float_as_uint(x), m = min(max((b >> 16) & 0x7FFFu, kBase), kTop) - (kBase - kHalf);
    return static_cast<int>((b >> 31) != 0 ? m : m ^ (kBins - 1));
  }
  // the logit of a bin of a whole bf16 (not of those of zero and the outermost)
  static __device__ __forceinline__ float value(int bin) {
    const uint32_t m = static_cast<uint32_t>(bin < kHalf ? bin ^ (kBins - 1) : bin) - kHalf;
    const uint32_t b = m == 0 ? 0 : (m + kBase) | (bin < kHalf ? 0u : 0x8000u);
    return __uint_as_float(b << 16);
  }
};

template <typename Elt>
struct SampleBinsShared;
template <>
struct SampleBinsShared<__nv_bfloat16> {
  uint32_t count[8192];
};
template <>
struct SampleBinsShared<float> {
  union {
    uint32_t count[8192];
    // once the counts are done with: the logits that may be kept, or half as many with their ids
    float list[8192];
    struct {
      float list_half[4096];
      int32_t list_id[4096];
    };
  };
  uint32_t lo[8192], hi[8192];  // halves of the sums
  unsigned long long near_weight[kNear];
  uint32_t near_key[kNear];
  int32_t near_id[kNear];
};

// A bit for each vector of a CTA's part in which a border's logit is: in the bins'
// place, once these are done with.
constexpr int kMarkWords = (SPECDEC_MAX_VOCAB / 4 + 2 + 31) / 32;
static_assert(sizeof(uint32_t) * kMarkWords <= sizeof(SampleBinsShared<__nv_bfloat16>), "the marks lie where the bins were");

struct SampleAnswer {
  uint32_t key, ids, all, bad;
  unsigned long long sum;
};

template <typename Elt>
struct SampleFast {
  union {
    alignas(16) SampleBinsShared<Elt> bins;
    uint32_t marks[kMarkWords];
  };
  unsigned long long group_sum[kSampleGroups + 2];  // of 16 bins, then before them
  uint32_t group_count[kSampleGroups + 2];
  ExpPair table[256];
  unsigned long long warp_sum[kSampleWarps];
  uint32_t warp_count[kSampleWarps][2];
  // what the cluster's CTAs tell each other
  uint32_t top[kSampleClusterMax], flag[kSampleClusterMax];
  int32_t id[kSampleClusterMax];
  uint32_t same[kSampleClusterMax][2];
  uint32_t listed, gathered, least_key;
  unsigned long long zero[2];   // bf16: sums of the bins of zero
  bool zeroed;                  // they are in use
  SamplePlace kept, drawn;
  bool simple, more;
  SampleAnswer answer;
  WeightScale scale;
  unsigned long long least;
};

static_assert(offsetof(SampleFast<__nv_bfloat16>, bins) == 0 && sizeof(SampleBinsShared<__nv_bfloat16>) <= 32768, "16 bits address a count");

template <typename Elt>
union SampleSmem {
  SampleFast<Elt> fast;
  SampleShared any;
};

// A bin and what is before it.
struct SampleBin {
  int bin;
  uint32_t c0, c;
  unsigned long long w0, w;
};

// Of 16 warps' values in shared memory: the sum of those before this warp's, and of
// all.
template <typename T>
__device__ __forceinline__ T sum_of_warps(const T* each, int stride, T* all) {
  static_assert(kSampleWarps == 16, "a half of the lanes has a warp's each");
  const int lane = threadIdx.x & 15, warp = threadIdx.x >> 5;
  const T mine = each[lane * stride];
  T upto = mine;
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const T o = __shfl_up_sync(0xFFFFFFFFu, upto, d, 16);
    if (lane >= d) upto += o;
  }
  *all = __shfl_sync(0xFFFFFFFFu, upto, 15);
  return __shfl_sync(0xFFFFFFFFu, upto - mine, warp);
}

template <typename Elt>
struct SampleJob {
  using Bins = SampleBinsOf<Elt>;
  static constexpr int E = SampleRow<Elt>::E;
  static constexpr int kGroups = kSampleGroups;
  static constexpr int kOfGroup = Bins::kBins / kGroups;
  SampleFast<Elt>& s;
  uint8_t* largest_of;   // bf16: coarse bin of a vector's largest logit
  const SampleRow<Elt> row;
  cooperative_groups::cluster_group cluster;
  int ctas, rank;
  int j0, j1;       // this CTA's vectors
  float top;        // the largest logit
  WeightScale scale;
  int in_list = -1;             // fp32: logits in this CTA's list, -1: there is none
  bool with_ids = false;        // fp32: a border's ids are known when its bin is listed
  SampleBin of_k = {-1, 0, 0, 0, 0};  // fp32: top-k's bin and its counts

  __device__ __forceinline__ SampleFast<Elt>& of(int cta) const { return *cluster.map_shared_rank(&s, cta); }
  // That the others have begun, so that their memory may be written: said early, and
  // waited for late.
  __device__ __forceinline__ void say_begun() const {
    if (ctas > 1) asm volatile("barrier.cluster.arrive;" ::: "memory");
  }
  __device__ __forceinline__ void wait_begun() const {
    if (ctas > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
  }
  __device__ __forceinline__ void meet() const {
    __syncwarp();
    if (ctas > 1)
      cluster.sync();
    else
      __syncthreads();
  }
  __device__ __forceinline__ unsigned long long weight(float x) const { return sample_weight(x, top, scale, s.table); }

  // A vector's words, -infinity for ids that the row does not have.
  __device__ __forceinline__ uint4 words(int j) const {
    const int first = E * j - row.phase;
    if (first >= 0 && first + E <= row.V) return reinterpret_cast<const uint4*>(row.p)[j];
    constexpr uint32_t kNone = sizeof(Elt) == 2 ? 0xFF80FF80u : 0xFF800000u;
    uint32_t w[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (first + e >= 0 && first + e < row.V) {
        const uint32_t b = bits(row.p[E * j + e]);
        if (sizeof(Elt) == 2)
          w[e * 4 / E] = e & 1 ? (w[e * 4 / E] & 0xFFFFu) | b << 16 : (w[e * 4 / E] & 0xFFFF0000u) | b;
        else
          w[e % 4] = b;
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // f(words, j) for this CTA's vectors.  kAtOnce are on their way together, and f's
  // code is there as often: 1 for a long one, which asks for the next before its own.
  template <int kAtOnce, typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lo = max(j0, row.phase != 0 ? 1 : 0), hi = min(j1, (row.phase + row.V) / E);  // whole ones
    const uint4* p = reinterpret_cast<const uint4*>(row.p);
    int j = lo + threadIdx.x;
    if constexpr (kAtOnce > 1) {
#pragma unroll 1
      for (; j + (kAtOnce - 1) * kSampleThreads < hi; j += kAtOnce * kSampleThreads) {
        uint4 q[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) q[i] = p[j + i * kSampleThreads];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) f(q[i], j + i * kSampleThreads);
      }
    }
    // the rest, and the row's ends, one by one
    uint4 ahead = j < hi ? p[j] : make_uint4(0, 0, 0, 0);
    const int end = threadIdx.x == 0 && row.phase != 0 && j0 == 0 ? 0
                    : threadIdx.x == 32 && j1 == row.vecs && row.vecs > hi && (row.vecs > 1 || row.phase == 0) ? row.vecs - 1 : -1;
#pragma unroll 1
    while (true) {
      const bool inside = j < hi;
      if (!inside && end < 0) break;
      const uint4 q = inside ? ahead : words(end);
      const int at = inside ? j : end;
      if (inside) {
        j += kSampleThreads;
        if (j < hi) ahead = p[j];
      }
      f(q, at);
      if (!inside) break;
    }
  }
  static_assert(kNear <= kSampleThreads, "a thread for each listed id");
  static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ uint32_t bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
  static __device__ __forceinline__ float logit(uint32_t b) { return plain_logit(__uint_as_float(sizeof(Elt) == 2 ? b << 16 : b)); }
  // f(logit, id) for all of this CTA's ids, and for ids that the row does not have,
  // with -infinity.
  template <int kAtOnce, typename F>
  __device__ __forceinline__ void each_id(F f) const {
    each<kAtOnce>([&](const uint4& q, int j) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      const int id = E * j - row.phase;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(Elt) == 2) {
          f(logit(w[i] & 0xFFFFu), id + 2 * i);
          f(logit(w[i] >> 16), id + 2 * i + 1);
        } else {
          f(logit(w[i]), id + i);
        }
      }
    });
  }

  // A bin's count and sum, over the cluster, from the CTA that added them up.
  __device__ __forceinline__ void bin_of_cluster(int bin, uint32_t* c, unsigned long long* w) const {
    const SampleFast<Elt>& o = ctas > 1 ? of(bin / (Bins::kBins / ctas)) : s;
    *c = o.bins.count[bin];
    if constexpr (sizeof(Elt) == 2)
      *w = *c == 0 ? 0 : (s.zeroed && (bin == Bins::kHalf - 1 || bin == Bins::kHalf) ? s.zero[bin - (Bins::kHalf - 1)] : *c * weight(Bins::value(bin)));
    else
      *w = (static_cast<unsigned long long>(o.bins.hi[bin]) << 32) + o.bins.lo[bin];
  }

  // Adds the CTAs' histograms up, a share of the bins each, and the sums of every
  // group, which all CTAs get.  A group is one thread's, or as many threads' as
  // there are CTAs.
  // (fp32: the counts, and later the sums)
  __device__ __forceinline__ void add_up(bool counts, bool sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, of_thread = kOfGroup / ctas;
    const int me = rank * kSampleThreads + threadIdx.x;
    uint32_t cs = 0;
    unsigned long long ws = 0;
#pragma unroll 2
    for (int i = 0; i < of_thread; i += 2) {
      const int bin = me * of_thread + i;
      uint2 c = make_uint2(0, 0);
      unsigned long long w = 0, x = 0;
      for (int o = 0; o < ctas; ++o) {
        const SampleFast<Elt>& from = ctas > 1 ? of(o) : s;
        if (counts) {
          const uint2 d = *reinterpret_cast<const uint2*>(&from.bins.count[bin]);
          c.x += d.x, c.y += d.y;
        }
        if constexpr (sizeof(Elt) == 4) {
          if (sums) {
            const uint2 lo = *reinterpret_cast<const uint2*>(&from.bins.lo[bin]), hi = *reinterpret_cast<const uint2*>(&from.bins.hi[bin]);
            w += (static_cast<unsigned long long>(hi.x) << 32) + lo.x;
            x += (static_cast<unsigned long long>(hi.y) << 32) + lo.y;
          }
        }
      }
      if (ctas > 1) {
        if (counts) *reinterpret_cast<uint2*>(&s.bins.count[bin]) = c;
        if constexpr (sizeof(Elt) == 4) {
          if (sums) {
            *reinterpret_cast<uint2*>(&s.bins.lo[bin]) = make_uint2(static_cast<uint32_t>(w), static_cast<uint32_t>(x));
            *reinterpret_cast<uint2*>(&s.bins.hi[bin]) = make_uint2(static_cast<uint32_t>(w >> 32), static_cast<uint32_t>(x >> 32));
          }
        }
      }
      if constexpr (sizeof(Elt) == 2) {
        if ((c.x | c.y) != 0) w = c.x * weight(Bins::value(bin)), x = c.y * weight(Bins::value(bin + 1));
      }
      cs += c.x + c.y;
      ws += w + x;
    }
    for (int d = 1; d < ctas; d <<= 1) {
      cs += __shfl_xor_sync(0xFFFFFFFFu, cs, d);
      ws += __shfl_xor_sync(0xFFFFFFFFu, ws, d);
    }
    SampleFast<Elt>& to = ctas > 1 ? of(threadIdx.x % ctas) : s;
    if (counts) to.group_count[me / ctas] = cs;
    if (sums) to.group_sum[me / ctas] = ws;
    meet();
    // sums before each group
    static_assert(kGroups == kSampleThreads, "a thread for each group");
    const uint32_t c = s.group_count[threadIdx.x];
    const unsigned long long w = s.group_sum[threadIdx.x];
    cs = c;
    ws = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t co = __shfl_up_sync(0xFFFFFFFFu, cs, d);
      const unsigned long long wo = __shfl_up_sync(0xFFFFFFFFu, ws, d);
      if (lane >= d) cs += co, ws += wo;
    }
    if (lane == 31) s.warp_count[warp][0] = cs, s.warp_sum[warp] = ws;
    __syncthreads();
    uint32_t c_all;
    unsigned long long w_all;
    cs += sum_of_warps(&s.warp_count[0][0], 2, &c_all);
    ws += sum_of_warps(&s.warp_sum[0], 1, &w_all);
    if (counts) {
      s.group_count[threadIdx.x] = cs - c;
      if (threadIdx.x == 0) s.group_count[kGroups] = c_all;
    }
    if (sums) {
      s.group_sum[threadIdx.x] = ws - w;
      if (threadIdx.x == 0) s.group_sum[kGroups] = w_all;
    }
    __syncthreads();
  }
  // min-p's key, by the last warp.
  __device__ __forceinline__ void find_least(const SampleAsk& ask) {
    if (ask.least == 0 || threadIdx.x < kSampleThreads - 32) return;
    const uint32_t key = least_key(kKeyFloor, key_of(top), ask.least);
    if (threadIdx.x % 32 == 0) s.least_key = key;
  }

  // The least logit of a bin and those before it (fp32).
  static __device__ __forceinline__ float end_of(int bin) {
    if (bin >= Bins::kBins - 1) return -INFINITY;
    if (bin < Bins::kHalf) return Bins::value(bin);
    return __uint_as_float(0x80000000u | (static_cast<uint32_t>(bin - Bins::kHalf) + Bins::kBase) << 16 | 0xFFFFu);
  }
  // fp32: this CTA's logits from `least` on into its list, in any order.
  __device__ __forceinline__ void gather(float least) {
    if constexpr (sizeof(Elt) == 4) {
      constexpr int kAtOnce = 4, kRoom = Bins::kBins;
      const int lane = threadIdx.x & 31;
      const uint4 none = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
#pragma unroll 1
      for (int j = j0 + static_cast<int>(threadIdx.x); j - lane < j1; j += kAtOnce * kSampleThreads) {
        uint4 q[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) q[i] = j + i * kSampleThreads < j1 ? words(j + i * kSampleThreads) : none;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const float f[4] = {__uint_as_float(q[i].x), __uint_as_float(q[i].y), __uint_as_float(q[i].z), __uint_as_float(q[i].w)};
          uint32_t m[4], n = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) m[e] = __ballot_sync(0xFFFFFFFFu, f[e] >= least), n += __popc(m[e]);
          if (n == 0) continue;
          uint32_t at = 0;
          if (lane == 0) at = atomicAdd(&s.gathered, n);
          at = __shfl_sync(0xFFFFFFFFu, at, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t mine = at + __popc(m[e] & ((1u << lane) - 1));
            if (f[e] >= least && mine < kRoom) {
              s.bins.list[mine] = f[e] + 0.f;
              if (with_ids && mine < kRoom / 2) s.bins.list_id[mine] = E * (j + i * kSampleThreads) - row.phase + e;
            }
            at += __popc(m[e]);
          }
        }
      }
      __syncthreads();
      if (s.gathered <= kRoom) in_list = static_cast<int>(s.gathered);
    }
  }
  // fp32: the weights into the bins.  Of ids that cannot be kept none is needed: those
  // in a bin past top-k's, and, where no top-p asks for a share of them, min-p's.  The
  // others are listed in the counts' place, where there is room for them (and for their
  // ids, for half as many), and nothing but the last pass reads the row again.  (Of 50001 ids the weights of 5000 took 35
  // us a row, as those of all, when each warp gathered its own 32 at a time.)
  __device__ __forceinline__ void add_weights(const SampleAsk& ask) {
    if constexpr (sizeof(Elt) == 4) {
      float least = of_key(s.least_key);
      bool few = ask.least > 0 && !(ask.p < 1.f);
      if (ask.k < row.V) {
        add_up(true, false);
        if (find(kByCount, ask.k, &of_k)) {
          // (the border itself is looked for among them: min-p does not shorten the list)
          least = fmaxf(end_of(of_k.bin), -3.402823466e38f);  // (-infinity is no id's)
          few = of_k.c0 + of_k.c <= Bins::kBins;
          with_ids = of_k.c0 + of_k.c <= Bins::kBins / 2;
        } else {
          of_k.bin = -1;
        }
        meet();  // (the counts' readers)
      }
      if (few)
        gather(least);
      else
        with_ids = true;
      auto one = [&](float x) {
        const int bin = Bins::one(x);
        const unsigned long long w = weight(x);
        const uint32_t lo = static_cast<uint32_t>(w);
        uint32_t hi = static_cast<uint32_t>(w >> 32);
        if (lo != 0) {
          const uint32_t old = atomicAdd(&s.bins.lo[bin], lo);
          hi += old + lo < old ? 1 : 0;
        }
        if (hi != 0) atomicAdd(&s.bins.hi[bin], hi);
      };
      if (in_list >= 0) {
#pragma unroll 2
        for (int i = threadIdx.x; i < in_list; i += kSampleThreads) one(s.bins.list[i]);
      } else {
        // four chains of instructions a thread
        each_id<1>([&](float x, int) {
          if (x != -INFINITY) one(x);
        });
      }
      meet();
      add_up(false, true);
    }
  }
  __device__ __forceinline__ void clear_bins() {
    uint4* z = reinterpret_cast<uint4*>(&s.bins);
    constexpr int kClear = (sizeof(Elt) == 2 ? 1 : 3) * Bins::kBins / 4;
    for (int i = threadIdx.x; i < kClear; i += kSampleThreads) z[i] = make_uint4(0, 0, 0, 0);
  }

  // The bins of zero have logits up to 2^-20, whose weights differ by that over T.
  // Whether they matter, by a warp; then each id's own weight is added.  (One address
  // for all ids: a row of 128256 logits of which half are 0 takes 0.2 ms with top-k 50,
  // where one without zeros takes 0.02.)
  __device__ __forceinline__ bool zeros_matter(uint32_t (&c)[2], unsigned long long (&w)[2]) const {
    bin_of_cluster(Bins::kHalf - 1, &c[0], &w[0]);
    bin_of_cluster(Bins::kHalf, &c[1], &w[1]);
    return static_cast<float>(w[0] + w[1]) * scale.hi * 0x1p21f > static_cast<float>(s.group_sum[kGroups]);
  }
  __device__ __forceinline__ void add_zeros() {
    uint32_t c[2];
    unsigned long long w[2];
    zeros_matter(c, w);
    meet();
    auto one = [&](float x) {
      const int i = Bins::one(x) - (Bins::kHalf - 1);
      if (x == -INFINITY || (i != 0 && i != 1)) return;
      const unsigned long long mine = weight(x);
      for (int o = 0; o < ctas; ++o) atomicAdd(&of(o).zero[i], mine);
    };
    each<4>([&](const uint4& q, int) {
      const uint32_t v[4] = {q.x, q.y, q.z, q.w};
      uint32_t m = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = min_u16x2(m, v[i] & 0x7FFF7FFFu);
      if ((m & 0xFFFFu) > Bins::kBase && (m >> 16) > Bins::kBase) return;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const uint32_t p = e & 4 ? (e & 2 ? v[3] : v[2]) : (e & 2 ? v[1] : v[0]);
        one(logit(e & 1 ? p >> 16 : p & 0xFFFFu));
      }
    });
    meet();
    const unsigned long long more[2] = {s.zero[0] - w[0], s.zero[1] - w[1]};
    constexpr int kFirst = (Bins::kHalf - 1) / kOfGroup;
    for (int g = threadIdx.x; g <= kGroups; g += kSampleThreads) s.group_sum[g] += (g > kFirst ? more[0] : 0) + (g > kFirst + 1 ? more[1] : 0);
    if (threadIdx.x == 0) s.zeroed = true;
    __syncthreads();
  }
  __device__ __forceinline__ bool decide(const SampleAsk& ask, int32_t* token, SamplePlace* kept, SamplePlace* drawn);

  // The least key of a logit of `Elt` whose weight is enough, by a warp; `no` has too
  // little and `yes` enough.
  __device__ __forceinline__ uint32_t least_key(uint32_t no, uint32_t yes, unsigned long long least) const {
    // (keys of bf16 logits differ in their first half)
    constexpr int kShift = sizeof(Elt) == 2 ? 16 : 0;
    constexpr uint32_t kRest = (1u << kShift) - 1;
    const int lane = threadIdx.x & 31;
    // negative logits' keys end in ones, the others' in zeros
    auto logit = [&](uint32_t k) { return of_key(kShift == 0 ? k : (k << kShift) | ((k >> 15) != 0 ? 0 : kRest)); };
    no >>= kShift;
    yes >>= kShift;
    while (yes - no > 1) {
      const uint32_t step = (yes - no + 31) / 32, at = no + step * (lane + 1);
      const bool enough = at >= yes || weight(logit(at)) >= least;
      const int first = __ffs(__ballot_sync(0xFFFFFFFFu, enough)) - 1;
      yes = min(no + step * (first + 1), yes);
      no += step * first;
    }
    return key_of(logit(yes));
  }

  // The bin in which a border lies, by each warp for itself; false if there is none.
  __device__ __forceinline__ bool find(SampleBorder by, unsigned long long target, SampleBin* f) const {
    constexpr int kStep = kGroups / 32;
    const int lane = threadIdx.x & 31;
    auto passed = [&](uint32_t c, unsigned long long w) { return by == kByCount ? c >= target : (by == kBySumTo ? w >= target : w > target); };
    uint32_t m = __ballot_sync(0xFFFFFFFFu, passed(s.group_count[(lane + 1) * kStep], s.group_sum[(lane + 1) * kStep]));
    if (m == 0) return false;
    int g = (__ffs(m) - 1) * kStep;
    m = __ballot_sync(0xFFFFFFFFu, lane >= kStep - 1 || passed(s.group_count[g + lane + 1], s.group_sum[g + lane + 1]));
    g += __ffs(m) - 1;
    within(g, [&](uint32_t c0, uint32_t c1, unsigned long long w0, unsigned long long w1, int) { return passed(c1, w1); }, f);
    return true;
  }
  // The bin itself and what is before it.
  __device__ __forceinline__ void look_up(int bin, SampleBin* f) const {
    within(bin / kOfGroup, [&](uint32_t, uint32_t, unsigned long long, unsigned long long, int lane) { return lane >= bin % kOfGroup; }, f);
  }
  template <typename F>
  __device__ __forceinline__ void within(int g, F passed, SampleBin* f) const {
    const int lane = threadIdx.x & 31;
    uint32_t c = 0;
    unsigned long long w = 0;
    if (lane < kOfGroup) bin_of_cluster(kOfGroup * g + lane, &c, &w);
    uint32_t c1 = c;
    unsigned long long w1 = w;
#pragma unroll
    for (int d = 1; d < kOfGroup; d <<= 1) {
      const uint32_t co = __shfl_up_sync(0xFFFFFFFFu, c1, d);
      const unsigned long long wo = __shfl_up_sync(0xFFFFFFFFu, w1, d);
      if (lane >= d) c1 += co, w1 += wo;
    }
    c1 += s.group_count[g];
    w1 += s.group_sum[g];
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, lane >= kOfGroup - 1 || passed(c1 - c, c1, w1 - w, w1, lane));
    const int at = __ffs(m) - 1;
    f->bin = kOfGroup * g + at;
    f->c0 = __shfl_sync(0xFFFFFFFFu, c1 - c, at);
    f->c = __shfl_sync(0xFFFFFFFFu, c, at);
    f->w0 = __shfl_sync(0xFFFFFFFFu, w1 - w, at);
    f->w = __shfl_sync(0xFFFFFFFFu, w, at);
  }

  // The key at which a border lies within its bin; for kByKey the key is the border
  // and all ids from it on are before it.  False: the bin does not say (for all CTAs
  // alike).
  // With a `token` (fp32, kBySumPast) it is written where the ids are known, and the
  // place's key is 0.
  __device__ __forceinline__ bool resolve(const SampleBin& f, SampleBorder by, unsigned long long target, SamplePlace* p, int32_t* token = nullptr) {
    if constexpr (sizeof(Elt) == 2) {
      if (f.bin == 0 || f.bin >= Bins::kBins - 1 || f.bin == Bins::kHalf - 1 || f.bin == Bins::kHalf) return false;
      p->key = key_of(Bins::value(f.bin));
      p->all = f.c;
      p->sum = f.w0;
      const unsigned long long w = weight(Bins::value(f.bin));
      p->ids = by == kByCount ? static_cast<uint32_t>(target) - f.c0
                              : static_cast<uint32_t>(by == kByKey ? f.c : (by == kBySumTo ? (target - f.w0 + w - 1) / w : (target - f.w0) / w + 1));
      return true;
    } else {
      SampleFast<Elt>& lead = ctas > 1 ? of(0) : s;
      auto list = [&](float x, int id) {
        const uint32_t at = atomicAdd(&lead.listed, 1u);
        if (at < kNear) lead.bins.near_key[at] = key_of(x), lead.bins.near_id[at] = id;
      };
      if (in_list >= 0) {
        for (int i = threadIdx.x; i < in_list; i += kSampleThreads) {
          const float x = s.bins.list[i];
          if (Bins::one(x) == f.bin) list(x, with_ids ? s.bins.list_id[i] : 0);
        }
      } else if (f.bin == 0 || f.bin == Bins::kBins - 1 || f.bin == Bins::kHalf - 1 || f.bin == Bins::kHalf) {
        each_id<1>([&](float x, int id) {
          if (x != -INFINITY && Bins::one(x) == f.bin) list(x, id);
        });
      } else {  // a bin of one beginning of 16 bits
        const uint32_t first = __float_as_uint(Bins::value(f.bin)) & 0xFFFF0000u;
        each<8>([&](const uint4& q, int j) {
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((w[i] ^ first) < 0x10000u) list(__uint_as_float(w[i]), E * j - row.phase + i);
        });
      }
      meet();
      if (rank == 0) {
        const uint32_t n = s.listed;
        if (threadIdx.x == 0) s.answer.bad = n > kNear ? 1 : 0, s.answer.sum = 0;
        if (n <= kNear) {
          for (uint32_t i = threadIdx.x; i < n; i += kSampleThreads) s.bins.near_weight[i] = weight(of_key(s.bins.near_key[i]));
          __syncthreads();
          for (uint32_t i = threadIdx.x; i < n; i += kSampleThreads) {
            const uint32_t key = s.bins.near_key[i];
            const unsigned long long w = s.bins.near_weight[i];
            if (by == kByKey) {
              if (key >= static_cast<uint32_t>(target)) atomicAdd(&s.answer.sum, w);
              continue;
            }
            uint32_t c0 = 0, same = 0;
            unsigned long long w0 = 0;
#pragma unroll 2
            for (uint32_t o = 0; o < n; ++o) {
              const uint32_t other = s.bins.near_key[o];
              if (other > key) ++c0, w0 += s.bins.near_weight[o];
              if (other == key) ++same;
            }
            c0 += f.c0;
            w0 += f.w0;
            if (crosses(by, c0, c0 + same, w0, w0 + same * w, target)) {  // (one key, whose ids all say the same)
              s.answer.key = key;
              s.answer.all = same;
              s.answer.sum = w0;
              s.answer.ids = by == kByCount ? static_cast<uint32_t>(target) - c0
                                            : static_cast<uint32_t>(by == kBySumTo ? (target - w0 + w - 1) / w : (target - w0) / w + 1);
            }
          }
        }
        __syncthreads();
        if (by == kByKey && threadIdx.x == 0) {
          s.answer.key = static_cast<uint32_t>(target);
          s.answer.all = s.answer.ids = 0;
          s.answer.sum += f.w0;
        }
        if (token != nullptr && with_ids && n <= kNear && threadIdx.x < n && s.bins.near_key[threadIdx.x] == s.answer.key) {
          const int id = s.bins.near_id[threadIdx.x];
          uint32_t before = 0;
          for (uint32_t o = 0; o < n; ++o) before += s.bins.near_key[o] == s.answer.key && s.bins.near_id[o] < id ? 1 : 0;
          if (before + 1 == s.answer.ids) *token = id;
        }
        __syncthreads();
        if (ctas > 1 && threadIdx.x >= 32 && threadIdx.x < 32 * ctas && threadIdx.x % 32 == 0) of(threadIdx.x / 32).answer = s.answer;
        if (threadIdx.x == 0) s.listed = 0;
      }
      meet();
      const SampleAnswer a = s.answer;
      p->key = token != nullptr && with_ids ? 0 : a.key;
      p->ids = a.ids;
      p->all = a.all;
      p->sum = a.sum;
      return a.bad == 0;
    }
  }

  // Room for the marks, where no one reads the bins any more.
  __device__ __forceinline__ void clear_marks() {
    meet();
    for (int i = threadIdx.x; i <= (j1 - j0) / 32; i += kSampleThreads) s.marks[i] = 0;
    __syncthreads();
  }
  // This CTA's part of the row, -infinity for ids whose key is below `least_kept`;
  // vectors with ids of key[i], where there is one (not 0), are marked.
  __device__ __forceinline__ void write(Elt* out, uint32_t least_kept, const uint32_t (&key)[2]) {
    const bool same = out != nullptr && (reinterpret_cast<uintptr_t>(out) & 15) == row.phase * sizeof(Elt);
    const float least = of_key(least_kept), nan = __uint_as_float(0x7FFFFFFFu);
    const bool look = key[0] != 0 || key[1] != 0;
    const float tie[2] = {key[0] != 0 ? of_key(key[0]) : nan, key[1] != 0 ? of_key(key[1]) : nan};
    auto mark = [&](int j) { atomicOr(&s.marks[(j - j0) >> 5], 1u << ((j - j0) & 31)); };
    auto store = [&](const uint32_t (&w)[4], int first) {
      if (same && first >= 0 && first + E <= row.V) {
        *reinterpret_cast<uint4*>(out + first) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (first + e >= 0 && first + e < row.V) {
            if constexpr (sizeof(Elt) == 2)
              out[first + e] = __ushort_as_bfloat16(static_cast<unsigned short>(e & 1 ? w[e / 2] >> 16 : w[e / 2]));
            else
              out[first + e] = __uint_as_float(w[e]);
          }
      }
    };
    if constexpr (sizeof(Elt) == 2) {
      const __nv_bfloat162 least2 = __float2bfloat162_rn(least);  // (borders are bf16)
      const __nv_bfloat162 tie2[2] = {__float2bfloat162_rn(tie[0]), __float2bfloat162_rn(tie[1])};
      // vectors without a logit to keep, or to mark where nothing is kept, are not read
      const uint32_t read = Bins::coarse(Bins::one(out != nullptr ? least : tie[0]));
      constexpr int kAtOnce = 4;
#pragma unroll 1
      for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += kAtOnce * kSampleThreads) {
        uint4 q[kAtOnce];
        bool wanted[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int at = j + i * kSampleThreads;
          wanted[i] = at < j1 && largest_of[at - j0] <= read;
          q[i] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
          if (wanted[i]) q[i] = words(at);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int at = j + i * kSampleThreads;
          if (at >= j1) break;
          uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
          if (wanted[i]) {
            uint32_t tied = 0;
#pragma unroll
            for (int l = 0; l < 4; ++l) {
              const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[l]);
              tied |= __heq2_mask(x, tie2[0]) | __heq2_mask(x, tie2[1]);
              const uint32_t m = __hge2_mask(x, least2);
              w[l] = (w[l] & m) | (~m & 0xFF80FF80u);
            }
            if (look && tied != 0) mark(at);
          }
          if (out != nullptr) store(w, E * at - row.phase);
        }
      }
    } else {
      each<4>([&](const uint4& q, int j) {
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
        bool tied = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __uint_as_float(w[i]);
          tied |= x == tie[0] || x == tie[1];
          w[i] = x >= least ? w[i] : 0xFF800000u;
        }
        if (tied) mark(j);
        if (out != nullptr) store(w, E * j - row.phase);
      });
    }
  }

  // f(id, which) for the ids of key[which] in the vectors that word `i` marks, in
  // their order.  (In place the row still has them.)
  template <typename F>
  __device__ __forceinline__ void tied(int i, const uint32_t (&key)[2], F f) const {
#pragma unroll 1
    for (uint32_t m = s.marks[i]; m != 0; m &= m - 1) {
      const int j = j0 + 32 * i + __ffs(m) - 1;
      float x[E];
      row.load(j, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t k = key_of(x[e]);
        if (k == key[0]) f(E * j + e - row.phase, 0);
        if (k == key[1]) f(E * j + e - row.phase, 1);
      }
    }
  }
  // Of the ids with key[i], the ids[0]-th is the token, and those past the ids[1]-th
  // are not kept.
  __device__ __forceinline__ void settle(Elt* out, int32_t* token, const uint32_t (&key)[2], const uint32_t (&ids)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a thread has neighbouring words
    const int words = (j1 - j0 + 31) / 32, part = (words + kSampleThreads - 1) / kSampleThreads;
    const int w0 = min(words, static_cast<int>(threadIdx.x) * part), w1 = min(words, w0 + part);
    __syncthreads();
    uint32_t n[2] = {0, 0}, upto[2];
    for (int i = w0; i < w1; ++i) tied(i, key, [&](int, int which) { ++n[which]; });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      upto[i] = n[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto[i], d);
        if (lane >= d) upto[i] += o;
      }
      if (lane == 31) s.warp_count[warp][i] = upto[i];
    }
    __syncthreads();
    if (ctas > 1) {
      if (threadIdx.x < 2 * ctas) {
        uint32_t all = 0;
        for (int w = 0; w < kSampleWarps; ++w) all += s.warp_count[w][threadIdx.x & 1];
        of(threadIdx.x >> 1).same[rank][threadIdx.x & 1] = all;
      }
      cluster.sync();
    }
    bool past = false;  // whether this thread has ids that are not kept
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t all;
      upto[i] += sum_of_warps(&s.warp_count[0][i], 2, &all);
      if (ctas > 1)
        for (int o = 0; o < rank; ++o) upto[i] += s.same[o][i];
      upto[i] -= n[i];
      if (i == 0)
        past = past || (ids[0] > upto[0] && ids[0] <= upto[0] + n[0]);
      else
        past = past || (ids[1] != 0 && upto[1] + n[1] > ids[1]);
    }
    if (!past) return;
    for (int i = w0; i < w1; ++i)
      tied(i, key, [&](int id, int which) {
        const uint32_t at = ++upto[which];
        if (which == 0 && at == ids[0]) *token = id;
        if (which == 1 && at > ids[1]) out[id] = static_cast<Elt>(-INFINITY);
      });
  }

  // Whether a logit of the row is finite and -4096 or below (bf16).
  __device__ __forceinline__ bool any_far() {
    bool far = false;
    each_id<4>([&](float x, int) { far |= x <= -4096.f && x != -INFINITY; });
    far = __syncthreads_or(far) != 0;
    if (ctas > 1) {
      if (threadIdx.x < ctas) of(threadIdx.x).flag[rank] = far ? 1 : 0;
      cluster.sync();
      for (int o = 0; o < ctas; ++o) far |= s.flag[o] != 0;
    }
    return far;
  }

  // The row with one id left (or none: -1), and that id's logit.
  __device__ __forceinline__ void write_one(Elt* out, int id) const {
    const Elt none = static_cast<Elt>(-INFINITY);
    const Elt* in = row.p + row.phase;
    Elt kept = none;
    const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(Elt)), vecs = (phase + row.V + E - 1) / E;
    if (id >= 0) kept = in[id];
    if (row.p + row.phase == out && ctas > 1) cluster.sync();  // (in place: everyone has read it)
    if (row.p + row.phase == out && ctas == 1) __syncthreads();
    const int share = (vecs + ctas - 1) / ctas, a = min(vecs, rank * share), b = min(vecs, a + share);
    const uint32_t word = sizeof(Elt) == 2 ? 0xFF80FF80u : 0xFF800000u;
    for (int j = a + static_cast<int>(threadIdx.x); j < b; j += kSampleThreads) {
      const int first = E * j - phase;
      if (first >= 0 && first + E <= row.V && !(id >= first && id < first + E)) {
        *reinterpret_cast<uint4*>(out + first) = make_uint4(word, word, word, word);
      } else {
#pragma unroll 1
        for (int e = 0; e < E; ++e)
          if (first + e >= 0 && first + e < row.V) out[first + e] = first + e == id ? kept : none;
      }
    }
  }

  // The largest logit's key and its first id, over the cluster.  With kCounted the ids
  // are counted in their bins.
  template <bool kCounted>
  __device__ __forceinline__ void largest(uint32_t* key, int* id) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float best = -INFINITY;
    int at = 0x7FFFFFFF;
    each_id<sizeof(Elt) == 4 ? 8 : 4>([&](float x, int i) {
      if (x > best || (x == best && i < at && x != -INFINITY)) best = x, at = i;
      if constexpr (kCounted) {
        if (x != -INFINITY) atomicAdd(&s.bins.count[Bins::one(x)], 1u);
      }
    });
    uint32_t k = key_of(best);
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, k);
    uint32_t who = __reduce_min_sync(0xFFFFFFFFu, k == most ? static_cast<uint32_t>(at) : 0x7FFFFFFFu);
    if (lane == 0) s.warp_count[warp][0] = most, s.warp_count[warp][1] = who;
    __syncthreads();
    if (threadIdx.x < ctas) {
      k = 0, who = 0x7FFFFFFF;
      for (int w = 0; w < kSampleWarps; ++w) {
        const uint32_t o = s.warp_count[w][0], i = s.warp_count[w][1];
        if (o > k || (o == k && i < who)) k = o, who = i;
      }
      of(threadIdx.x).top[rank] = k;
      of(threadIdx.x).id[rank] = static_cast<int>(who);
    }
    meet();
    *key = 0, *id = 0x7FFFFFFF;
    for (int o = 0; o < ctas; ++o)
      if (s.top[o] > *key) *key = s.top[o], *id = s.id[o];  // (the first CTA has the lower ids)
  }
};

// What is kept and which logit (fp32: or token) is drawn; false: the bins do not say.  bf16: by any
// warp, fp32: by all.
template <typename Elt>
__device__ __forceinline__ bool SampleJob<Elt>::decide(const SampleAsk& ask, int32_t* token, SamplePlace* kept, SamplePlace* drawn) {
  SampleBin f;
  unsigned long long weights = s.group_sum[kGroups];
  bool cut = false;  // by top-k
  if constexpr (sizeof(Elt) == 4) {
    cut = of_k.bin >= 0;
    if (cut) {
      look_up(of_k.bin, &f);  // (its sums; the counts are gone)
      f.c0 = of_k.c0, f.c = of_k.c;
    }
  } else {
    cut = ask.k < row.V && find(kByCount, ask.k, &f);
  }
  if (cut) {
    if (!resolve(f, kByCount, ask.k, kept)) return false;
    weights = kept->sum + kept->ids * weight(of_key(kept->key));
  }
  if (ask.p < 1.f) {
    unsigned long long target = static_cast<unsigned long long>(ceil(static_cast<double>(ask.p) * static_cast<double>(weights)));
    target = target < 1 ? 1 : (target > weights ? weights : target);
    SamplePlace at;
    find(kBySumTo, target, &f);
    if (!resolve(f, kBySumTo, target, &at)) return false;
    // (a beginning of what top-k left)
    if (at.key > kept->key || (at.key == kept->key && at.ids < kept->ids)) {
      *kept = at;
      weights = kept->sum + kept->ids * weight(of_key(kept->key));
    }
  }
  if (ask.least > 0 && s.least_key > kept->key) {
    const uint32_t key = s.least_key;
    look_up(Bins::one(of_key(key)), &f);
    if (!resolve(f, kByKey, key, kept)) return false;
    kept->key = key;
    kept->ids = kept->all;
    weights = sizeof(Elt) == 2 ? kept->sum + f.w : kept->sum;
  }
  if (token != nullptr) {
    unsigned long long target = static_cast<unsigned long long>(static_cast<double>(ask.u) * static_cast<double>(weights));
    if (target >= weights) target = weights - 1;
    find(kBySumPast, target, &f);
    if (!resolve(f, kBySumPast, target, drawn, token)) return false;
  }
  return true;
}

__device__ __forceinline__ WeightScale scale_of(double c) {
  const float hi = static_cast<float>(c);
  return {hi, static_cast<float>(c - static_cast<double>(hi))};
}
// Of higher temperatures (from 1.8e30 on) the scale's rest ends below the normal floats,
// and logits that are as far apart as matters have differences above the largest float:
// their rows are sample_any's, which takes logits in 2^64.  (bf16 rows within 4096 have
// weights of 1 at such a temperature, whatever is left of the scale.)
constexpr float kLeastScale = 0x1p-100f;

// One cluster a row.
template <typename Elt>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const SampleArgs a, int ctas) {
  extern __shared__ __align__(16) unsigned char sample_smem[];
  using Bins = SampleBinsOf<Elt>;
  SampleSmem<Elt>& smem = *reinterpret_cast<SampleSmem<Elt>*>(sample_smem);
  SampleFast<Elt>& s = smem.fast;
  const int tid = threadIdx.x;
  const int rank = ctas > 1 ? static_cast<int>(blockIdx.x % ctas) : 0;
  const int row_of = static_cast<int>(blockIdx.x / ctas);  // (65536 requests of 65 rows)
  const int b = row_of / (a.n_max + 1), place = row_of - b * (a.n_max + 1);
  const long long r = row_of;
  uint32_t bad = 0;
  // (all loads of the request's numbers at once)
  int n = a.draft_len != nullptr ? a.draft_len[b] : a.n_max;
  const float T = a.temperature != nullptr ? a.temperature[b] : 1.f;
  float m = a.min_p != nullptr ? a.min_p[b] : 0.f;
  SampleAsk ask;
  ask.p = a.top_p != nullptr ? a.top_p[b] : 1.f;
  ask.u = a.uniform != nullptr ? a.uniform[r] : 0.f;
  ask.k = a.top_k != nullptr ? a.top_k[b] : 0;
  if (n < 0 || n > a.n_max) {
    bad |= SPECDEC_DEV_ERR_DRAFT_LEN;
    n = max(0, min(n, a.n_max));
  }
  const bool first = rank == 0 && tid == 0;
  if (place > n) {
    if (first && a.tokens != nullptr) a.tokens[r] = -1;
    if (first && bad != 0 && a.err != nullptr) atomicOr(a.err, bad);
    return;
  }
  const Elt* logits = static_cast<const Elt*>(a.logits) + r * a.V;
  Elt* out = a.out != nullptr ? static_cast<Elt*>(a.out) + r * a.V : nullptr;
  int32_t* token = a.tokens != nullptr ? a.tokens + r : nullptr;
  if (ask.k <= 0 || ask.k > a.V) ask.k = a.V;
  const bool cold = !(T >= 1e-6f) || T > 3e38f;  // the largest logit alone
  if (cold && T != 0.f) bad |= SPECDEC_DEV_ERR_TEMPERATURE;
  if (!(ask.p >= 0.f) || !(m <= 1.f) || !(m >= 0.f)) {
    bad |= SPECDEC_DEV_ERR_SAMPLE;
    if (!(ask.p >= 0.f)) ask.p = 1.f;
    m = !(m >= 0.f) ? 0.f : fminf(m, 1.f);
  }
  if (!(ask.u >= 0.f && ask.u < 1.f)) {
    bad |= SPECDEC_DEV_ERR_SAMPLE;
    ask.u = ask.u >= 1.f ? 1.f - 0x1p-24f : 0.f;
  }
  SampleRow<Elt> row(logits, a.V);
  const int share = (row.vecs + ctas - 1) / ctas;
  SampleJob<Elt> job = {s, sample_smem + sizeof(SampleSmem<Elt>), row, cooperative_groups::this_cluster(), ctas, rank, min(row.vecs, rank * share),
                        min(row.vecs, rank * share + share), 0.f, {}};
  job.say_begun();
  if (cold || ask.k == 1) {
    uint32_t key;
    int id;
    job.wait_begun();
    job.template largest<false>(&key, &id);
    if (key <= kKeyFloor) bad |= SPECDEC_DEV_ERR_SAMPLE, id = -1;
    if (first && token != nullptr) *token = id;
    if (first && bad != 0 && a.err != nullptr) atomicOr(a.err, bad);
    if (out != nullptr) job.write_one(out, id);
    if (ctas > 1) job.cluster.sync();
    return;
  }

  // the histogram, and the largest logit
  job.clear_bins();
  if (tid < 256) s.table[tid] = kExp2Table[tid];
  if (tid == 0) s.listed = s.gathered = 0, s.zeroed = false, s.zero[0] = s.zero[1] = 0;
  __syncthreads();
  if (tid == kSampleThreads - 1) {
    // (64-bit arithmetic by one thread, beside the others' work: it has 1/64 of the rate)
    s.scale = scale_of(1.4426950408889634074 / static_cast<double>(T));
    s.least = m > 0.f ? static_cast<unsigned long long>(ceil(static_cast<double>(m) * static_cast<double>(kWeightOne))) : 0;
  }
  bool simple = true;
  if constexpr (sizeof(Elt) == 2) {
    uint32_t least = 0xFFFFFFFFu;
    // Both counts' addresses are made at once, in 16 bits each beside the window's own:
    // the bins are at the start of the CTA's memory, whose place in a cluster is above.
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(s.bins.count)), counts = (base & 0xFFFFu) * 0x10001u;
    const bool placed = (base & 0xFFFFu) <= 0x8000u;
    auto add = [&](uint32_t d) {
      const uint32_t at = d * 4 + counts;
      asm volatile("red.shared::cta.add.u32 [%0], 1;" ::"r"(__byte_perm(at, base, 0x7610)) : "memory");
      asm volatile("red.shared::cta.add.u32 [%0], 1;" ::"r"(__byte_perm(at, base, 0x7632)) : "memory");
    };
    if (placed) job.template each<4>([&](const uint4& q, int j) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint32_t first = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = Bins::two(w[i]);
        first = min_u16x2(first, d);
        add(d);
      }
      least = min_u16x2(least, first);
      job.largest_of[j - job.j0] = static_cast<uint8_t>(Bins::coarse(min(first & 0xFFFFu, first >> 16)));
    });
    least = __reduce_min_sync(0xFFFFFFFFu, min(least & 0xFFFFu, least >> 16));
    if ((tid & 31) == 0) s.warp_count[tid >> 5][0] = least;
    job.wait_begun();
    __syncthreads();
    ask.scale = job.scale = s.scale;
    ask.least = s.least;
    // (-infinity and what is -4096 or below it does not count)
    if (tid == kSampleThreads - 1) s.bins.count[Bins::kBins - 1] = 0;
    if (tid < ctas) {
      for (int w = 0; w < kSampleWarps; ++w) least = min(least, s.warp_count[w][0]);
      job.of(tid).top[rank] = least;
    }
    job.meet();
    least = Bins::kBins;
    for (int o = 0; o < ctas; ++o) least = min(least, s.top[o]);
    // rows whose order or weights the bins do not tell
    const int top = static_cast<int>(least);
    simple = placed && top > 0 && top < Bins::kBins - 1 && top != Bins::kHalf - 1 && top != Bins::kHalf;
    job.top = Bins::value(top);
  } else {
    uint32_t key;
    int id;
    job.wait_begun();
    if (ask.k < a.V)
      job.template largest<true>(&key, &id);
    else
      job.template largest<false>(&key, &id);
    ask.scale = job.scale = s.scale;
    ask.least = s.least;
    simple = key > kKeyFloor && key < key_of(INFINITY) && job.scale.hi >= kLeastScale;
    job.top = of_key(key);
    if (simple) {
      job.find_least(ask);
      __syncthreads();
      job.add_weights(ask);
    }
  }

  SamplePlace kept = {kKeyFloor + 1, kAnyIds, 0, 0}, drawn = {0, 0, 0, 0};
  if (simple) {
    if constexpr (sizeof(Elt) == 2) {
      job.find_least(ask);
      job.add_up(true, true);
      // logits of -4096 and below are not counted: they have no weight and are not kept, or the row is another's
      const uint32_t ids = s.group_count[kSampleGroups];
      if ((ask.k < a.V && static_cast<uint32_t>(ask.k) > ids) || !((job.top + 4096.f) * ask.scale.hi > 49.f)) simple = !job.any_far();
      // every warp could, but one is enough, while another looks at the bins of zero
      for (int again = 0; simple; ++again) {
        if (tid < 32) {
          const bool sure = job.decide(ask, token, &kept, &drawn);
          if (tid == 0) s.kept = kept, s.drawn = drawn, s.simple = sure;
        } else if (tid < 64) {
          uint32_t c[2];
          unsigned long long w[2];
          const bool more = again == 0 && job.zeros_matter(c, w);
          if (tid == 32) s.more = more;
        }
        __syncthreads();
        if (!s.more) break;
        job.add_zeros();
        if (tid < 32) kept = {kKeyFloor + 1, kAnyIds, 0, 0};
      }
      if (simple) kept = s.kept, drawn = s.drawn, simple = s.simple;
    } else {
      simple = job.decide(ask, token, &kept, &drawn);
    }
  }
  if (!simple) {
    // by the first CTA alone, whose memory nobody reads any more
    ask.unit = 1.f;
    if (ask.scale.hi < kLeastScale) {
      ask.unit = 0x1p-64f;
      ask.scale = scale_of(0x1p64 * 1.4426950408889634074 / static_cast<double>(a.temperature[b]));
    }
    job.meet();
    if (rank == 0) {
      if (!sample_any(smem.any, row, ask, out, token)) bad |= SPECDEC_DEV_ERR_SAMPLE;
      if (first && bad != 0 && a.err != nullptr) atomicOr(a.err, bad);
    }
    return;
  }
  if (first && bad != 0 && a.err != nullptr) atomicOr(a.err, bad);
  const bool part = out != nullptr && kept.ids < kept.all;
  // (the token, where it is not known yet, and ids of the last logit that is kept)
  const uint32_t keys[2] = {token != nullptr ? drawn.key : 0, part ? kept.key : 0};
  const uint32_t ids[2] = {token != nullptr ? drawn.ids : 0, part ? kept.ids : 0};
  const bool some = keys[0] != 0 || part;
  if (some) job.clear_marks();
  if (some || out != nullptr) job.write(out, kept.key, keys);
  if (some) job.settle(out, token, keys, ids);
  if (ctas > 1) job.cluster.sync();  // (memory that others may still read)
}

}  // namespace specdec
