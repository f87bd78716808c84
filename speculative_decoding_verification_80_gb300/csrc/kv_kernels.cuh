// kv_kernels.cuh — the paged cache's bookkeeping (kv_block_step) and the
// writer of its 8-bit blocks (kv_append).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace specdec {

// ------------------------------------------------------------ kv_block_step
//
// Prefix sums over the requests (blocks asked for, then tokens, blocks taken
// and given of those that are granted), then the slots of the tokens and the
// table's new entries.  A few KB to some MB: bound by latency, so one launch
// and few dependent loads.  Each CTA makes the whole plan for itself, in shared
// memory, and writes its share of the tokens: a thread four neighbouring ones,
// whose request it finds by bisection.  Measured on the device: 12 us for 1024
// requests of 5600 tokens in all, 9 us for 512 prompts of 640 000 (5 MB), 36 us
// with 8 CTAs in a cluster, which would let the outputs be the inputs' arrays.
struct BlockArgs {
  int32_t B, bs, max_blocks, num_blocks, capacity;
  const int32_t* kv_len;
  const int32_t* accepted_len;
  const int32_t* new_tokens;
  const int32_t* held;
  int32_t* table;
  int32_t* ring;
  const int32_t* ring_state;
  int32_t* kv_len_out;
  int32_t* held_out;
  int32_t* ring_state_out;
  int32_t* cu_tokens;
  int32_t* cu_blocks;
  int32_t* slot_map;
  int32_t* positions;
  uint32_t* err;
  int32_t slots_vec, positions_vec;  // they lie on 16 bytes
};

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

// The index b in [0, n) with cu[b] <= t < cu[b + 1]; cu is non-decreasing,
// cu[0] <= t < cu[n].
__device__ __forceinline__ int owner_of(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// What a step decides, as the writing needs it: the outputs' arrays, or copies
// in shared memory.
struct BlockPlan {
  int32_t* cu_tokens;  // [B + 1]
  int32_t* cu_blocks;  // [B + 1]
  int32_t* kept;       // [B]
  int32_t* held;       // [B] blocks after the step
};

// (before < 2 N)
__device__ __forceinline__ int ring_at(const BlockArgs& a, int head, long long i) {
  long long at = head + i;
  if (at >= a.num_blocks) at -= a.num_blocks;
  if (at >= a.num_blocks) at -= a.num_blocks;
  return static_cast<int>(at);
}

// Slots and positions of tokens t .. t + 3; reads the ring and the entries that
// were there before.
__device__ __forceinline__ void fill_tokens(const BlockArgs& a, const BlockPlan& plan, int bs_log2, int head, int t, int total) {
  int slot[4], pos[4], b = -1, end = 0, kept = 0, first = 0, taken_at = 0, before = 0, j_last = -1, block = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    slot[k] = pos[k] = -1;
    if (t + k >= total) continue;
    if (t + k >= end) {
      b = owner_of(plan.cu_tokens, a.B, t + k);
      first = plan.cu_tokens[b];
      end = plan.cu_tokens[b + 1];
      kept = plan.kept[b];
      taken_at = plan.cu_blocks[b];
      before = plan.held[b];
      const int taken = plan.cu_blocks[b + 1] - taken_at;
      before = taken > 0 ? before - taken : 0x7FFFFFFF;
      j_last = -1;
    }
    const int p = kept + (t + k - first), j = p >> bs_log2;
    if (j != j_last) {
      block = j >= before ? a.ring[ring_at(a, head, static_cast<long long>(taken_at) + (j - before))]
                          : a.table[static_cast<long long>(b) * a.max_blocks + j];
      j_last = j;
    }
    slot[k] = (block << bs_log2) + (p & ((1 << bs_log2) - 1));
    pos[k] = p;
  }
  auto store = [&](int32_t* to, const int (&x)[4], bool vec) {
    if (vec && t + 4 <= a.capacity) {
      *reinterpret_cast<int4*>(to + t) = make_int4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t + k < a.capacity) to[t + k] = x[k];
    }
  };
  store(a.slot_map, slot, a.slots_vec);
  store(a.positions, pos, a.positions_vec);
}
// The i-th block taken goes into its table.
__device__ __forceinline__ void fill_block(const BlockArgs& a, const BlockPlan& plan, int head, int i) {
  const int b = owner_of(plan.cu_blocks, a.B, i);
  const int at = plan.held[b] - plan.cu_blocks[b + 1] + i;
  a.table[static_cast<long long>(b) * a.max_blocks + at] = a.ring[ring_at(a, head, i)];
}

// The step's lengths, grants and prefix sums, by one CTA of `ctas` that do the
// same; and the blocks that go back, of its share of the requests.
__device__ __forceinline__ int block_plan(const BlockArgs& a, const BlockPlan& plan, int rank, int ctas, int* ring_out, uint32_t* bad_out) {
  __shared__ uint32_t part1[33][1], part3[33][3];
  const int tid = threadIdx.x, lane = tid & 31;
  const int N = a.num_blocks;
  int head = a.ring_state[0], count = a.ring_state[1];
  uint32_t bad = 0;
  if (head < 0 || head >= N || count < 0 || count > N) {
    bad = 1;
    head = head < 0 || head >= N ? 0 : head;
    count = max(0, min(count, N));
  }
  uint32_t asked = 0, tokens = 0, took = 0, gave = 0;
  for (int b0 = 0; b0 < a.B; b0 += kBlockThreads) {
    const int b = b0 + tid;
    const bool in = b < a.B;
    int kept = 0, want = 0, held = 0, need = 0;
    if (in) {
      const int fresh = a.new_tokens[b], len = a.kv_len[b], accepted = a.accepted_len != nullptr ? a.accepted_len[b] : -1;
      held = a.held[b];
      if (held < 0 || held > a.max_blocks) {
        bad = 1;
        held = max(0, min(held, a.max_blocks));
      }
      want = max(fresh, 0);
      if (fresh >= 0) {
        long long k = len + (max(accepted, -1) + 1LL);
        if (k < 0 || k > static_cast<long long>(held) * a.bs) {
          bad = 1;
          k = max(0LL, min(k, static_cast<long long>(held) * a.bs));
        }
        kept = static_cast<int>(k);
      }
      need = static_cast<int>(min(0x7FFFFFFFLL, (static_cast<long long>(kept) + want + a.bs - 1) / a.bs));
    }
    const bool fits = need <= a.max_blocks;
    const int grow = fits ? max(need - held, 0) : 0;
    const uint32_t x1[1] = {static_cast<uint32_t>(grow)};
    uint32_t before1[1], sum1[1];
    block_prefix(x1, part1, before1, sum1);
    const bool granted = in && fits && (grow == 0 || capped_sum(capped_sum(asked, before1[0]), grow) <= static_cast<uint32_t>(count));
    asked = capped_sum(asked, sum1[0]);
    if (in && !granted) bad = 1;
    const int taken = granted ? grow : 0;
    const int given = granted ? max(held - need, 0) : 0;
    // (grants are a prefix of the requests that ask for blocks)
    const uint32_t x[3] = {static_cast<uint32_t>(granted ? want : 0), static_cast<uint32_t>(taken), static_cast<uint32_t>(given)};
    uint32_t before[3], sum[3];
    block_prefix(x, part3, before, sum);
    const uint32_t tok_at = capped_sum(tokens, before[0]), take_at = capped_sum(took, before[1]), give_at = capped_sum(gave, before[2]);
    tokens = capped_sum(tokens, sum[0]);
    took = capped_sum(took, sum[1]);
    gave = capped_sum(gave, sum[2]);
    if (in) {
      if (granted && tok_at + want > static_cast<uint32_t>(a.capacity)) bad = 1;
      plan.kept[b] = kept;
      plan.held[b] = held + taken - given;
      plan.cu_tokens[b] = static_cast<int>(min(tok_at, static_cast<uint32_t>(a.capacity)));
      plan.cu_blocks[b] = static_cast<int>(take_at);
    }
    // blocks that go back, a warp to a request
    uint32_t m = (b0 + tid) / 32 % ctas == rank ? __ballot_sync(0xFFFFFFFFu, given > 0) : 0;
    while (m) {
      const int src = __ffs(m) - 1;
      m &= m - 1;
      const int n = __shfl_sync(0xFFFFFFFFu, given, src);
      const int from = __shfl_sync(0xFFFFFFFFu, held - given, src);
      const uint32_t to = __shfl_sync(0xFFFFFFFFu, give_at, src);
      const long long row = static_cast<long long>(b - lane + src) * a.max_blocks;
      for (int i = lane; i < n; i += 32)
        a.ring[static_cast<int>((static_cast<long long>(head) + count + to + i) % N)] = a.table[row + from + i];
    }
  }
  if (tid == 0) {
    plan.cu_tokens[a.B] = static_cast<int>(min(tokens, static_cast<uint32_t>(a.capacity)));
    plan.cu_blocks[a.B] = static_cast<int>(took);
  }
  ring_out[0] = ring_at(a, head, took);
  ring_out[1] = static_cast<int>(min(static_cast<uint32_t>(N), capped_sum(count - took, gave)));
  *bad_out = bad;
  return head;
}

// All in one launch, where no output is an input's array (another CTA may
// still read it) and the plan fits shared memory.  Blocks that go back lie
// behind the ring's free ones and in other rows than those that are taken.
constexpr int kBlockShared = 8192;  // requests
__global__ void __launch_bounds__(kBlockThreads) block_step_kernel(const BlockArgs a) {
  extern __shared__ __align__(16) int32_t plan_words[];
  const BlockPlan plan = {plan_words, plan_words + (a.B + 1), plan_words + 2 * (a.B + 1), plan_words + 3 * (a.B + 1)};
  const int rank = blockIdx.x, bs_log2 = __ffs(a.bs) - 1;
  int ring[2];
  uint32_t bad;
  const int head = block_plan(a, plan, rank, gridDim.x, ring, &bad);
  __syncthreads();
  const int me = rank * kBlockThreads + threadIdx.x, all = static_cast<int>(gridDim.x) * kBlockThreads;
  for (int b = me; b <= a.B; b += all) {
    a.cu_tokens[b] = plan.cu_tokens[b];
    a.cu_blocks[b] = plan.cu_blocks[b];
    if (b < a.B) {
      a.kv_len_out[b] = plan.kept[b];
      a.held_out[b] = plan.held[b];
    }
  }
  if (me == 0) {
    a.ring_state_out[0] = ring[0];
    a.ring_state_out[1] = ring[1];
  }
  if (rank == 0 && bad && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_BLOCKS);
  const int total = plan.cu_tokens[a.B], blocks = plan.cu_blocks[a.B];
  for (long long t = 4LL * me; t < a.capacity; t += 4LL * all) fill_tokens(a, plan, bs_log2, head, static_cast<int>(t), total);
  for (int i = me; i < blocks; i += all) fill_block(a, plan, head, i);
}

// Otherwise: the plan by one CTA, in the outputs' arrays, then the rest by many.
__global__ void __launch_bounds__(kBlockThreads) block_plan_kernel(const BlockArgs a) {
  const BlockPlan plan = {a.cu_tokens, a.cu_blocks, a.kv_len_out, a.held_out};
  int ring[2];
  uint32_t bad;
  block_plan(a, plan, 0, 1, ring, &bad);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.ring_state_out[0] = ring[0];
    a.ring_state_out[1] = ring[1];
  }
  if (bad && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_BLOCKS);
}
__global__ void __launch_bounds__(256) block_fill_kernel(const BlockArgs a) {
  const BlockPlan plan = {a.cu_tokens, a.cu_blocks, a.kv_len_out, a.held_out};
  const int total = a.cu_tokens[a.B], blocks = a.cu_blocks[a.B], N = a.num_blocks, bs_log2 = __ffs(a.bs) - 1;
  const int head = static_cast<int>((static_cast<long long>(a.ring_state_out[0]) + N - blocks) % N);
  const int me = static_cast<int>(blockIdx.x) * blockDim.x + threadIdx.x, all = static_cast<int>(gridDim.x) * blockDim.x;
  for (int i = me; i < blocks; i += all) fill_block(a, plan, head, i);
  if (4LL * me < a.capacity) fill_tokens(a, plan, bs_log2, head, 4 * me, total);
}

// ---------------------------------------------------------------- kv_append
struct AppendArgs {
  const void* x[2];  // k, v
  long long token_stride[2], head_stride[2];  // bytes
  uint8_t* cache[2];
  float* scale[2];
  const int32_t* slot_map;
  int32_t T, H, bs, num_blocks;
  int32_t window;   // tokens whose runs' starts one CTA takes
  int32_t team;     // threads of a run's head, 32 to 256
  int32_t pairs;    // heads of k and v that one CTA takes
};

constexpr int kAppendThreads = 256;
constexpr int kMaxBlockSize = 128;

// The least power of two s with amax <= 448 s, for a finite amax > 0; 0 of 0.
// amax = f 2^e with f in [1, 2): 448 = 1.75 * 2^8, so s = 2^(e - 8), twice
// that for f > 1.75.  Subnormal amax counts as the least normal number.
__device__ __forceinline__ float pow2_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  const int e = max(static_cast<int>(u >> 23), 1) + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0) - 8;
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}
// The least power of two at or above a block's scale (its own, where this
// writer set it); 0 for what is no scale.
__device__ __forceinline__ float pow2_ceil(float s) {
  if (!(s > 0.f) || isinf(s)) return 0.f;
  const uint32_t u = __float_as_uint(s);
  const uint32_t e = (u >> 23) + ((u & 0x7FFFFFu) != 0 ? 1 : 0);
  return __uint_as_float(min(max(e, 1u), 253u) << 23);
}
// 1 / s of a power of two s (0 of 0): exact.
__device__ __forceinline__ float pow2_inverse(float s) {
  return s > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(s)) : 0.f;
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
  return __half22float2(__half2(h));
}

template <typename Elt>
__device__ __forceinline__ void unpack16(const uint4& q, float* f);
template <>
__device__ __forceinline__ void unpack16<float>(const uint4& q, float* f) {
  f[0] = __uint_as_float(q.x), f[1] = __uint_as_float(q.y), f[2] = __uint_as_float(q.z), f[3] = __uint_as_float(q.w);
}
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4& q, float* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The largest magnitude of 16 bytes and `top`, in bits: for bf16 one in each
// half.  No number is above infinity.
template <typename Elt>
__device__ __forceinline__ uint32_t max_bits(uint32_t top, const uint4& q) {
  if (sizeof(Elt) == 4)
    return max(max(top, q.x & 0x7FFFFFFFu), max(q.y & 0x7FFFFFFFu, max(q.z & 0x7FFFFFFFu, q.w & 0x7FFFFFFFu)));
  return __vmaxu2(__vmaxu2(top, q.x & 0x7FFF7FFFu), __vmaxu2(q.y & 0x7FFF7FFFu, __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu)));
}
// The largest finite one, as a float's bits.
template <typename Elt>
__device__ __forceinline__ uint32_t finite_max_bits(uint32_t top, const uint4& q) {
  float f[16 / sizeof(Elt)];
  unpack16<Elt>(q, f);
  for (float x : f) top = max(top, fabsf(x) < INFINITY ? __float_as_uint(fabsf(x)) : 0);
  return top;
}

// A team of warps takes a run's rows of one head of k or v: as many threads as
// hold a whole block's rows in registers, kVecs loads of 16 bytes each, so that
// the rows are read once and all at a time.  A CTA has the runs that start in
// its window of tokens; its teams go through their pairs of a run and a head,
// and runs that a warp holds are a warp's.  Bound by the rows read and the codes
// written, as long as few instructions are spent on a value: on 50 000 bf16
// tokens of 8 heads of 128 in blocks of 64 (308 MB) 54 us, 5.7 TB/s, with 8
// loads a thread and four CTAs an SM; 60 with three; 83 with 16 loads and two,
// which is left for blocks of 64 KB.  Asking for the next pair's rows before
// this one's codes are made costs a CTA, and 14 us.
template <typename Elt, int D, int kVecs>
__global__ void __launch_bounds__(kAppendThreads, kVecs <= 8 ? 4 : 2) append_kernel(const AppendArgs a) {
  constexpr int E = 16 / sizeof(Elt);  // values of a 16-byte load
  constexpr int VR = D / E;            // loads of a row
  static_assert(32 % VR == 0, "a warp's threads hold whole rows");
  constexpr int kSpan = 2 * kMaxBlockSize;
  __shared__ int32_t slots[kSpan + 1];
  __shared__ uint32_t breaks[kSpan / 32 + 1];  // tokens that do not go on in the run before them
  __shared__ int32_t starts[kMaxBlockSize], runs;
  __shared__ uint32_t red[kAppendThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const long long t0 = static_cast<long long>(blockIdx.x) * a.window;
  const int span = static_cast<int>(min(static_cast<long long>(a.window) + a.bs, a.T - t0));  // tokens looked at
  const int most = a.num_blocks * a.bs, bs_log2 = __ffs(a.bs) - 1;
  for (int i = tid; i <= span; i += kAppendThreads) {
    const long long t = t0 + i - 1;
    const int s = t >= 0 ? __ldg(a.slot_map + t) : -1;
    slots[i] = s >= most ? -1 : s;
  }
  if (tid == 0) runs = 0;
  __syncthreads();
  {
    const int i = tid;  // (the span is at most the CTA's threads)
    const int s = i < span ? slots[i + 1] : -1, before = i < span ? slots[i] : -1;
    const bool starts_here = s >= 0 && !(before >= 0 && before + 1 == s && (s & (a.bs - 1)) != 0);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, s < 0 || starts_here);
    if (lane == 0) breaks[tid >> 5] = m;
    if (starts_here && i < a.window) starts[atomicAdd(&runs, 1)] = i;
  }
  static_assert(kSpan <= kAppendThreads, "a thread for each token looked at");
  __syncthreads();
  const int pair0 = blockIdx.y * a.pairs, pairs = min(a.pairs, 2 * a.H - pair0);
  // Runs that a warp holds are a warp's, longer ones a team's.
#pragma unroll 1
  for (int width = a.team;; width = 32) {
    const int team = tid / width, k0 = tid - team * width;
    auto team_barrier = [&]() {
      if (width == 32)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(width) : "memory");
    };
#pragma unroll 1
    for (int item = team; item < runs * pairs; item += kAppendThreads / width) {
      const int run = item / pairs, pair = pair0 + item - run * pairs;
      const int which = pair >= a.H ? 1 : 0, h = pair - which * a.H, i = starts[run], s = slots[i + 1];
      const int block = s >> bs_log2, off = s & (a.bs - 1);
      // the run goes on to the next break
      int n = min(span - i, a.bs - off);
      {
        const int w = (i + 1) >> 5;
        uint32_t m = breaks[w] & (0xFFFFFFFFu << ((i + 1) & 31));
        int at = w;
        while (m == 0 && ++at < kSpan / 32) m = breaks[at];
        if (m != 0) n = min(n, at * 32 + __ffs(m) - 1 - i);
      }
      if ((width == 32) != (n * VR <= 32 * kVecs)) continue;
      const long long stride = which ? a.token_stride[1] : a.token_stride[0];
      const char* row = static_cast<const char*>(which ? a.x[1] : a.x[0]) + h * (which ? a.head_stride[1] : a.head_stride[0]) + (t0 + i) * stride;
      float* sp = (which ? a.scale[1] : a.scale[0]) + static_cast<long long>(block) * a.H + h;
      uint8_t* tile = (which ? a.cache[1] : a.cache[0]) + (static_cast<long long>(block) * a.H + h) * a.bs * D;
      const float old = off > 0 ? *sp : 0.f;
      // (a team's threads hold whole rows: a thread's loads are as far from
      // their rows' starts)
      const char* from = row + (k0 / VR) * stride + (k0 % VR) * 16;
      const long long step = width / VR * stride;
      uint4 x[kVecs];
#pragma unroll
      for (int v = 0; v < kVecs; ++v, from += step)
        x[v] = k0 + v * width < n * VR ? __ldg(reinterpret_cast<const uint4*>(from)) : make_uint4(0, 0, 0, 0);
      uint32_t top = 0;
      auto team_max = [&]() {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (width > 32) {
          if (lane == 0) red[tid >> 5] = top;
          team_barrier();
          top = __reduce_max_sync(0xFFFFFFFFu, lane < width / 32 ? red[team * (width / 32) + lane] : 0);
        }
      };
#pragma unroll
      for (int v = 0; v < kVecs; ++v) top = max_bits<Elt>(top, x[v]);
      if (sizeof(Elt) == 2) top = max(top << 16, top & 0xFFFF0000u);
      team_max();
      if (top >= 0x7F800000u) {  // infinities and NaN do not count
        team_barrier();
        top = 0;
#pragma unroll 1
        for (int k = k0; k < n * VR; k += width)
          top = finite_max_bits<Elt>(top, __ldg(reinterpret_cast<const uint4*>(row + (k / VR) * stride) + k % VR));
        team_max();
      }
      const float amax = __uint_as_float(top);
      const float now = fmaxf(pow2_scale(amax), pow2_ceil(old));
      // (scale 0: the finite values are zeros, and an infinity stays one for its code)
      const float inv = now > 0.f ? pow2_inverse(now) : 1.f;
      if (off > 0 && now > old) {  // the older tokens move to the new scale
        const float ratio = old * inv;
        for (int k = k0; k < off * (D / 16); k += width) {
          uint4* c = reinterpret_cast<uint4*>(tile) + k;
          uint4 q = *c;
          uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 lo = e4m3_values(w[e] & 0xFFFFu), hi = e4m3_values(w[e] >> 16);
            w[e] = e4m3_pair(lo.x * ratio, lo.y * ratio) | e4m3_pair(hi.x * ratio, hi.y * ratio) << 16;
          }
          *c = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      uint8_t* to = tile + off * D + k0 * E;
#pragma unroll
      for (int v = 0; v < kVecs; ++v, to += width * E) {
        if (k0 + v * width >= n * VR) break;
        float f[E];
        unpack16<Elt>(x[v], f);
        uint32_t w[E / 4];
#pragma unroll
        for (int e = 0; e < E / 4; ++e)
          w[e] = e4m3_pair(f[4 * e] * inv, f[4 * e + 1] * inv) | (e4m3_pair(f[4 * e + 2] * inv, f[4 * e + 3] * inv) << 16);
        if (E == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[E / 4 - 1]);
        else
          *reinterpret_cast<uint32_t*>(to) = w[0];
      }
      team_barrier();  // everyone has read the old scale, and `red`
      if (k0 == 0) *sp = now;
    }
    if (width == 32) break;
  }
}

}  // namespace specdec
