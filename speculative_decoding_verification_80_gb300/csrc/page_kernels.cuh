// page_kernels.cuh — the blocks of a paged cache beyond a step's growth: requests
// that go on from others' tokens (kv_fork), blocks moved to the lowest ids
// (kv_compact), and the copies that both ask for (kv_copy).
//
// kv_fork and kv_compact are one launch each, whose three steps are a barrier of all
// its CTAs apart: of a cluster for little work, of a cooperative grid of up to a CTA an
// SM for more.  A few KB to some MB: bound by latency (10 to 17 us on the device for 7
// to 4700 moves: the launch, two barriers and the loads between them) and, a call, by
// the host, which three launches cost 7 us and one 4.
#pragma once
#include <cooperative_groups.h>
#include <stdint.h>

#include "block_prefix.cuh"
#include "page_work.cuh"

namespace specdec {

// ------------------------------------------------------------------ kv_fork
struct ForkArgs {
  int32_t P, B, bs_log2, max_blocks, num_blocks;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* accepted_len;
  const int32_t* held;
  const int32_t* parent;
  const int32_t* keep;
  const int32_t* shares;
  int32_t* ring;
  const int32_t* ring_state;
  int32_t* table_out;
  int32_t* kv_len_out;
  int32_t* held_out;
  int32_t* shares_out;
  int32_t* ring_state_out;
  int32_t* copies;
  int32_t* count;
  uint32_t* err;
  PageWork work;
};

// All CTAs of the launch, which are one cluster or a cooperative grid.
constexpr int kPageCluster = 8;
template <bool kCluster>
__device__ __forceinline__ void page_sync() {
  if constexpr (kCluster)
    cooperative_groups::this_cluster().sync();
  else
    cooperative_groups::this_grid().sync();
}

constexpr int kPageThreads = kBlockThreads;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kPageSegment = 256;  // entries of a row that a warp takes

__device__ __forceinline__ int clamped_held(const ForkArgs& a, int p, uint32_t* bad) {
  const int h = a.held[p];
  if (h < 0 || h > a.max_blocks) *bad = 1;
  return max(0, min(h, a.max_blocks));
}

// The tokens that new request b goes on from, of `parent` (-1: none).
__device__ __forceinline__ int fork_tokens(const ForkArgs& a, int b, int* parent, uint32_t* bad) {
  int p = a.parent[b];
  if (p < -1 || p >= a.P) *bad = 1;
  if (p < 0 || p >= a.P) {
    *parent = -1;
    return 0;
  }
  *parent = p;
  const long long room = static_cast<long long>(clamped_held(a, p, bad)) << a.bs_log2;
  long long n = static_cast<long long>(a.kv_len[p]) + (a.accepted_len != nullptr ? max(a.accepted_len[p], -1) + 1LL : 0LL);
  if (n < 0 || n > room) {
    *bad = 1;
    n = max(0LL, min(n, room));
  }
  if (a.keep != nullptr) n = max(0LL, min(n, static_cast<long long>(a.keep[b])));
  return static_cast<int>(n);
}

// How often each block is named, and who would write it: a warp a part of a row.
__device__ __forceinline__ void fork_count(const ForkArgs& a) {
  const int lane = threadIdx.x & 31, warps = static_cast<int>(gridDim.x) * kPageWarps;
  const int parts = (a.max_blocks + kPageSegment - 1) / kPageSegment;
  uint32_t bad = 0;
  for (long long i = static_cast<long long>(blockIdx.x) * kPageWarps + (threadIdx.x >> 5); i < static_cast<long long>(a.P + a.B) * parts; i += warps) {
    // (the rows' first parts first: most rows have no others)
    const int r = static_cast<int>(i % (a.P + a.B)), j0 = static_cast<int>(i / (a.P + a.B)) * kPageSegment;
    const bool fresh = r >= a.P;
    int p = r, n = 0, part = -1;
    if (fresh) {
      const int tokens = fork_tokens(a, r - a.P, &p, &bad);
      n = static_cast<int>((static_cast<long long>(tokens) + (1 << a.bs_log2) - 1) >> a.bs_log2);
      if ((tokens & ((1 << a.bs_log2) - 1)) != 0) part = n - 1;
    } else {
      n = clamped_held(a, r, &bad);
    }
    const int32_t* row = a.table + static_cast<long long>(max(p, 0)) * a.max_blocks;
    uint32_t* to = fresh ? a.work.news : a.work.olds;
#pragma unroll 4
    for (int j = j0 + lane; j < min(n, j0 + kPageSegment); j += 32) {
      const int x = row[j];
      if (x < 0 || x >= a.num_blocks) {
        bad = 1;
        continue;
      }
      atomicAdd(to + x, 1u);
      if (j == part) {
        atomicAdd(a.work.writers + x, 1u);
        atomicMax(a.work.last + x, static_cast<uint32_t>(r - a.P + 1));
      }
    }
  }
  if (bad != 0 && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_BLOCKS);
}

// Holders of a block after the step, before anyone takes a copy.
__device__ __forceinline__ long long holders_of(const ForkArgs& a, int x) {
  return static_cast<long long>(a.shares[x]) + 1 - a.work.olds[x] + a.work.news[x];
}

// Which blocks go back: the last CTAs.  Who copies, into which block: the first.
__device__ __forceinline__ void fork_plan(const ForkArgs& a) {
  const int tid = threadIdx.x, lane = tid & 31, N = a.num_blocks;
  const int ctas = static_cast<int>(gridDim.x), others = ctas > 1 ? ctas - 1 : 1;
  if (blockIdx.x > 0 || ctas == 1) {
    const int words = (N + 31) / 32;
    for (int w = (ctas > 1 ? static_cast<int>(blockIdx.x) - 1 : 0) * kPageWarps + (tid >> 5); w < words; w += others * kPageWarps) {
      const long long x = 32LL * w + lane;
      const bool back = x < N && a.work.olds[x] != 0 && holders_of(a, static_cast<int>(x)) <= 0;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, back);
      if (lane == 0) a.work.gone[w] = m;
    }
  }
  if (blockIdx.x > 0) return;
  __shared__ uint32_t part[33][1];
  int head = a.ring_state[0], count = a.ring_state[1];
  uint32_t bad = 0, asked = 0;
  if (head < 0 || head >= N || count < 0 || count > N) {
    bad = 1;
    head = head < 0 || head >= N ? 0 : head;
    count = max(0, min(count, N));
  }
  if (tid == 0) a.work.ring[0] = head, a.work.ring[1] = count;
  for (int b0 = 0; b0 < a.B; b0 += kBlockThreads) {
    const int b = b0 + tid;
    int p = -1, tokens = 0, x = -1;
    if (b < a.B) tokens = fork_tokens(a, b, &p, &bad);
    const int full = tokens >> a.bs_log2;
    const bool partial = (tokens & ((1 << a.bs_log2) - 1)) != 0;
    bool ask = false;
    if (partial) {
      x = a.table[static_cast<long long>(p) * a.max_blocks + full];
      // all but the last of those that write a block, where no one else holds it
      ask = x >= 0 && x < N && !(a.work.writers[x] == holders_of(a, x) && a.work.last[x] == static_cast<uint32_t>(b + 1));
    }
    const uint32_t v[1] = {ask ? 1u : 0u};
    uint32_t before[1], sum[1];
    block_prefix(v, part, before, sum);
    const int number = static_cast<int>(asked + before[0]);
    asked += sum[0];
    const bool got = ask && number < count;
    if (ask && !got) bad = 1;
    if (b < a.B) {
      a.work.number[b] = got ? number : -1;
      a.held_out[b] = full + (partial && (!ask || got) ? 1 : 0);
      a.kv_len_out[b] = ask && !got ? full << a.bs_log2 : tokens;
      if (got) {
        const int to = a.ring[(static_cast<long long>(head) + number) % N];
        if (to < 0 || to >= N) bad = 1;
        a.copies[2 * number] = x;
        a.copies[2 * number + 1] = to;
      }
    }
  }
  if (tid == 0) *a.count = static_cast<int>(min(asked, static_cast<uint32_t>(count)));
  if (bad != 0 && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_BLOCKS);
}

// Bits before word `upto` of `words`, over the CTA.
__device__ __forceinline__ uint32_t bits_before(const uint32_t* words, int upto) {
  __shared__ uint32_t sums[kPageWarps];
  uint32_t n = 0;
  for (int i = threadIdx.x; i < upto; i += kPageThreads) n += __popc(words[i]);
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int i = 0; i < kPageWarps; ++i) n += sums[i];
  return n;
}

// This CTA's share of a bitmap's words.
__device__ __forceinline__ void share_of_words(int words, int* w0, int* w1) {
  const int share = (words + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  *w0 = min(words, static_cast<int>(blockIdx.x) * share);
  *w1 = min(words, *w0 + share);
}

// The new rows, the blocks' holders, the ring's new end, and the counts cleared.
__device__ __forceinline__ void fork_finish(const ForkArgs& a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_blocks;
  const long long all = static_cast<long long>(gridDim.x) * kPageThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kPageThreads + tid; i < static_cast<long long>(a.B) * a.max_blocks; i += all) {
    const int b = static_cast<int>(i / a.max_blocks), j = static_cast<int>(i - static_cast<long long>(b) * a.max_blocks), n = a.held_out[b];
    int x = -1;
    if (j < n) {
      const int number = j == n - 1 ? a.work.number[b] : -1;
      x = number >= 0 ? a.copies[2 * number + 1] : a.table[static_cast<long long>(a.parent[b]) * a.max_blocks + j];
    }
    a.table_out[i] = x;
  }
  const int words = (N + 31) / 32;
  int w0, w1;
  share_of_words(words, &w0, &w1);
  const int head = a.work.ring[0], count = a.work.ring[1];
  uint32_t before = bits_before(a.work.gone, w0);
  if (blockIdx.x == gridDim.x - 1) {
    const uint32_t gone = bits_before(a.work.gone, words);
    if (tid == 0) {
      const int taken = *a.count;
      a.ring_state_out[0] = static_cast<int>((static_cast<long long>(head) + taken) % N);
      a.ring_state_out[1] = static_cast<int>(min(static_cast<long long>(N), static_cast<long long>(count) - taken + gone));
    }
  }
  // warps take words in turn; a warp's own bits before are counted as it goes
  for (int w = w0 + warp, from = w0; w < w1; w += kPageWarps) {
    for (; from + 32 <= w; from += 32) before += __reduce_add_sync(0xFFFFFFFFu, __popc(a.work.gone[from + lane]));
    const uint32_t near = __reduce_add_sync(0xFFFFFFFFu, from + lane < w ? __popc(a.work.gone[from + lane]) : 0);
    const uint32_t m = a.work.gone[w];
    const long long x = 32LL * w + lane;
    if (x >= N) continue;
    const uint32_t olds = a.work.olds[x];
    int now = a.shares[x];
    if (olds != 0) {
      const long long h = holders_of(a, static_cast<int>(x));
      const uint32_t writers = a.work.writers[x];
      const long long after = h == writers ? min(h, 1LL) : h - writers;
      now = static_cast<int>(max(0LL, min(after - 1, 0x7FFFFFFFLL)));
      a.work.olds[x] = a.work.news[x] = a.work.writers[x] = a.work.last[x] = 0;
    }
    a.shares_out[x] = now;
    if ((m >> lane) & 1)
      a.ring[(static_cast<long long>(head) + count + before + near + __popc(m & ((1u << lane) - 1))) % N] = static_cast<int>(x);
  }
}

template <bool kCluster>
__global__ void __launch_bounds__(kPageThreads) fork_kernel(const ForkArgs a) {
  fork_count(a);
  page_sync<kCluster>();
  fork_plan(a);
  page_sync<kCluster>();
  fork_finish(a);
}

// --------------------------------------------------------------- kv_compact
struct CompactArgs {
  int32_t B, max_blocks, num_blocks;
  const int32_t* table;
  const int32_t* held;
  const int32_t* shares;
  const int32_t* ring;
  const int32_t* ring_state;
  int32_t* table_out;
  int32_t* shares_out;
  int32_t* ring_out;
  int32_t* ring_state_out;
  int32_t* renamed;
  int32_t* copies;
  int32_t* count;
  uint32_t* err;
  PageWork work;
};

// A bit for each free block.
__device__ __forceinline__ void compact_mark(const CompactArgs& a) {
  const int N = a.num_blocks, all = static_cast<int>(gridDim.x) * kPageThreads;
  int head = a.ring_state[0], count = a.ring_state[1];
  uint32_t bad = 0;
  if (head < 0 || head >= N || count < 0 || count > N) {
    bad = 1;
    head = head < 0 || head >= N ? 0 : head;
    count = max(0, min(count, N));
  }
  for (int i = static_cast<int>(blockIdx.x) * kPageThreads + threadIdx.x; i < count; i += all) {
    const int x = a.ring[(static_cast<long long>(head) + i) % N];
    if (x < 0 || x >= N)
      bad = 1;
    else
      atomicOr(a.work.marks + (x >> 5), 1u << (x & 31));
  }
  if (bad != 0 && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_BLOCKS);
}

// With n blocks in use: the i-th in use from n on moves to the i-th free one
// before it.
__device__ __forceinline__ void compact_plan(const CompactArgs& a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_blocks;
  const int words = (N + 31) / 32;
  int w0, w1;
  share_of_words(words, &w0, &w1);
  const uint32_t* marks = a.work.marks;
  const uint32_t free_all = bits_before(marks, words);
  const int n = N - static_cast<int>(free_all);
  uint32_t holes = bits_before(marks, n >> 5);  // free before n
  if ((n & 31) != 0) holes += __popc(marks[n >> 5] & ((1u << (n & 31)) - 1));
  uint32_t before = bits_before(marks, w0);
  if (blockIdx.x == 0 && tid == 0) {
    *a.count = static_cast<int>(holes);
    a.ring_state_out[0] = 0;
    a.ring_state_out[1] = static_cast<int>(free_all);
  }
  for (int w = w0 + warp, from = w0; w < w1; w += kPageWarps) {
    for (; from + 32 <= w; from += 32) before += __reduce_add_sync(0xFFFFFFFFu, __popc(marks[from + lane]));
    const uint32_t near = __reduce_add_sync(0xFFFFFFFFu, from + lane < w ? __popc(marks[from + lane]) : 0);
    const uint32_t m = marks[w];
    const int x = 32 * w + lane;
    if (x >= N) continue;
    const int free_before = static_cast<int>(before + near + __popc(m & ((1u << lane) - 1)));
    const bool free = (m >> lane) & 1;
    int rank = free ? -1 : -2;  // -1: free, -2: stays
    if (x < n && free) {
      a.copies[2 * free_before + 1] = x;
    } else if (x >= n && !free) {
      rank = (x - n) - (free_before - static_cast<int>(holes));
      a.copies[2 * rank] = x;
    } else if (x < n) {
      a.shares_out[x] = a.shares[x];
    } else {
      a.shares_out[x] = 0;
    }
    a.work.rank[x] = rank;
    if (x >= n) a.ring_out[x - n] = x;
  }
}

// The blocks' new names, in the tables too, and the marks cleared.
__device__ __forceinline__ void compact_finish(const CompactArgs& a) {
  const int N = a.num_blocks;
  const long long me = static_cast<long long>(blockIdx.x) * kPageThreads + threadIdx.x, all = static_cast<long long>(gridDim.x) * kPageThreads;
  for (long long i = me; i < N; i += all) {
    const int x = static_cast<int>(i), rank = a.work.rank[x];
    int to = rank == -2 ? x : -1;
    if (rank >= 0) {
      to = a.copies[2 * rank + 1];
      a.shares_out[to] = a.shares[x];
      a.shares_out[x] = 0;
    }
    a.renamed[x] = to;
    if ((x & 31) == 0) a.work.marks[x >> 5] = 0;
  }
  uint32_t bad = 0;
  for (long long i = me; i < static_cast<long long>(a.B) * a.max_blocks; i += all) {
    const int b = static_cast<int>(i / a.max_blocks), j = static_cast<int>(i - static_cast<long long>(b) * a.max_blocks);
    int n = a.held[b], y = -1;
    if (n < 0 || n > a.max_blocks) bad = 1;
    n = max(0, min(n, a.max_blocks));
    if (j < n) {
      const int x = a.table[i], rank = x >= 0 && x < N ? a.work.rank[x] : -1;
      y = rank == -2 ? x : (rank >= 0 ? a.copies[2 * rank + 1] : -1);
      if (y < 0) bad = 1;
    }
    a.table_out[i] = y;
  }
  if (bad != 0 && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_BLOCKS);
}

template <bool kCluster>
__global__ void __launch_bounds__(kPageThreads) compact_kernel(const CompactArgs a) {
  compact_mark(a);
  page_sync<kCluster>();
  compact_plan(a);
  page_sync<kCluster>();
  compact_finish(a);
}

// ------------------------------------------------------------------ kv_copy
constexpr int kCopyThreads = 256;
constexpr int kCopyLayers = 64;  // of a launch
struct CopyLayer {
  void* k;
  void* v;
  float* ks;
  float* vs;
};
struct CopyArgs {
  CopyLayer layer[kCopyLayers];
  int32_t layers, capacity, num_blocks, H;
  int64_t bytes;    // of a block of k or v, a multiple of 1024
  int32_t chunk;    // a warp's part of it
  int32_t chunks;
  const int32_t* pairs;
  const int32_t* count;
};

// A warp takes a part of a block of one layer's keys or values: 8 KB, of which eight
// loads of 16 bytes a lane are on their way at once; its first part takes the scales
// along.  Bytes bound it: 4692 blocks of two layers (616 MB read and written) take 95
// us, 6.5 TB/s; 379 blocks of four layers (198 MB) 29 us and 7 of sixteen 6.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int kLoads = 8;
  const int lane = threadIdx.x & 31;
  const int count = max(0, min(*a.count, a.capacity));
  const long long items = static_cast<long long>(count) * a.layers * 2 * a.chunks;
  const long long warps = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  for (long long i = static_cast<long long>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5); i < items; i += warps) {
    const long long block = i / a.chunks;
    const int c = static_cast<int>(i - block * a.chunks);
    const int l2 = static_cast<int>(block % (2 * a.layers));
    const int pair = static_cast<int>(block / (2 * a.layers));
    const int from = a.pairs[2 * pair], to = a.pairs[2 * pair + 1];
    if (from < 0 || from >= a.num_blocks || to < 0 || to >= a.num_blocks || from == to) continue;
    const CopyLayer& layer = a.layer[l2 >> 1];
    char* base = static_cast<char*>((l2 & 1) ? layer.v : layer.k) + static_cast<long long>(c) * a.chunk;
    const uint4* x = reinterpret_cast<const uint4*>(base + from * a.bytes);
    uint4* y = reinterpret_cast<uint4*>(base + to * a.bytes);
    const int n = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.bytes - static_cast<int64_t>(c) * a.chunk)) / 16;
    for (int k = lane; k < n; k += 32 * kLoads) {
      uint4 q[kLoads];
#pragma unroll
      for (int e = 0; e < kLoads; ++e)
        if (k + 32 * e < n) q[e] = x[k + 32 * e];
#pragma unroll
      for (int e = 0; e < kLoads; ++e)
        if (k + 32 * e < n) y[k + 32 * e] = q[e];
    }
    if (c == 0) {
      float* s = (l2 & 1) ? layer.vs : layer.ks;
      for (int h = lane; h < a.H; h += 32) s[static_cast<long long>(to) * a.H + h] = s[static_cast<long long>(from) * a.H + h];
    }
  }
}

}  // namespace specdec
