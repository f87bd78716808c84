// logits_kernel.cuh — penalties, biases and grammar masks on the rows that the
// verify step reads (spec_process_logits).
//
// Few entries of a row change by a penalty or a bias: those of tokens that the
// request's history, drafts or biases name.  An item is a request and `share`
// neighbouring entries of the vocabulary; a CTA (one an SM) works on its items
// in four roles, which run ahead of one another:
//
//   - a warp copies the items' part of each row, and of its mask, into a ring
//     in shared memory;
//   - two teams of four warps take turns in counting the coming items' entries
//     in the history (a 32-bit word an entry), and list those they meet: every
//     item reads the whole history of its request, from L2 after the first;
//   - two teams of eight warps take turns in the rows: they change the listed
//     entries, a thread each, and set masked ones to -infinity;
//   - a warp copies the rows out.
//
// In place, a row without a mask is not copied: its entries are changed where
// they lie, which pays while few are (64 requests with histories of up to 2048
// ids: 30 us without masks; 256 with up to 8192, so that one entry in 18 has a
// sector read and written for it: 450 us, where copies take 200).  Bound by the
// rows' bytes, read and written once.  (With an item's steps one after the other,
// the copies' and the history's latencies took twice the time, however many CTAs
// an SM had.)  Measured: 64 requests of up to 5
// rows of 128256 bf16 (132 MB) 35 us, 3.8 TB/s; 256 of up to 8 rows of 152064
// (980 MB) 200 us, 4.9 TB/s, of which the copies alone are 166 us.  Rows of 8
// KB in a ring of 12 take 53 and 309 us, and equal parts of all rows in their
// order, one for each CTA, 39 and 257 us: CTAs that work side by side on one
// request's rows keep what they read close together.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"
#include "waits.cuh"

namespace specdec {

constexpr int kLogitTeam = 256;          // threads of a team of the rows
constexpr int kCountTeam = 128;          // and of one that counts
constexpr int kLogitThreads = 2 * kLogitTeam + 2 * kCountTeam + 64;
constexpr int kLogitRowBytes = 16384;    // of a row of an item, at most
constexpr int kLogitLeastBytes = 1024;
constexpr int kLogitRing = 6;            // rows in shared memory
constexpr int kBiasList = 256;           // biases of an item kept in shared memory
constexpr uint32_t kInPrompt = 1u << 31;
constexpr uint32_t kHasBias = 1u << 30;
constexpr uint32_t kIsDraft = 1u << 29;  // (a history is shorter than that)
constexpr uint32_t kCountMask = kIsDraft - 1;
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
  int32_t share;       // vocabulary entries of an item, a multiple of 128 (a mask of them is whole 16 bytes)
  int32_t chunks;      // items of a request
  int32_t same_phase;  // logits and out are alike modulo 16 bytes
};

struct LogitParams {  // one request's penalties
  float rep, pres, freq;
};

// l after penalties; the token was made c times.
__device__ __forceinline__ float penalised(float l, uint32_t c, bool in_prompt, float bias, const LogitParams& p) {
  if (c != 0 || in_prompt) l = l > 0.f ? l / p.rep : l * p.rep;
  l -= p.freq * static_cast<float>(c);
  if (c != 0) l -= p.pres;
  return l + bias;
}

__device__ __forceinline__ float elt_to_float(float x) { return x; }
__device__ __forceinline__ float elt_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void float_to_elt(float x, float& y) { y = x; }
__device__ __forceinline__ void float_to_elt(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// Sets the entries of 16 bytes whose bit is 0 to -infinity.
template <typename Elt>
__device__ __forceinline__ void mask_vector(uint4& y, uint32_t allow) {
  uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(Elt) == 4) {
      if (!(allow >> i & 1)) w[i] = 0xFF800000u;
    } else {
      const uint32_t keep = (allow >> 2 * i & 1) * 0xFFFFu | (allow >> (2 * i + 1) & 1) * 0xFFFF0000u;
      w[i] = (w[i] & keep) | (0xFF80FF80u & ~keep);
    }
  }
  y = make_uint4(w[0], w[1], w[2], w[3]);
}

// What is known of a request, brought into range.
struct LogitRequest {
  int32_t drafts, history, prompt, lo, hi;
  LogitParams p;
  bool bad;
  __device__ __forceinline__ LogitRequest(const LogitArgs& a, int b) {
    drafts = a.draft_len != nullptr ? __ldg(a.draft_len + b) : a.n_max;
    p.rep = a.repetition != nullptr ? __ldg(a.repetition + b) : 1.f;
    p.pres = a.presence != nullptr ? __ldg(a.presence + b) : 0.f;
    p.freq = a.frequency != nullptr ? __ldg(a.frequency + b) : 0.f;
    history = a.history_stride > 0 ? __ldg(a.history_len + b) : 0;
    prompt = a.history_stride > 0 ? __ldg(a.prompt_len + b) : 0;
    lo = a.bias_offsets != nullptr ? __ldg(a.bias_offsets + b) : 0;
    hi = a.bias_offsets != nullptr ? __ldg(a.bias_offsets + b + 1) : 0;
    bad = drafts < 0 || drafts > a.n_max;
    drafts = max(0, min(drafts, a.n_max));
    if (!(p.rep > 0.f) || isinf(p.rep)) bad = true, p.rep = 1.f;
    if (!isfinite(p.pres)) bad = true, p.pres = 0.f;
    if (!isfinite(p.freq)) bad = true, p.freq = 0.f;
    if (history < 0 || history > a.history_stride || prompt < 0 || prompt > history) bad = true;
    history = max(0, min(history, a.history_stride));
    prompt = max(0, min(prompt, history));
    if (lo < 0 || hi < lo || hi > a.num_bias) {
      bad = true;
      lo = max(0, min(lo, a.num_bias));
      hi = max(lo, min(hi, a.num_bias));
    }
  }
};

// An item as the second role leaves it to the third and fourth.
struct LogitItem {
  LogitParams p;
  int32_t rows, lo, hi;
  int32_t listed;                       // entries of the list
  int32_t biases;                       // of the item's entries
  int32_t draft[SPECDEC_MAX_DRAFT];
  int32_t mask[SPECDEC_MAX_DRAFT + 1];  // of the rows, -1 for none
  int32_t bias_at[kBiasList];           // entry, from the item's first on
  float bias[kBiasList];                // value
  float bias_sum[kBiasList];            // of the entry from here on
  bool bias_first[kBiasList];           // none of the entry's is before it
};
struct LogitShared {
  uint64_t row_full[kLogitRing], row_done[kLogitRing], row_empty[kLogitRing], item_full[2], item_empty[2];
  LogitItem item[2];
};

// Dynamic shared memory: words of two items, the rows, the lists of two items.
template <typename Elt>
struct LogitLayout {
  // a row may start anywhere in its first 16 bytes
  static __host__ __device__ int row_bytes(int share) { return share * static_cast<int>(sizeof(Elt)) + 16; }
  // a row's mask may start at any word of 16 bytes
  static __host__ __device__ int slot_bytes(int share) { return row_bytes(share) + share / 8 + 32; }
  static __host__ __device__ int bytes(int share) { return 2 * share * 6 + kLogitRing * slot_bytes(share); }
};

template <typename Elt>
__global__ void __launch_bounds__(kLogitThreads, 1) process_logits_kernel(const LogitArgs a) {
  extern __shared__ __align__(16) uint32_t words_of[];
  __shared__ LogitShared sh;
  constexpr int kElt = sizeof(Elt), N = 16 / kElt;
  const int row_bytes = LogitLayout<Elt>::row_bytes(a.share), slot_bytes = LogitLayout<Elt>::slot_bytes(a.share);
  unsigned char* ring = reinterpret_cast<unsigned char*>(words_of + 2 * a.share);
  uint16_t* list_of = reinterpret_cast<uint16_t*>(ring + kLogitRing * slot_bytes);
  const int rows_max = a.n_max + 1, items = a.B * a.chunks, grid = gridDim.x;
  const bool in_place = a.out == a.logits;
  const uintptr_t in_first = reinterpret_cast<uintptr_t>(a.logits);
  const uintptr_t in_end = in_first + static_cast<unsigned long long>(a.B) * rows_max * a.V * kElt;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kLogitRing; ++i) {
      ptx::mbar_init(ptx::smem_addr(&sh.row_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.row_done[i]), kLogitTeam / 32);
      ptx::mbar_init(ptx::smem_addr(&sh.row_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&sh.item_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.item_empty[i]), 2 * kLogitTeam / 32 + 1);
      sh.item[i].listed = 0;
    }
    ptx::fence_mbarrier_init();
  }
  for (int i = threadIdx.x; i < a.share / 2; i += kLogitThreads) reinterpret_cast<uint4*>(words_of)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();

  // Where a wait for an item runs out, its role ends there: what the item's place
  // holds then is not looked at.  The other roles' waits run out in turn.
  Waiter wait;
  // A CTA's i-th item.  (Which of a request's items it is changes from one to
  // the next: low ids, and so work, are often the first's.)
  auto item_of = [&](int i) { return i * grid + static_cast<int>((blockIdx.x + 7u * i) % grid); };
  auto row_at = [&](int b, int j, int v0) { return (static_cast<long long>(b) * rows_max + j) * a.V + v0; };
  // Bytes [from, to) are copied as whole 16 bytes, as far as they are of the
  // tensor [first, end): what is not the item's among them is not used, and
  // what is left out of the item's (`head` and `tail` bytes) the third role
  // reads.
  struct Span {
    uintptr_t lo, hi;
    int head, tail;
    __device__ __forceinline__ Span(uintptr_t from, uintptr_t to, uintptr_t first, uintptr_t end)
        : lo(from & ~static_cast<uintptr_t>(15)), hi((to + 15) & ~static_cast<uintptr_t>(15)), head(0), tail(0) {
      if (lo < first) {
        lo += 16;
        head = static_cast<int>(min(lo, to) - from);
      }
      if (hi > end) {
        hi -= 16;
        tail = static_cast<int>(to - max(hi, from + head));
      }
    }
    __device__ __forceinline__ uint32_t bytes() const { return hi > lo ? static_cast<uint32_t>(hi - lo) : 0; }
  };
  auto row_span = [&](int b, int j, int v0, int n) {
    const uintptr_t from = in_first + row_at(b, j, v0) * kElt;
    return Span(from, from + n * kElt, in_first, in_end);
  };
  const uintptr_t mask_first = reinterpret_cast<uintptr_t>(a.mask);
  auto mask_at = [&](int m, int v0) { return mask_first + (static_cast<long long>(m) * a.mask_words + (v0 >> 5)) * 4; };
  auto mask_span = [&](int m, int v0, int n) {
    const uintptr_t from = mask_at(m, v0);
    return Span(from, from + (n + 31) / 32 * 4, mask_first, mask_first + static_cast<long long>(a.mask_count) * a.mask_words * 4);
  };
  int rows_copied = 0;  // counted by each role but the second

  auto gave_up = [&]() { return __any_sync(0xFFFFFFFFu, wait.dead()); };  // any thread of the warp
  auto warp_arrive = [&](const uint64_t& bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_addr(&bar));
  };

  if (threadIdx.x >= 2 * kLogitTeam + 2 * kCountTeam + 32) {
    // ---------------------------------------------------------- rows out of the ring
    const int lane = threadIdx.x & 31;
    for (int i = 0; item_of(i) < items; ++i) {
      const int item = item_of(i), b = item / a.chunks, v0 = (item - b * a.chunks) * a.share, n = min(a.share, a.V - v0);
      const LogitItem& it = sh.item[i & 1];
      wait(sh.item_full[i & 1], i >> 1 & 1);
      if (gave_up()) break;
#pragma unroll 1
      for (int j = 0; j < it.rows; ++j) {
        if (in_place && it.mask[j] < 0) continue;
        const int slot = rows_copied % kLogitRing;
        wait(sh.row_done[slot], rows_copied / kLogitRing & 1);
        if (gave_up()) break;
        ++rows_copied;
        // whole 16 bytes by a copy, the ends by threads
        const long long at = row_at(b, j, v0);
        const Elt* row = reinterpret_cast<const Elt*>(ring + slot * slot_bytes + static_cast<int>((in_first + at * kElt) & 15));
        Elt* dst = static_cast<Elt*>(a.out) + at;
        const int first = a.same_phase ? min(n, static_cast<int>(-reinterpret_cast<uintptr_t>(dst) & 15) / kElt) : n, count = (n - first) / N * N;
        if (lane == 0 && count > 0)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + first), "r"(ptx::smem_addr(row + first)),
                       "r"(count * kElt)
                       : "memory");
        for (int e = lane; e < first; e += 32) dst[e] = row[e];
        if (lane < n - first - count) dst[first + count + lane] = row[first + count + lane];
        if (lane == 0) {
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        // the row before this one has left
        if (rows_copied > 1) warp_arrive(sh.row_empty[(rows_copied - 2) % kLogitRing]);
      }
      warp_arrive(sh.item_empty[i & 1]);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  } else if (threadIdx.x >= 2 * kLogitTeam + 2 * kCountTeam) {
    // ---------------------------------------------------------- rows into the ring
    const int lane = threadIdx.x & 31;
    int next_drafts = 0, next_mask[3];
    auto look_ahead = [&](int item) {
      if (item >= items) return;
      const int b = item / a.chunks;
      next_drafts = a.draft_len != nullptr ? __ldg(a.draft_len + b) : a.n_max;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int j = lane + 32 * k;
        next_mask[k] = a.mask_rows != nullptr && j < rows_max ? __ldg(a.mask_rows + static_cast<long long>(b) * rows_max + j) : -1;
      }
    };
    look_ahead(item_of(0));
    bool stop = false;
    for (int i = 0; item_of(i) < items && !stop; ++i) {
      const int item = item_of(i), b = item / a.chunks, v0 = (item - b * a.chunks) * a.share, n = min(a.share, a.V - v0);
      const int rows = max(0, min(next_drafts, a.n_max)) + 1;
      const int masks[3] = {next_mask[0], next_mask[1], next_mask[2]};
      look_ahead(item_of(i + 1));
#pragma unroll 1
      for (int j = 0; j < rows; ++j) {
        const int m = __shfl_sync(0xFFFFFFFFu, j < 32 ? masks[0] : j < 64 ? masks[1] : masks[2], j & 31);
        const bool masked = m >= 0 && m < a.mask_count;
        if (in_place && !masked) continue;
        const int slot = rows_copied % kLogitRing;
        if (rows_copied >= kLogitRing) wait(sh.row_empty[slot], (rows_copied / kLogitRing - 1) & 1);
        if (gave_up()) {
          stop = true;
          break;
        }
        ++rows_copied;
        if (lane == 0) {
          const Span row = row_span(b, j, v0, n);
          const uint32_t bar = ptx::smem_addr(&sh.row_full[slot]), dst = ptx::smem_addr(ring + slot * slot_bytes);
          uint32_t bytes = row.bytes();
          if (masked) bytes += mask_span(m, v0, n).bytes();
          ptx::mbar_arrive_expect_tx(bar, bytes);
          if (row.bytes() != 0) ptx::bulk_g2s_nohint(dst + (row.head != 0 ? 16 : 0), reinterpret_cast<const void*>(row.lo), row.bytes(), bar);
          if (masked) {
            const Span mask = mask_span(m, v0, n);
            if (mask.bytes() != 0)
              ptx::bulk_g2s_nohint(dst + row_bytes + (mask.head != 0 ? 16 : 0), reinterpret_cast<const void*>(mask.lo), mask.bytes(), bar);
          }
        }
        __syncwarp();
      }
    }
    // no copy is in flight when the CTA ends
    Waiter drain;
    for (int k = max(0, rows_copied - kLogitRing); k < rows_copied; ++k) drain(sh.row_full[k % kLogitRing], k / kLogitRing & 1);
    if (drain.dead()) wait.looks = 0;
  } else if (threadIdx.x >= 2 * kLogitTeam) {
    // ---------------------------------------------------------- named entries
    const int tid = threadIdx.x % kCountTeam, team = 1 + (threadIdx.x - 2 * kLogitTeam) / kCountTeam;  // 1 or 2
    for (int i = team - 1; item_of(i) < items; i += 2) {
      const int item = item_of(i), b = item / a.chunks, v0 = (item - b * a.chunks) * a.share, n = min(a.share, a.V - v0);
      LogitItem& it = sh.item[i & 1];
      uint32_t* words = words_of + (i & 1) * a.share;
      uint16_t* list = list_of + (i & 1) * a.share;
      const LogitRequest rq(a, b);
      // what does not need the item's place is on its way while that is waited for
      const int m = a.mask_rows != nullptr && tid < rows_max ? __ldg(a.mask_rows + static_cast<long long>(b) * rows_max + tid) : -1;
      const int draft = tid < rq.drafts ? __ldg(a.draft_tokens + static_cast<long long>(b) * a.n_max + tid) : -1;
      // ids by fours where they lie on 16 bytes
      const int32_t* h = a.history + static_cast<long long>(b) * a.history_stride;
      const int head = min(rq.history, static_cast<int>(-(reinterpret_cast<uintptr_t>(h) >> 2) & 3)), fours = (rq.history - head) / 4;
      const int4* h4 = reinterpret_cast<const int4*>(h + head);
      const int tail = head + 4 * fours + tid;
      const int id_head = tid < head ? __ldg(h + tid) : -1, id_tail = tail < rq.history ? __ldg(h + tail) : -1;
      constexpr int kFours = 4;  // in flight a thread
      int4 id[kFours];
      auto load_ids = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kFours; ++k) id[k] = i0 + k * kCountTeam < fours ? __ldg(h4 + i0 + k * kCountTeam) : make_int4(-1, -1, -1, -1);
      };
      load_ids(tid);
      int bias_id = -1;
      float bias_value = 0.f;
      auto load_bias = [&](int k) {
        bias_id = k < rq.hi ? __ldg(a.bias_ids + k) : -1;
        bias_value = k < rq.hi ? __ldg(a.bias_values + k) : 0.f;
      };
      if (tid < 32) load_bias(rq.lo + tid);
      if (i >= 2) wait(sh.item_empty[i & 1], ((i >> 1) - 1) & 1);
      const int was = it.listed;
      for (int k = tid; k < was; k += kCountTeam) words[list[k]] = 0;
      if (named_any(team, kCountTeam, wait.dead())) break;
      if (tid == 0) {
        it.p = rq.p;
        it.rows = rq.drafts + 1;
        it.lo = rq.lo;
        it.hi = rq.hi;
        it.listed = it.biases = 0;
      }
      const bool no_mask = tid <= rq.drafts && (m < -1 || m >= a.mask_count);
      if (((rq.bad && tid == 0) || no_mask) && a.err != nullptr && v0 == 0) atomicOr(a.err, SPECDEC_DEV_ERR_PENALTY);
      if (tid <= rq.drafts) it.mask[tid] = no_mask ? -1 : m;
      if (tid < rq.drafts) it.draft[tid] = draft;
      named_barrier(team, kCountTeam);
      auto add = [&](int v, uint32_t flag) {  // counted, or flagged
        const uint32_t off = static_cast<uint32_t>(v) - static_cast<uint32_t>(v0);
        if (off >= static_cast<uint32_t>(n)) return;
        const uint32_t old = flag == 1 ? atomicAdd(words + off, 1u) : atomicOr(words + off, flag);
        if (old == 0) list[atomicAdd(&it.listed, 1)] = static_cast<uint16_t>(off);
      };
      add(id_head, tid < rq.prompt ? kInPrompt : 1u);
      add(id_tail, tail < rq.prompt ? kInPrompt : 1u);
#pragma unroll 1
      for (int i0 = tid; i0 < fours; i0 += kFours * kCountTeam) {
        if (i0 != tid) load_ids(i0);
#pragma unroll
        for (int k = 0; k < kFours; ++k) {
          const int at = head + 4 * (i0 + k * kCountTeam);
          const int v[4] = {id[k].x, id[k].y, id[k].z, id[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) add(v[e], at + e < rq.prompt ? kInPrompt : 1u);
        }
      }
      add(draft, kIsDraft);
      if (tid < 32) {  // the biases, in their order
        int count = 0;
        for (int k0 = rq.lo; k0 < rq.hi; k0 += 32) {
          if (k0 != rq.lo) load_bias(k0 + tid);
          const int v = bias_id;
          const bool mine = v >= v0 && v < v0 + n;
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
          if (mine) {
            const int k = count + __popc(m & ((1u << tid) - 1));
            if (k < kBiasList) {
              it.bias_at[k] = v - v0;
              it.bias[k] = bias_value;
            }
            add(v, kHasBias);
          }
          count += __popc(m);
        }
        if (tid == 0) it.biases = count;
      }
      named_barrier(team, kCountTeam);
      const int biases = it.biases;
      if (biases > 0 && biases <= kBiasList) {
        for (int q = tid; q < biases; q += kCountTeam) {
          float sum = 0.f;
          bool is_first = true;
          for (int k = q; k < biases; ++k)
            if (it.bias_at[k] == it.bias_at[q]) sum += it.bias[k];
          for (int k = 0; k < q; ++k) is_first = is_first && it.bias_at[k] != it.bias_at[q];
          it.bias_sum[q] = sum;
          it.bias_first[q] = is_first;
        }
        named_barrier(team, kCountTeam);
      }
#ifdef SPECDEC_TEST_WAIT_RUNS_OUT
      // Failure-path test builds only: the first CTA keeps its second item to
      // itself, so every other role's wait of that CTA runs out in turn.
      if (blockIdx.x == 0 && i == 1) continue;
#endif
      if (tid == 0) ptx::mbar_arrive(ptx::smem_addr(&sh.item_full[i & 1]));
    }
  } else {
    // ---------------------------------------------------------- the rows
    const int tid = threadIdx.x % kLogitTeam, team = threadIdx.x / kLogitTeam;
    constexpr uint32_t kAll = (1u << N) - 1;
    for (int i = 0; item_of(i) < items; ++i) {
      const int item = item_of(i), b = item / a.chunks, v0 = (item - b * a.chunks) * a.share, n = min(a.share, a.V - v0);
      const LogitItem& it = sh.item[i & 1];
      const uint32_t* words = words_of + (i & 1) * a.share;
      const uint16_t* list = list_of + (i & 1) * a.share;
      wait(sh.item_full[i & 1], i >> 1 & 1);
      if (named_any(3 + team, kLogitTeam, wait.dead())) break;
      const int rows = it.rows, listed = it.listed, biases = it.biases;
      const bool few = biases <= kBiasList;  // all of them are in shared memory
      const LogitParams p = it.p;
      auto change = [&](Elt* row, int j, int off, uint32_t word, float bias, bool biased) {
        uint32_t c = word & kCountMask;
        if (word & kIsDraft)
          for (int d = 0; d < j; ++d) c += it.draft[d] == v0 + off;
        if (c == 0 && !(word & kInPrompt) && !biased) return;
        float_to_elt(penalised(elt_to_float(row[off]), c, word & kInPrompt, bias, p), row[off]);
      };
      // the q-th listed entry; and those with biases
      auto change_listed = [&](Elt* row, int j, int q) {
        const int off = list[q];
        const uint32_t word = words[off];
        const bool biased = word & kHasBias;
        float bias = 0.f;
        if (biased) {
          if (few) return;
          for (int k = it.lo; k < it.hi; ++k)
            if (__ldg(a.bias_ids + k) == v0 + off) bias += __ldg(a.bias_values + k);
        }
        change(row, j, off, word, bias, biased);
      };
      auto change_biased = [&](Elt* row, int j, int q) {
        if (it.bias_first[q]) change(row, j, it.bias_at[q], words[it.bias_at[q]], it.bias_sum[q], true);
      };
      if (in_place) {
        // where they lie: every pair of an entry and a row is a thread's
        Elt* out = static_cast<Elt*>(a.out) + row_at(b, 0, v0);
        for (int q = threadIdx.x; q < (listed + (few ? biases : 0)) * rows; q += 2 * kLogitTeam) {
          const int e = q / rows, j = q - e * rows;
          if (it.mask[j] >= 0) continue;
          Elt* row = out + static_cast<long long>(j) * a.V;
          if (e < listed)
            change_listed(row, j, e);
          else
            change_biased(row, j, e - listed);
        }
      }
#pragma unroll 1
      for (int j = 0; j < rows; ++j) {
        const int m = it.mask[j];
        if (in_place && m < 0) continue;
        const int r = rows_copied++;
        if ((r & 1) != team) continue;
        const int slot = r % kLogitRing;
        unsigned char* buf = ring + slot * slot_bytes;
        const uintptr_t from = in_first + row_at(b, j, v0) * kElt;
        const int ph = static_cast<int>(from & 15);
        Elt* row = reinterpret_cast<Elt*>(buf + ph);
        const Span s = row_span(b, j, v0, n);
        wait(sh.row_full[slot], r / kLogitRing & 1);
        // what the copies left out at the tensors' ends, by bytes
        auto fill = [&](unsigned char* dst, uintptr_t from, int bytes, const Span& s) {
          const unsigned char* src = reinterpret_cast<const unsigned char*>(from);
          if (tid < s.head) dst[tid] = src[tid];
          if (tid < s.tail) dst[bytes - s.tail + tid] = src[bytes - s.tail + tid];
        };
        if (s.head + s.tail > 0) {
          fill(buf + ph, from, n * kElt, s);
          named_barrier(3 + team, kLogitTeam);
        }
        for (int q = tid; q < listed; q += kLogitTeam) change_listed(row, j, q);
        for (int q = tid; few && q < biases; q += kLogitTeam) change_biased(row, j, q);
        if (m >= 0) {
          const Span ms = mask_span(m, v0, n);
          const uint32_t* mask = reinterpret_cast<const uint32_t*>(buf + row_bytes + (mask_at(m, v0) & 15));
          if (ms.head + ms.tail > 0) fill(buf + row_bytes + (mask_at(m, v0) & 15), mask_at(m, v0), (n + 31) / 32 * 4, ms);
          named_barrier(3 + team, kLogitTeam);
          const int last = (n - 1) >> 5;
#pragma unroll 4
          for (int i = tid; i * 16 < ph + n * kElt; i += kLogitTeam) {
            const int v = i * N - ph / kElt;  // the vector's first entry, from the item's on (below 0: entries of no one)
            const uint32_t allow = v < 0 ? mask[0] << -v : __funnelshift_r(mask[v >> 5], mask[min((v >> 5) + 1, last)], v & 31);
            if ((allow & kAll) == kAll) continue;
            uint4* x = reinterpret_cast<uint4*>(buf + i * 16);
            uint4 y = *x;
            mask_vector<Elt>(y, allow);
            *x = y;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        warp_arrive(sh.row_done[slot]);
      }
      warp_arrive(sh.item_empty[i & 1]);
    }
  }
  if (wait.dead() && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_TIMEOUT);
}

}  // namespace specdec
