// logits_kernel.cuh — penalties, biases and grammar masks on the rows that the
// verify step reads (spec_process_logits).
//
// Few entries of a row change by a penalty or a bias: those of tokens that the
// request's history, drafts or biases name.  So the rows go through shared
// memory as they are, by bulk copies in and out, and only the named entries
// (and the masked ones) are touched there.
//
// An item is a request and `share` neighbouring entries of the vocabulary.  A
// CTA counts the item's tokens in shared memory, a 32-bit word an entry, and
// lists those it meets; every CTA reads the whole history of its item's request
// (from L2, after the first).  Then the item's rows pass through a ring of
// buffers, one load ahead and one store behind the row in work.  In place, a
// row without a mask is not copied at all: its named entries are changed where
// they lie.  Bound by the rows' bytes, read and written once.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace specdec {

constexpr int kLogitThreads = 256;
constexpr int kLogitRing = 3;        // rows in shared memory
constexpr int kLogitShare = 4096;    // most entries of an item
constexpr int kLogitLeastShare = 512;
constexpr int kBiasList = 512;       // biases of an item kept in shared memory
constexpr uint32_t kInPrompt = 1u << 31;
constexpr uint32_t kHasBias = 1u << 30;
constexpr uint32_t kIsDraft = 1u << 29;
constexpr uint32_t kCountMask = kIsDraft - 1;
// A wait gives up after this many cycles (a second).
#ifndef SPECDEC_LOGIT_WAIT_CYCLES
#define SPECDEC_LOGIT_WAIT_CYCLES 2000000000ll
#endif

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
  int32_t share;       // vocabulary entries of an item, a multiple of 32
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

// What an item needs to know of its request, as it stands in the arrays.
struct LogitRequest {
  int32_t drafts, history, prompt, lo, hi;
  LogitParams p;
  __device__ __forceinline__ void load(const LogitArgs& a, int b) {
    drafts = a.draft_len != nullptr ? __ldg(a.draft_len + b) : a.n_max;
    p.rep = a.repetition != nullptr ? __ldg(a.repetition + b) : 1.f;
    p.pres = a.presence != nullptr ? __ldg(a.presence + b) : 0.f;
    p.freq = a.frequency != nullptr ? __ldg(a.frequency + b) : 0.f;
    history = a.history_stride > 0 ? __ldg(a.history_len + b) : 0;
    prompt = a.history_stride > 0 ? __ldg(a.prompt_len + b) : 0;
    lo = a.bias_offsets != nullptr ? __ldg(a.bias_offsets + b) : 0;
    hi = a.bias_offsets != nullptr ? __ldg(a.bias_offsets + b + 1) : 0;
  }
  __device__ __forceinline__ static int rows(const LogitArgs& a, int drafts) { return max(0, min(drafts, a.n_max)) + 1; }
  // Brings all into range; whether something was out of it.
  __device__ __forceinline__ bool mend(const LogitArgs& a) {
    bool bad = drafts < 0 || drafts > a.n_max;
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
    return bad;
  }
};

struct LogitShared {
  uint64_t full[kLogitRing];
  int32_t listed;            // entries of the list
  int32_t biases;            // of the item
  int32_t draft[SPECDEC_MAX_DRAFT];
  int32_t bias_at[kBiasList];  // entry, from the item's first on
  float bias[kBiasList];       // value
  float bias_sum[kBiasList];   // of the entry from here on
  uint8_t bias_first[kBiasList];  // none of the entry's is before it
};

template <typename Elt>
struct LogitLayout {
  static __host__ __device__ int row_bytes(int share) { return share * static_cast<int>(sizeof(Elt)) + 16; }
  static __host__ __device__ int bytes(int share) { return share * 6 + kLogitRing * row_bytes(share); }
};

template <typename Elt>
__global__ void __launch_bounds__(kLogitThreads, 4) process_logits_kernel(const LogitArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ LogitShared sh;
  constexpr int kElt = sizeof(Elt);
  constexpr int N = 16 / kElt;
  uint32_t* words = reinterpret_cast<uint32_t*>(raw);
  unsigned char* ring = raw + a.share * 4;
  const int row_bytes = LogitLayout<Elt>::row_bytes(a.share);
  uint16_t* list = reinterpret_cast<uint16_t*>(ring + kLogitRing * row_bytes);
  const int tid = threadIdx.x, lane = tid & 31;
  const int items = a.B * a.chunks;
  const int rows_max = a.n_max + 1;
  const bool in_place = a.out == a.logits;
  const char* in_base = static_cast<const char*>(a.logits);
  const uintptr_t in_first = reinterpret_cast<uintptr_t>(in_base);
  const uintptr_t in_end = in_first + static_cast<unsigned long long>(a.B) * rows_max * a.V * kElt;
  bool dead = false;

  // byte of entry v0 of row j of request b
  auto at = [&](int b, int j, int v0) { return ((static_cast<long long>(b) * rows_max + j) * a.V + v0) * kElt; };

  if (tid == 0) {
    for (int i = 0; i < kLogitRing; ++i) ptx::mbar_init(ptx::smem_addr(&sh.full[i]), 1);
    ptx::fence_mbarrier_init();
    sh.listed = 0;
  }
  for (int i = tid; i < a.share / 4; i += kLogitThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();

  // The first warp goes ahead through the rows that are copied, in order.
  int next_item = blockIdx.x;  // of the coming rows
  unsigned long long next_rows = 0;
  bool next_last = false;      // row 64 is one of them
  int ahead_drafts = 0, ahead_mask[2] = {-1, -1};  // of the item after that
  auto look_ahead = [&](int item) {
    if (item >= items) return;
    const int b = item / a.chunks;
    ahead_drafts = a.draft_len != nullptr ? __ldg(a.draft_len + b) : a.n_max;
    if (in_place && a.mask_rows != nullptr) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < rows_max) ahead_mask[i] = __ldg(a.mask_rows + static_cast<long long>(b) * rows_max + lane + 32 * i);
    }
  };
  auto take_ahead = [&]() {
    const int rows = LogitRequest::rows(a, ahead_drafts);
    next_rows = rows >= 64 ? ~0ull : (1ull << rows) - 1;
    next_last = rows > 64;
    if (in_place) {
      const uint32_t m0 = __ballot_sync(0xFFFFFFFFu, ahead_mask[0] >= 0 && ahead_mask[0] < a.mask_count);
      const uint32_t m1 = __ballot_sync(0xFFFFFFFFu, ahead_mask[1] >= 0 && ahead_mask[1] < a.mask_count);
      next_rows &= static_cast<unsigned long long>(m1) << 32 | m0;
    }
  };
  int loads = 0;
  auto load_next = [&]() {
    while (next_item < items) {
      int j = -1;
      if (next_rows != 0) {
        j = __ffsll(next_rows) - 1;
        next_rows &= next_rows - 1;
      } else if (next_last) {
        j = 64;
        next_last = false;
      }
      if (j >= 0) {
        const int b = next_item / a.chunks, v0 = (next_item - b * a.chunks) * a.share;
        const uintptr_t from = in_first + at(b, j, v0), to = from + min(a.share, a.V - v0) * kElt;
        // whole 16 bytes, as far as they are the tensor's
        uintptr_t lo = from & ~static_cast<uintptr_t>(15), hi = (to + 15) & ~static_cast<uintptr_t>(15);
        uint32_t dst = ptx::smem_addr(ring + loads % kLogitRing * row_bytes);
        if (lo < in_first) lo += 16, dst += 16;
        if (hi > in_end) hi -= 16;
        const uint32_t bar = ptx::smem_addr(&sh.full[loads % kLogitRing]);
        if (lane == 0) {
          const uint32_t bytes = hi > lo ? static_cast<uint32_t>(hi - lo) : 0;
          ptx::mbar_arrive_expect_tx(bar, bytes);
          if (bytes != 0) ptx::bulk_g2s_nohint(dst, reinterpret_cast<const void*>(lo), bytes, bar);
        }
        ++loads;
        return;
      }
      next_item += gridDim.x;
      take_ahead();
      look_ahead(next_item + gridDim.x);
    }
  };
  LogitRequest ahead;
  if (static_cast<int>(blockIdx.x) < items) ahead.load(a, blockIdx.x / a.chunks);
  if (tid < 32) {
    look_ahead(next_item);
    take_ahead();
    look_ahead(next_item + gridDim.x);
    for (int i = 0; i < kLogitRing; ++i) load_next();
  }

  int step = 0;  // rows copied
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int b = item / a.chunks, v0 = (item - b * a.chunks) * a.share, n = min(a.share, a.V - v0);
    LogitRequest rq = ahead;
    if (item + static_cast<int>(gridDim.x) < items) ahead.load(a, (item + gridDim.x) / a.chunks);
    if (rq.mend(a) && a.err != nullptr && v0 == 0 && tid == 0) atomicOr(a.err, SPECDEC_DEV_ERR_PENALTY);
    const LogitParams p = rq.p;
    auto add = [&](int v, uint32_t flag) {  // an entry is named: counted, or flagged
      const uint32_t off = static_cast<uint32_t>(v) - static_cast<uint32_t>(v0);
      if (off >= static_cast<uint32_t>(n)) return;
      const uint32_t old = flag == 1 ? atomicAdd(words + off, 1u) : atomicOr(words + off, flag);
      if (old == 0) list[atomicAdd(&sh.listed, 1)] = static_cast<uint16_t>(off);
    };
    const int32_t* h = a.history + static_cast<long long>(b) * a.history_stride;
    constexpr int kIds = 8;  // in flight a thread
    for (int i0 = tid; i0 < rq.history; i0 += kIds * kLogitThreads) {
      int id[kIds];
#pragma unroll
      for (int k = 0; k < kIds; ++k) id[k] = i0 + k * kLogitThreads < rq.history ? __ldg(h + i0 + k * kLogitThreads) : -1;
#pragma unroll
      for (int k = 0; k < kIds; ++k) add(id[k], i0 + k * kLogitThreads < rq.prompt ? kInPrompt : 1u);
    }
    if (tid < rq.drafts) {
      const int v = __ldg(a.draft_tokens + static_cast<long long>(b) * a.n_max + tid);
      sh.draft[tid] = v;
      add(v, kIsDraft);
    }
    if (rq.lo < rq.hi) {
      // the item's biases, in their order
      if (tid < 32) {
        int count = 0;
        for (int i = rq.lo + lane; i - lane < rq.hi; i += 32) {
          const int v = i < rq.hi ? __ldg(a.bias_ids + i) : -1;
          const bool mine = v >= v0 && v < v0 + n;
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
          if (mine) {
            const int k = count + __popc(m & ((1u << lane) - 1));
            if (k < kBiasList) {
              sh.bias_at[k] = v - v0;
              sh.bias[k] = __ldg(a.bias_values + i);
            }
            add(v, kHasBias);
          }
          count += __popc(m);
        }
        if (lane == 0) sh.biases = count;
      }
    } else if (tid == 0) {
      sh.biases = 0;
    }
    __syncthreads();
    const int listed = sh.listed, biases = sh.biases;
    const bool few = biases <= kBiasList;  // all of them are in shared memory
    if (biases > 0 && few) {
      for (int i = tid; i < biases; i += kLogitThreads) {
        bool is_first = true;
        for (int k = 0; k < i; ++k) is_first = is_first && sh.bias_at[k] != sh.bias_at[i];
        float sum = 0.f;
        for (int k = i; k < biases; ++k)
          if (sh.bias_at[k] == sh.bias_at[i]) sum += sh.bias[k];
        sh.bias_first[i] = is_first;
        sh.bias_sum[i] = sum;
      }
      __syncthreads();
    }

    for (int j = 0; j <= rq.drafts; ++j) {
      int m = a.mask_rows != nullptr ? __ldg(a.mask_rows + static_cast<long long>(b) * rows_max + j) : -1;
      const bool masked = m >= 0 && m < a.mask_count;
      const bool copied = !in_place || masked || j == 64;
      const long long at_row = at(b, j, v0);
      const int ph = static_cast<int>((in_first + at_row) & 15);
      unsigned char* buf = ring + step % kLogitRing * row_bytes;
      Elt* row;
      if (copied) {
        if (!dead && !ptx::mbar_wait_bounded(ptx::smem_addr(&sh.full[step % kLogitRing]), step / kLogitRing & 1, SPECDEC_LOGIT_WAIT_CYCLES))
          dead = true;
        row = reinterpret_cast<Elt*>(buf + ph);
        // what the copy left out at the tensor's ends
        const uintptr_t from = in_first + at_row, to = from + static_cast<uintptr_t>(n) * kElt;
        const bool head = (from & ~static_cast<uintptr_t>(15)) < in_first, tail = ((to + 15) & ~static_cast<uintptr_t>(15)) > in_end;
        if (head || tail) {
          const Elt* src = reinterpret_cast<const Elt*>(from);
          const int first = head ? min(n, (16 - ph) / kElt) : 0;
          const int last = tail ? max(first, n - static_cast<int>(to & 15) / kElt) : n;
          if (tid < first) row[tid] = src[tid];
          if (last + tid < n) row[last + tid] = src[last + tid];
          __syncthreads();
        }
      } else {
        row = reinterpret_cast<Elt*>(static_cast<char*>(a.out) + at_row);
      }
      auto change = [&](int off, uint32_t word, float bias, bool biased) {
        uint32_t c = word & kCountMask;
        if (word & kIsDraft) {
          for (int k = 0; k < j; ++k) c += sh.draft[k] == v0 + off;
        }
        if (c == 0 && !(word & kInPrompt) && !biased) return;
        Elt x = row[off];
        float_to_elt(penalised(elt_to_float(x), c, word & kInPrompt, bias, p), x);
        row[off] = x;
      };
      for (int i = tid; i < listed; i += kLogitThreads) {
        const int off = list[i];
        const uint32_t word = words[off];
        const bool biased = word & kHasBias;
        float bias = 0.f;
        if (biased) {
          if (few) continue;  // below
          for (int k = rq.lo; k < rq.hi; ++k)
            if (__ldg(a.bias_ids + k) == v0 + off) bias += __ldg(a.bias_values + k);
        }
        change(off, word, bias, biased);
      }
      if (few) {
        for (int i = tid; i < biases; i += kLogitThreads)
          if (sh.bias_first[i]) change(sh.bias_at[i], words[sh.bias_at[i]], sh.bias_sum[i], true);
      }
      if (!copied) continue;
      if (masked) {
        __syncthreads();
        const uint32_t* mask = a.mask + static_cast<long long>(m) * a.mask_words;
        for (int i = tid; i * 16 < ph + n * kElt; i += kLogitThreads) {
          const int v = v0 + i * N - ph / kElt;  // the vector's first entry
          const uint32_t all = (1u << N) - 1;
          uint32_t allow;
          if (v >= 0) {
            const int w = v >> 5;
            allow = __funnelshift_r(__ldg(mask + w), __ldg(mask + min(w + 1, a.mask_words - 1)), v & 31);
          } else {
            allow = __ldg(mask) << -v;
          }
          if ((allow & all) != all) {
            Elt* x = reinterpret_cast<Elt*>(buf + i * 16);
            union {
              uint4 q;
              Elt e[N];
            } y;
            y.q = *reinterpret_cast<const uint4*>(x);
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (!((allow >> e) & 1)) float_to_elt(-INFINITY, y.e[e]);
            *reinterpret_cast<uint4*>(x) = y.q;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      // out: whole 16 bytes by a copy, the ends by threads
      Elt* dst = reinterpret_cast<Elt*>(static_cast<char*>(a.out) + at_row);
      int first = 0, last = 0;
      if (a.same_phase) {
        first = min(n, ph == 0 ? 0 : (16 - ph) / kElt);
        last = max(first, n - ((ph + n * kElt) & 15) / kElt);
        if (tid < first) dst[tid] = row[tid];
      }
      if (tid < 32) {
        if (lane == 0) {
          if (last > first)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + first),
                         "r"(ptx::smem_addr(row + first)), "r"((last - first) * kElt)
                         : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          // the store before this one has left its buffer, and all threads theirs
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        __syncwarp();
        if (step > 0) load_next();
      }
      for (int i = last + tid; i < n; i += kLogitThreads) dst[i] = row[i];
      ++step;
    }
    // the words as they were
    __syncthreads();
    for (int i = tid; i < listed; i += kLogitThreads) words[list[i]] = 0;
    if (tid == 0) sh.listed = 0;
    __syncthreads();
  }
  if (tid == 0) {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    // after a wait that gave up: no copy is in flight when the CTA ends
    for (int i = max(0, loads - kLogitRing); dead && i < loads; ++i)
      ptx::mbar_wait_bounded(ptx::smem_addr(&sh.full[i % kLogitRing]), i / kLogitRing & 1, SPECDEC_LOGIT_WAIT_CYCLES);
  }
  if (dead && a.err != nullptr) atomicOr(a.err, SPECDEC_DEV_ERR_TIMEOUT);
}

}  // namespace specdec
