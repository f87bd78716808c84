// waits.cuh — barriers of some of a CTA's warps, and waits that give up, for the
// kernels whose warps have roles (spec_attention, spec_process_logits).
#pragma once
#include <stdint.h>

#include "ptx.cuh"

// A wait gives up after this many looks: two seconds (measured: 3.7 us a look,
// most of it the look itself, which suspends the thread).  No wait is for another
// CTA; the longest is for a segment of the attention, at most some 100 ms.
#ifndef SPECDEC_STEP_WAIT_LOOKS
#define SPECDEC_STEP_WAIT_LOOKS (1u << 19)
#endif

namespace specdec {

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whether `x` holds for any thread of the barrier.
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// A wait that gives up once; after that the thread goes on without waiting, so
// that every barrier still gets its arrivals, to the end of its segment or item.
// What decides how often a group of warps meets at a barrier is agreed on at
// one.  (It is in some 50 places of the attention, and the instruction cache is
// small: it counts looks where a clock would take twice the code.  A clock also
// goes on while the context does not run.)
struct Waiter {
  uint32_t looks = SPECDEC_STEP_WAIT_LOOKS;  // 0: gave up
  __device__ __forceinline__ bool dead() const { return looks == 0; }
  __device__ __forceinline__ void operator()(const uint64_t& bar, uint32_t parity, uint32_t pause = 32) {
    const uint32_t at = ptx::smem_addr(&bar);
    uint32_t left = looks;
#pragma unroll 1
    while (!ptx::mbar_try_wait(at, parity)) {
      if (left == 0) {
        looks = 0;
        break;
      }
      --left;
      __nanosleep(pause);
    }
  }
};

}  // namespace specdec
