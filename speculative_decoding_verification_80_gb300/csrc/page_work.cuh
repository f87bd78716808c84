// page_work.cuh — the workspace of kv_fork and kv_compact.  Host code: its test
// compiles it without nvcc.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "specdec.h"

namespace specdec {

// What is zero between two calls lies from the start on: counts of a block's names in
// the old and new tables, requests that write it, the last of those; a bit a free
// block.  Scratch lies before the end: a bit a block that goes back, a block's place
// among the moves, a request's number among those that copy.  So a pool of any size
// that the workspace is large enough for finds its counts zero after another's call:
// both parts grow with N, and the largest N's meet at most.
struct PageWork {
  uint32_t* olds;
  uint32_t* news;
  uint32_t* writers;
  uint32_t* last;       // request + 1
  uint32_t* marks;
  uint32_t* gone;
  int32_t* rank;
  int32_t* number;
  int32_t* ring;        // head, count as they were, clamped
};

inline size_t page_scratch_words(int64_t N) { return static_cast<size_t>(N + (N + 31) / 32 + SPECDEC_MAX_BATCH + 2); }
inline size_t page_words(int64_t N) { return static_cast<size_t>(4 * N + (N + 31) / 32) + page_scratch_words(N); }

inline PageWork page_work(void* workspace, size_t bytes, int64_t N) {
  uint32_t* at = static_cast<uint32_t*>(workspace);
  PageWork w;
  w.olds = at;
  w.news = w.olds + N;
  w.writers = w.news + N;
  w.last = w.writers + N;
  w.marks = w.last + N;
  w.gone = at + (bytes / 4 - page_scratch_words(N));
  w.rank = reinterpret_cast<int32_t*>(w.gone + (N + 31) / 32);
  w.number = w.rank + N;
  w.ring = w.number + SPECDEC_MAX_BATCH;
  return w;
}

}  // namespace specdec
