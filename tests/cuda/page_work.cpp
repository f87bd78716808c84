// Test helper (host code): where kv_fork's and kv_compact's arrays lie in their
// workspace (csrc/page_work.cuh), in words from its start: begin and end of each.
#include "page_work.cuh"

using namespace specdec;

extern "C" long long words_of(long long N) { return static_cast<long long>(page_words(N)); }

extern "C" void arrays_of(void* workspace, long long bytes, long long N, long long (*at)[2]) {
  const PageWork w = page_work(workspace, static_cast<size_t>(bytes), N);
  const uint32_t* base = static_cast<const uint32_t*>(workspace);
  const long long bits = (N + 31) / 32;
  const void* start[9] = {w.olds, w.news, w.writers, w.last, w.marks, w.gone, w.rank, w.number, w.ring};
  const long long size[9] = {N, N, N, N, bits, bits, N, SPECDEC_MAX_BATCH, 2};
  for (int i = 0; i < 9; ++i) {
    at[i][0] = static_cast<const uint32_t*>(start[i]) - base;
    at[i][1] = at[i][0] + size[i];
  }
}
