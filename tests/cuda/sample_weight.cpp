// Test helper (host code): weights of many logits by spec_sample's function
// (csrc/sample_weight.cuh).
#include "sample_weight.cuh"

using namespace specdec;

extern "C" void weights(const float* x, int n, float max, double scale, uint64_t* out) {
  WeightScale s;
  s.hi = static_cast<float>(scale);
  s.lo = static_cast<float>(scale - s.hi);
  for (int i = 0; i < n; ++i) out[i] = sample_weight(x[i], max, s, kExp2Table);
}
