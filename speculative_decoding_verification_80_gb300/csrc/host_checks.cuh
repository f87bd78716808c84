// host_checks.cuh — what the entry points of the step's operators check and ask
// on the host.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "specdec.h"

namespace specdec {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline specdec_status_t launched() { return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA; }

inline bool block_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

// Whether p is memory that the CUDA runtime gave out (false without a device).
inline bool on_device(const void* p) {
  cudaPointerAttributes at;
  if (p == nullptr) return false;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

// Memory that a call reads or writes.  An output may be one input where `same` names it.
struct Span {
  const void* at;
  size_t bytes;
  const void* same = nullptr;
};

inline bool overlap(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.at), b = reinterpret_cast<uintptr_t>(y.at);
  if (x.at == nullptr || y.at == nullptr || x.bytes == 0 || y.bytes == 0) return false;
  return a <= b ? b - a < x.bytes : a - b < y.bytes;
}

// Whether an output lies on another output, or on an input that it may not be.
template <int I, int O>
bool outputs_collide(const Span (&in)[I], const Span (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(out[o], in[i]) && !(out[o].at == in[i].at && out[o].same == in[i].at && out[o].bytes == in[i].bytes)) return true;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return true;
  }
  return false;
}

// SMs of the current device, which is asked once.
inline cudaError_t device_sms(int* dev, int* sms) {
  static int known[64] = {0};
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= 64) return cudaErrorInvalidDevice;
  if (known[*dev] == 0) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev);
    if (e != cudaSuccess) return e;
    known[*dev] = n;
  }
  *sms = known[*dev];
  return cudaSuccess;
}

}  // namespace specdec
