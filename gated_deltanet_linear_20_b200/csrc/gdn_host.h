// Host-side checks shared by the C-ABI files.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace gdn {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// One array of a call, for the overlap checks.
struct Span {
  const void* p;
  size_t bytes;
};

// Whether any of the written arrays overlaps an input or another written
// array; an output may be exactly the input named in same[i] (or -1).
inline bool any_alias(const Span* outs, int n_out, const Span* ins, int n_in, const int* same) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j) {
      if (j == same[i] && outs[i].p == ins[j].p) continue;
      if (overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
    }
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
}

// Raises a kernel's dynamic shared-memory limit once per device to `most` bytes
// (up to 32 KB need no raising beside at most 16 KB of static shared memory).
template <auto Kernel>
bool raise_smem(size_t most) {
  static std::atomic<uint64_t> done{0};  // bit d: device d
  int dev = 0;
  if (most <= 32 * 1024) return true;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  const uint64_t bit = uint64_t(1) << dev;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most)) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

// The current device must be compute capability 10.0; *sms is its SM count.
// GDN_OK or a negative code.
int require_device(int* sms);

}  // namespace gdn
