// host_checks.h -- what the entry points of the prompt side and of the 8-bit
// cache check their arguments with, and the device's size.
#pragma once

#include <stdint.h>

#include <atomic>

#include <cuda_runtime.h>

namespace npk {

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b without int64 overflow (a, b >= 0)
inline bool mul_fits(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

// An array of n bytes.
struct Span {
  const void* p;
  int64_t n;
};

inline bool overlaps(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p && y.p && x.n > 0 && y.n > 0 && a < b + (uintptr_t)y.n && b < a + (uintptr_t)x.n;
}

// Whether one of the first `written` spans shares a byte with any other span.
template <int N>
inline bool any_overlap(const Span (&s)[N], int written) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < N; ++j)
      if (overlaps(s[i], s[j])) return true;
  return false;
}

// The current device's SMs; 0: no device.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, s = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64) s = known[dev].load();
  if (s == 0) {
    if (cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(s);
  }
  return s;
}

}  // namespace npk
