// host_checks.h -- what the entry points of the 8-bit cache check their
// arguments with.
#pragma once

#include <stdint.h>

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

}  // namespace npk
