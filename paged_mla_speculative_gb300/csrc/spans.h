// Memory that a call is given, and whether what it writes lies in any other.
// Plain C++: its tests run on the host.
#pragma once

#include <stdint.h>

namespace mlav {

// `rows` rows of `bytes` bytes, `stride` bytes apart (at least `bytes`).
struct Span {
  uintptr_t base;
  int64_t rows, stride, bytes;
};
inline Span flat_span(const void* p, int64_t bytes) { return Span{reinterpret_cast<uintptr_t>(p), 1, 0, bytes}; }
inline Span row_span(const void* p, int64_t rows, int64_t stride, int64_t bytes) {
  return Span{reinterpret_cast<uintptr_t>(p), rows, stride, bytes};
}

// Whether a byte is in both.
inline bool overlap(const Span& a, const Span& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.bytes <= 0 || b.bytes <= 0) return false;
  const auto end = [](const Span& s) { return s.base + static_cast<uintptr_t>((s.rows - 1) * s.stride + s.bytes); };
  if (a.base >= end(b) || b.base >= end(a)) return false;
  // Each row of the one with fewer, and of the other the first row that ends
  // behind the row's beginning.
  const Span& few = a.rows <= b.rows ? a : b;
  const Span& many = a.rows <= b.rows ? b : a;
  for (int64_t i = 0; i < few.rows; ++i) {
    const int64_t from = static_cast<int64_t>(few.base + static_cast<uintptr_t>(i * few.stride) - many.base);   // beside `many`
    const int64_t first = from < many.bytes || many.rows == 1 ? 0 : (from - many.bytes) / many.stride + 1;
    if (first < many.rows && first * many.stride < from + few.bytes && from < first * many.stride + many.bytes) return true;
  }
  return false;
}

// Whether any of the spans that are written overlaps another of them or one that is read.
inline bool any_overlap(const Span* written, int nwritten, const Span* read, int nread) {
  for (int i = 0; i < nwritten; ++i) {
    for (int k = i + 1; k < nwritten; ++k)
      if (overlap(written[i], written[k])) return true;
    for (int k = 0; k < nread; ++k)
      if (overlap(written[i], read[k])) return true;
  }
  return false;
}

}  // namespace mlav
