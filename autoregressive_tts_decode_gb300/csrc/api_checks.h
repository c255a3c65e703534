// api_checks.h -- checks of host-side arguments that the C entries over
// caller-owned buffers share (ops_api.cu, kv8_api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace {

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// [p, p + n) and [q, q + m) share a byte
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + m && b < a + n;
}

// Rows of a call: n of `bytes` bytes, `stride` (at least bytes) apart.
struct Span {
  const void* p;
  size_t bytes, stride;
  long long n;
};
inline uintptr_t start_of(const Span& r) { return (uintptr_t)r.p; }
inline uintptr_t end_of(const Span& r) { return (uintptr_t)r.p + (size_t)(r.n - 1) * r.stride + r.bytes; }

// A row of a and a row of b share a byte (rows that lie between each other's, as
// the fields of records do, need not).
inline bool rows_overlap(const Span& a, const Span& b) {
  if (!a.bytes || !b.bytes || a.n < 1 || b.n < 1) return false;
  if (start_of(a) >= end_of(b) || start_of(b) >= end_of(a)) return false;
  if (a.stride == b.stride) {
    // row i + d of b starts diff + d stride after row i of a: the least d in range for
    // which it does not end before that row, and whether it then starts before its end
    const long long st = (long long)a.stride, diff = (long long)start_of(b) - (long long)start_of(a);
    long long d = (-diff - (long long)b.bytes) / st - 1;
    while (diff + d * st <= -(long long)b.bytes) ++d;  // (two steps at most)
    d = std::max(d, 1 - a.n);
    return d < b.n && diff + d * st < (long long)a.bytes;
  }
  uintptr_t x = start_of(a), y = start_of(b);
  for (long long i = 0, j = 0; i < a.n && j < b.n;) {
    if (x + a.bytes <= y) {  // (all of a's rows up to the one that y may meet)
      const long long skip = (long long)((y - x - a.bytes) / a.stride) + 1;
      i += skip;
      x += (size_t)skip * a.stride;
    } else if (y + b.bytes <= x) {
      const long long skip = (long long)((x - y - b.bytes) / b.stride) + 1;
      j += skip;
      y += (size_t)skip * b.stride;
    } else {
      return true;
    }
  }
  return false;
}

}  // namespace
