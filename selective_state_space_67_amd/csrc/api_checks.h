// Host-side checks shared by the C-ABI front ends (api.cpp, api_delta.cpp):
// the error text, element sizes, overflow-safe products, alignment and byte
// ranges. Plain host arithmetic; nothing here touches the HIP runtime.
#pragma once

#include <cstddef>
#include <cstdint>
#include <limits>

#include "ssm_scan.h"

namespace ssm {

// Sets the calling thread's error text and returns `s` (defined in api.cpp).
ssm_status fail(ssm_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the error text.
ssm_status ok();

inline bool valid_dtype(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
inline size_t dtype_size(int32_t t) { return t == SSM_BF16 ? 2 : 4; }

// a * b without overflow for non-negative operands.
inline bool mul_ok(int64_t a, int64_t b, int64_t* r) {
  if (a != 0 && b > std::numeric_limits<int64_t>::max() / a) return false;
  *r = a * b;
  return true;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A byte range [p, p + n) of one tensor; empty when p is null.
struct Range {
  const char* p;
  size_t n;
  const char* name;
};

inline bool overlaps(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  return a.p < b.p + b.n && b.p < a.p + a.n;
}

inline Range range(const void* p, int64_t count, size_t esize, const char* name) {
  return Range{static_cast<const char*>(p), p ? static_cast<size_t>(count) * esize : 0, name};
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace ssm
