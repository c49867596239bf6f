// Host-side checks shared by the C-ABI front ends (api.cpp, api_delta.cpp,
// api_glr.cpp, api_block.cpp):
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

// Element counts stay below this, so that their bytes can be added up.
inline constexpr int64_t kLim = std::numeric_limits<int64_t>::max() / 16;

// Elements spanned by `tokens` tokens `stride` apart, each `size` long.
inline bool span(int64_t tokens, int64_t stride, int64_t size, int64_t* n) {
  *n = 0;
  if (tokens == 0 || size == 0) return true;
  int64_t m;
  if (!mul_ok(tokens - 1, stride, &m) || m > kLim - size) return false;
  *n = m + size;
  return true;
}

struct Need {
  const void* ptr;
  int64_t count;
  size_t align;
  const char* name;
  bool required;
};

// Required pointers are there (a pointer to an empty tensor may be NULL) and
// every pointer is aligned.
template <int N>
ssm_status check_pointers(const Need (&needs)[N]) {
  for (const Need& n : needs)
    if (n.required && !n.ptr && n.count > 0) return fail(SSM_ERR_NULL_POINTER, "%s is NULL", n.name);
  for (const Need& n : needs)
    if (n.ptr && !aligned(n.ptr, n.align))
      return fail(SSM_ERR_MISALIGNED, "%s is not aligned to %zu bytes", n.name, n.align);
  return SSM_OK;
}

template <int NI, int NO>
ssm_status check_overlaps(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return fail(SSM_ERR_ALIAS, "%s overlaps %s", out[i].name, r.name);
    for (int j = i + 1; j < NO; ++j)
      if (overlaps(out[i], out[j])) return fail(SSM_ERR_ALIAS, "%s overlaps %s", out[i].name, out[j].name);
  }
  return SSM_OK;
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace ssm
