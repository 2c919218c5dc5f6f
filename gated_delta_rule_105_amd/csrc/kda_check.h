// Host-side argument checks of the C front end kda_layer_api.cpp (the same
// rules as kda_api.cpp's own).  Plain C++, internal linkage.
#pragma once

#include "kda.h"

#include <stdint.h>
#include <string.h>

namespace {

constexpr size_t kWsAlign = 256;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
Range range(const void* p, size_t bytes) { return Range{(uintptr_t)p, (uintptr_t)p + bytes}; }
bool overlap(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

// Multiply non-negative sizes, flagging overflow of size_t.
bool mul(size_t a, size_t b, size_t* out) {
  if (a != 0 && b > SIZE_MAX / a) return false;
  *out = a * b;
  return true;
}

// Enum-typed arguments as their int representation: a C caller may store any
// int in them, and loading a value outside the enumerators through the enum
// type is undefined in C++, so they are only ever read this way.
template <typename E>
int as_int(const E& e) {
  static_assert(sizeof(E) == sizeof(int), "C enums are int-sized here");
  int v;
  memcpy(&v, &e, sizeof v);
  return v;
}

size_t elem_size(int t) { return t == KDA_DTYPE_BF16 ? 2 : 4; }

}  // namespace
