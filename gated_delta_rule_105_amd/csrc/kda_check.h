// Host-side argument checks of the C front ends kda_layer_api.cpp and
// kda_block_api.cpp (the same rules as kda_api.cpp's own).  Plain C++,
// internal linkage.
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

struct Tokens {
  size_t n;     // tokens of the whole batch
  size_t seqs;  // sequences
};

// The batch of B rows of T tokens, or n_seqs packed sequences.
int check_tokens(int B, int T, int n_seqs, int dtype, Tokens* t) {
  if (B < 1 || T < 0 || n_seqs < 0) return KDA_ERR_INVALID_ARGUMENT;
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARGUMENT;
  if (n_seqs > 0 && B != 1) return KDA_ERR_INVALID_ARGUMENT;
  t->n = (size_t)B * (size_t)T;
  t->seqs = n_seqs > 0 ? (size_t)n_seqs : (size_t)B;
  return t->n > (size_t)INT32_MAX ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// Bytes between the first and the last element of `rows` rows of `row`
// elements, `ld` elements apart; ld 0 means contiguous.  False: ld is shorter
// than a row, or the size overflows.
bool strided(size_t rows, size_t row, int64_t* ld, size_t esz, size_t* bytes) {
  if (*ld == 0) *ld = (int64_t)row;
  if (*ld < 0 || (size_t)*ld < row) return false;
  if (rows == 0) {
    *bytes = 0;
    return true;
  }
  size_t last;
  if (!mul(rows - 1, (size_t)*ld, &last) || last > SIZE_MAX - row || !mul(last + row, esz, bytes)) return false;
  return *bytes <= SIZE_MAX / 2;
}

bool bytes_of(size_t a, size_t b, size_t c, size_t esz, size_t* out) {
  size_t ab, abc;
  return mul(a, b, &ab) && mul(ab, c, &abc) && mul(abc, esz, out) && *out <= SIZE_MAX / 2;
}

// Ranges of a call's inputs and outputs; outputs overlap nothing.
struct Buffers {
  Range in[16], out[16];
  int n_in = 0, n_out = 0;
  bool fine = true;
  void input(const void* p, size_t bytes, size_t align) {
    fine = fine && aligned(p, align);
    in[n_in++] = range(p, p ? bytes : 0);
  }
  void output(const void* p, size_t bytes, size_t align) {
    fine = fine && aligned(p, align);
    out[n_out++] = range(p, p ? bytes : 0);
  }
  bool valid() const {
    if (!fine) return false;
    for (int i = 0; i < n_out; ++i) {
      for (int j = 0; j < n_in; ++j)
        if (overlap(out[i], in[j])) return false;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return false;
    }
    return true;
  }
};

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return KDA_OK;
  if (!ws || !aligned(ws, kWsAlign)) return KDA_ERR_INVALID_ARGUMENT;
  return have < need ? KDA_ERR_WORKSPACE_TOO_SMALL : KDA_OK;
}

int hip_status(int e) { return e == 0 ? KDA_OK : KDA_ERR_HIP; }

}  // namespace
