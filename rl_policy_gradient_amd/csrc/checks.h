// Argument checks shared by the host sources of the operators.
#pragma once

#include "api.h"

namespace plp {

inline bool known_dtype(int dtype) { return dtype == PLP_DTYPE_F32 || dtype == PLP_DTYPE_BF16; }

inline bool misaligned(const void* p, size_t to) { return (uintptr_t)p % to != 0; }

// Whether [a, a + na) and [b, b + nb) share a byte (NULL or empty: no).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

struct Range {
  const void* p;
  size_t n;
};

// No output may share a byte with an input or with another output.
template <size_t I, size_t O>
int check_apart(const Range (&in)[I], const Range (&out)[O]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Range& q : in)
      if (overlap(out[i].p, out[i].n, q.p, q.n)) return fail(PLP_E_INVALID, "an output must not overlap an input");
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(PLP_E_INVALID, "outputs must not overlap each other");
  }
  return PLP_OK;
}

}  // namespace plp
