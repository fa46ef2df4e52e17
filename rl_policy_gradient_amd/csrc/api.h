// What the host sources of the C ABI share: error reporting, the checks and
// the carving of the caller's workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/plp.h"

namespace plp {

// Stores the message plp_last_error() returns and gives `code` back; ok()
// clears it and returns PLP_OK.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 31;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline size_t esize(int dtype) { return dtype == PLP_DTYPE_F32 ? 4 : 2; }

// Sequential carving of the caller's workspace.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base((char*)b) {}
  template <typename T>
  T* take(size_t count) {
    if (count == 0) return nullptr;
    T* p = base ? (T*)(base + off) : nullptr;
    off += align_up(count * sizeof(T));
    return p;
  }
};

int check_ws(void* ws, size_t have, size_t need);

#define HIP_TRY(expr)                                                                   \
  do {                                                                                  \
    hipError_t e_ = (expr);                                                             \
    if (e_ != hipSuccess) return fail(PLP_E_HIP, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

}  // namespace plp
