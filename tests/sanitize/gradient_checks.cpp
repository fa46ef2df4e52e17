// Host-side checks of the embedding and the gradients' norm, for a build with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code (no GPU:
// every call here returns before any launch).
#include <math.h>
#include <stdio.h>

#include <vector>

#include "plp.h"

static int g_fail = 0;

#define CHECK(cond)                                                    \
  do {                                                                 \
    if (!(cond)) {                                                     \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      g_fail = 1;                                                      \
    }                                                                  \
  } while (0)

// made-up device addresses, far apart; never followed
static char* at(int i) { return (char*)((uintptr_t)(i + 1) << 44); }

int main() {
  size_t bytes = 0;
  const int64_t Ns[] = {INT64_MIN, -1, 0, 1, 4096, 4097, 100000, ((int64_t)1 << 31) - 1, (int64_t)1 << 31, INT64_MAX};
  const int32_t Vs[] = {INT32_MIN, -1, 0, 1, 1023, 1024, 151936, 1 << 20, INT32_MAX};
  const int32_t Hs[] = {INT32_MIN, 0, 1, 7, 512, 513, 65536, 65537, INT32_MAX};
  for (int64_t n : Ns)
    for (int32_t v : Vs)
      for (int32_t h : Hs)
        for (int dt = -1; dt < 3; ++dt)
          for (int acc = 0; acc < 2; ++acc) {
            const bool ok = n >= 0 && n < (int64_t)1 << 31 && v >= 1 && h >= 1 && h <= 65536 && (dt == 0 || dt == 1);
            CHECK((plp_embedding_bwd_workspace_size(n, h, v, dt, &bytes) == PLP_OK) == ok);
            if (!ok) continue;
            CHECK(bytes % 256 == 0 && bytes >= (size_t)n * 8);
            // everything but the workspace in order: refused by its size alone
            if (n > 0)
              CHECK(plp_embedding_bwd((const int64_t*)at(0), at(20), n, h, v, dt, 0, 1.f, acc, at(200), at(900), bytes - 1,
                                      nullptr) == PLP_E_WORKSPACE);
            CHECK(plp_embedding_fwd((const int64_t*)at(0), at(20), n, h, v, dt, INFINITY, at(200), nullptr) ==
                  PLP_E_INVALID);
          }
  // lists around the ends of a launch and of a tile, whose tables are made before the workspace is looked at
  for (int count : {0, 1, 239, 240, 241, 501, 5000})
    for (int64_t numel : {(int64_t)0, (int64_t)1, (int64_t)2047, (int64_t)2049, (int64_t)1 << 27}) {
      std::vector<plp_grad_tensor> t(count);
      for (int i = 0; i < count; ++i) t[i] = plp_grad_tensor{at(0), numel + i % 3, i % 2, 0};
      CHECK(plp_grad_norm_workspace_size(t.data(), count, &bytes) == PLP_OK);
      CHECK(bytes >= (size_t)count * 12 && bytes % 256 == 0);
      if (count > 0)
        CHECK(plp_grad_norm(t.data(), count, 1.0, 0.0, nullptr, (float*)at(20), (float*)at(21), (float*)at(22), at(23),
                            bytes - 1, nullptr) == PLP_E_WORKSPACE);
      CHECK(plp_grad_norm(t.data(), count, NAN, 0.0, nullptr, (float*)at(20), (float*)at(21), nullptr, at(23), bytes,
                          nullptr) == PLP_E_INVALID);
      CHECK(plp_clip_grads(t.data(), count, nullptr, nullptr) == PLP_E_INVALID);
    }
  CHECK(plp_grad_norm_workspace_size(nullptr, 1, &bytes) == PLP_E_INVALID);
  CHECK(plp_grad_norm_workspace_size(nullptr, INT32_MIN, &bytes) == PLP_E_INVALID);
  if (!g_fail) printf("gradient checks passed\n");
  return g_fail;
}
