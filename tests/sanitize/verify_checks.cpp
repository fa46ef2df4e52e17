// Host-side checks of the verification of drafted tokens, for a build with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code (no GPU:
// every call here returns before any launch).
#include <math.h>
#include <stdio.h>
#include <string.h>

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
static char* at(int i) { return (char*)((uintptr_t)(i + 1) << 56); }

int main() {
  size_t bytes = 0;
  const int64_t Bs[] = {INT64_MIN, -1, 0, 1, 100, ((int64_t)1 << 31) - 1, (int64_t)1 << 31, INT64_MAX};
  const int32_t Ks[] = {INT32_MIN, -1, 0, 1, 1024, 1025, INT32_MAX};
  const int32_t Vs[] = {INT32_MIN, 0, 1, 255, 257, 1 << 20, (1 << 20) + 1, INT32_MAX};
  const int64_t strides[] = {INT64_MIN, -1, 0, 1, 1000, (int64_t)1 << 40, INT64_MAX};
  for (int64_t B : Bs)
    for (int32_t K : Ks)
      for (int32_t V : Vs)
        for (int drafts = 0; drafts < 2; ++drafts) {
          const bool ok = B >= 0 && B < (int64_t)1 << 31 && K >= 0 && K <= 1024 && V >= 1 && V <= 1 << 20;
          CHECK((plp_verify_tokens_workspace_size(B, K, V, drafts, &bytes) == PLP_OK) == ok);
          if (ok) CHECK(bytes % 256 == 0);
          for (int64_t s : strides)
            for (int64_t r : strides) {
              plp_verify_args a;
              memset(&a, 0, sizeof(a));
              a.struct_size = sizeof(a);
              a.dtype = PLP_DTYPE_BF16;
              a.B = B, a.K = K, a.V = V;
              a.logits = at(0);
              a.draft_logits = drafts ? at(10) : nullptr;
              a.seq_stride = a.draft_row_stride = s;
              a.row_stride = a.draft_seq_stride = r;
              a.draft_tokens = (const int64_t*)at(20);
              a.uniforms = (const float*)at(30);
              a.tokens_out = (int64_t*)at(40);
              a.accepted_out = (int32_t*)at(50);
              a.target.temperature = a.draft.temperature = a.target.top_p = a.draft.top_p = 1.f;
              const int rc = plp_verify_tokens(&a, nullptr, 0, nullptr);
              if (ok && B == 0 && s >= 0 && r >= 0) CHECK(rc == PLP_OK);
              else CHECK(rc != PLP_OK);
            }
        }
  CHECK(plp_verify_tokens(nullptr, nullptr, 0, nullptr) == PLP_E_INVALID);
  if (!g_fail) printf("verify checks passed\n");
  return g_fail;
}
