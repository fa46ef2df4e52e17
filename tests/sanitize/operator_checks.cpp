// Host-side checks of the operators around the fused loss, for a build with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code (no GPU:
// every call here returns before any launch).
#include <stdio.h>
#include <string.h>

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
static char* at(int i) { return (char*)((uintptr_t)(i + 1) << 36); }

static plp_sample_args sample_args() {
  plp_sample_args a;
  memset(&a, 0, sizeof(a));
  a.struct_size = sizeof(a);
  a.dtype = PLP_DTYPE_BF16;
  a.N = 4;
  a.V = 1000;
  a.row_stride = 1000;
  a.logits = at(0);
  a.uniforms = (const float*)at(1);
  a.token_out = (int64_t*)at(2);
  a.temperature = 1.f;
  a.top_p = 1.f;
  return a;
}

static plp_adamw_tensor tensor(int i, int64_t n, int bits) {
  plp_adamw_tensor t;
  memset(&t, 0, sizeof(t));
  t.param = at(8 * i);
  t.grad = at(8 * i + 1);
  t.master = (float*)at(8 * i + 2);
  t.exp_avg = at(8 * i + 3);
  t.exp_avg_sq = at(8 * i + 4);
  if (bits == 8) {
    t.exp_avg_scale = (float*)at(8 * i + 5);
    t.exp_avg_sq_scale = (float*)at(8 * i + 6);
  }
  t.numel = n;
  t.param_dtype = PLP_DTYPE_BF16;
  t.grad_dtype = PLP_DTYPE_F32;
  t.state_bits = bits;
  return t;
}

static plp_adamw_args adamw_args() {
  plp_adamw_args a;
  memset(&a, 0, sizeof(a));
  a.struct_size = sizeof(a);
  a.tensor_size = sizeof(plp_adamw_tensor);
  a.lr = 1e-3;
  a.beta1 = 0.9;
  a.beta2 = 0.999;
  a.eps = 1e-8;
  a.step = 1;
  return a;
}

int main() {
  size_t bytes = 0;
  // sizes, at both ends of every range
  const int64_t Ns[] = {-1, 0, 1, 7, 4096, ((int64_t)1 << 31) - 1, (int64_t)1 << 31, INT64_MAX, INT64_MIN};
  const int32_t Vs[] = {INT32_MIN, -1, 0, 1, 255, 256, 257, 151936, 1 << 20, (1 << 20) + 1, INT32_MAX};
  for (int64_t n : Ns)
    for (int32_t v : Vs) {
      const int rc = plp_sample_tokens_workspace_size(n, v, &bytes);
      const bool ok = n >= 0 && n < (int64_t)1 << 31 && v >= 1 && v <= 1 << 20;
      CHECK((rc == PLP_OK) == ok);
      if (ok) CHECK(bytes % 256 == 0 && bytes >= (size_t)n * 12);
      for (int dt = -1; dt < 3; ++dt) {
        const bool okn = n >= 0 && n < (int64_t)1 << 31 && v >= 1 && v <= 65536 && (dt == 0 || dt == 1);
        CHECK((plp_layer_norm_bwd_workspace_size(n, v, dt, &bytes) == PLP_OK) == okn);
        if (okn) CHECK(bytes >= (size_t)v * 8 && bytes <= ((size_t)64 << 20));
      }
    }
  CHECK(plp_sample_tokens_workspace_size(1, 1, nullptr) == PLP_E_INVALID);
  CHECK(plp_layer_norm_bwd_workspace_size(1, 1, 0, nullptr) == PLP_E_INVALID);

  // sampling
  CHECK(plp_sample_tokens(nullptr, nullptr, 0, nullptr) == PLP_E_INVALID);
  {
    plp_sample_args a = sample_args();
    CHECK(plp_sample_tokens(&a, nullptr, 0, nullptr) == PLP_E_WORKSPACE);
    a.N = 0;
    CHECK(plp_sample_tokens(&a, nullptr, 0, nullptr) == PLP_OK);
    a = sample_args();
    a.struct_size = 4;
    CHECK(plp_sample_tokens(&a, at(5), 1 << 20, nullptr) == PLP_E_INVALID);
    const float bad[] = {-1.f, 1.f / 0.f, 0.f / 0.f};
    for (float x : bad) {
      a = sample_args();
      a.temperature = x;
      CHECK(plp_sample_tokens(&a, at(5), 1 << 20, nullptr) == PLP_E_INVALID);
      a = sample_args();
      a.top_p = x;
      CHECK(plp_sample_tokens(&a, at(5), 1 << 20, nullptr) == PLP_E_INVALID);
      a = sample_args();
      a.min_p = x;
      CHECK(plp_sample_tokens(&a, at(5), 1 << 20, nullptr) == PLP_E_INVALID);
    }
    a = sample_args();
    a.row_stride = INT64_MIN;
    CHECK(plp_sample_tokens(&a, at(5), 1 << 20, nullptr) == PLP_E_INVALID);
    a = sample_args();
    a.logits = at(0) + 1;
    CHECK(plp_sample_tokens(&a, at(5), 1 << 20, nullptr) == PLP_E_INVALID);
  }

  // the norm
  CHECK(plp_layer_norm_fwd(nullptr, nullptr, nullptr, 1, 8, 0, 0, 1e-5, nullptr, nullptr, nullptr, nullptr) ==
        PLP_E_INVALID);
  CHECK(plp_layer_norm_fwd(at(0), at(1), nullptr, 8, 65536, 0, 0, 1e-5, at(0) + 8 * 65536 * 4 - 1, nullptr, nullptr,
                           nullptr) == PLP_E_INVALID);
  CHECK(plp_layer_norm_fwd(at(0), at(1), nullptr, ((int64_t)1 << 31) - 1, 65536, 1, 0, 1e-5, at(0), nullptr, nullptr,
                           nullptr) == PLP_E_INVALID);
  CHECK(plp_layer_norm_bwd(at(0), at(1), at(2), nullptr, (float*)at(3), 8, 64, 1, 0, at(4), at(5), at(6), at(7),
                           1 << 20, nullptr) == PLP_E_INVALID);
  CHECK(plp_layer_norm_bwd(at(0), at(1), at(2), nullptr, (float*)at(3), 8, 64, 1, 1, at(4), at(5), at(6), at(7), 16,
                           nullptr) == PLP_E_WORKSPACE);

  // AdamW: a long list whose last tensor is bad
  for (int bits : {8, 32}) {
    std::vector<plp_adamw_tensor> list;
    for (int i = 0; i < 200; ++i) list.push_back(tensor(i, i * 37 % 5000, bits));
    plp_adamw_args a = adamw_args();
    list.back() = tensor(199, -1, bits);
    CHECK(plp_adamw_step(&a, list.data(), (int)list.size(), nullptr) == PLP_E_INVALID);
    CHECK(strstr(plp_last_error(), "tensor 199") != nullptr);
    list.back() = tensor(199, INT64_MAX, bits);
    CHECK(plp_adamw_step(&a, list.data(), (int)list.size(), nullptr) == PLP_E_INVALID);
    list.back() = tensor(199, 1000, bits);
    list.back().exp_avg = (char*)list.back().param + 1000;
    CHECK(plp_adamw_step(&a, list.data(), (int)list.size(), nullptr) == PLP_E_INVALID);
    for (auto& t : list) t.numel = 0;
    CHECK(plp_adamw_step(&a, list.data(), (int)list.size(), nullptr) == PLP_OK);
    a.step = INT64_MIN;
    CHECK(plp_adamw_step(&a, list.data(), 1, nullptr) == PLP_E_INVALID);
  }
  if (g_fail) return 1;
  puts("operator checks passed");
  return 0;
}
