// Host side of the operators around the fused loss: argument checks and
// workspace sizes of the norm, the AdamW step and token sampling. No
// allocation, no host synchronisation.
#include <math.h>

#include <algorithm>

#include "../../include/plp.h"
#include "api.h"
#include "ops.h"

using namespace plp;

namespace {

bool known_dtype(int dtype) { return dtype == PLP_DTYPE_F32 || dtype == PLP_DTYPE_BF16; }

bool misaligned(const void* p, size_t to) { return (uintptr_t)p % to != 0; }

// Whether [a, a + na) and [b, b + nb) share a byte (NULL or empty: no).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

constexpr int kMaxNormH = 65536;

int check_norm_sizes(int64_t N, int32_t H, int32_t dtype) {
  if (!known_dtype(dtype)) return fail(PLP_E_INVALID, "unknown dtype %d", dtype);
  if (N < 0 || N >= kMaxRows) return fail(PLP_E_INVALID, "N=%lld outside [0, 2^31)", (long long)N);
  if (H < 1) return fail(PLP_E_INVALID, "H must be >= 1 (got %d)", H);
  if (H > kMaxNormH) return fail(PLP_E_UNSUPPORTED, "H=%d is above %d", H, kMaxNormH);
  return PLP_OK;
}

}  // namespace

extern "C" {

PLP_API int plp_layer_norm_fwd(const void* x, const void* weight, const void* bias, int64_t N, int32_t H,
                               int32_t dtype, int32_t rms, double eps, void* y, float* mean_out, float* rstd_out,
                               hipStream_t st) {
  int rc = check_norm_sizes(N, H, dtype);
  if (rc) return rc;
  if (!(eps >= 0.0) || !isfinite(eps)) return fail(PLP_E_INVALID, "eps must be finite and >= 0");
  if (!weight) return fail(PLP_E_INVALID, "weight is required");
  if (rms && mean_out) return fail(PLP_E_INVALID, "the norm without a mean (rms) has no mean_out");
  if (N == 0) return ok();
  if (!x || !y) return fail(PLP_E_INVALID, "x and y are required");
  const size_t e = esize(dtype), xb = (size_t)N * H * e;
  if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, e) || misaligned(bias, e))
    return fail(PLP_E_INVALID, "a tensor is not aligned to its elements");
  if (overlap(y, xb, x, xb) || overlap(y, xb, weight, H * e) || overlap(y, xb, bias, H * e))
    return fail(PLP_E_INVALID, "y must not overlap an input");
  HIP_TRY(launch_norm_fwd(NormFwd{x, weight, bias, y, mean_out, rstd_out, N, H, dtype, rms ? 1 : 0, (float)eps}, st));
  return ok();
}

PLP_API int plp_layer_norm_bwd_workspace_size(int64_t N, int32_t H, int32_t dtype, size_t* bytes) {
  if (!bytes) return fail(PLP_E_INVALID, "bytes is NULL");
  int rc = check_norm_sizes(N, H, dtype);
  if (rc) return rc;
  Carver c(nullptr);
  c.take<float>((size_t)2 * norm_bwd_groups(N, H) * H);
  *bytes = c.off;
  return ok();
}

PLP_API int plp_layer_norm_bwd(const void* grad_y, const void* x, const void* weight, const float* mean,
                               const float* rstd, int64_t N, int32_t H, int32_t dtype, int32_t rms, void* grad_x,
                               void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, hipStream_t st) {
  size_t need = 0;
  int rc = plp_layer_norm_bwd_workspace_size(N, H, dtype, &need);
  if (rc) return rc;
  if (!weight) return fail(PLP_E_INVALID, "weight is required");
  if (N > 0 && (!grad_y || !x || !rstd || (!rms && !mean)))
    return fail(PLP_E_INVALID, "grad_y, x, rstd and (but for rms) mean are required");
  const size_t e = esize(dtype), xb = (size_t)N * H * e, wb = (size_t)H * e;
  if (misaligned(grad_y, e) || misaligned(x, e) || misaligned(weight, e) || misaligned(grad_x, e) ||
      misaligned(grad_weight, e) || misaligned(grad_bias, e))
    return fail(PLP_E_INVALID, "a tensor is not aligned to its elements");
  const struct {
    const void* p;
    size_t n;
  } in[] = {{grad_y, xb}, {x, xb}, {weight, wb}}, out[] = {{grad_x, xb}, {grad_weight, wb}, {grad_bias, wb}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& q : in)
      if (overlap(out[i].p, out[i].n, q.p, q.n)) return fail(PLP_E_INVALID, "a gradient must not overlap an input");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(PLP_E_INVALID, "the gradients must not overlap each other");
  }
  rc = check_ws(ws, ws_bytes, grad_weight || grad_bias ? need : 0);
  if (rc) return rc;
  HIP_TRY(launch_norm_bwd(NormBwd{grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias, (float*)ws, N, H,
                                  dtype, rms ? 1 : 0},
                          st));
  return ok();
}

}  // extern "C"
