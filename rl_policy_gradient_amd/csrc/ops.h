// Launchers of the operators around the fused loss: the norm, the AdamW step
// and token sampling. Each enqueues on `st` and returns the launch's
// hipError_t; every argument has been checked by the host (operators_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace plp {

// y = (x - mean) * rstd * w + b over rows of H, statistics into mean (layer
// only) and rstd, either of which may be NULL.
struct NormFwd {
  const void *x, *w, *b;
  void* y;
  float *mean, *rstd;
  int64_t N;
  int H, dtype, rms;
  float eps;
};
hipError_t launch_norm_fwd(const NormFwd& a, hipStream_t st);

// The gradients of that; gx, gw and gb may each be NULL. part: 2 x
// norm_bwd_groups(N, H) x H floats when gw or gb is asked for.
struct NormBwd {
  const void *gy, *x, *w;
  const float *mean, *rstd;
  void *gx, *gw, *gb;
  float* part;
  int64_t N;
  int H, dtype, rms;
};
hipError_t launch_norm_bwd(const NormBwd& a, hipStream_t st);
// Row groups whose partial sums of the weight's gradient are added up at the
// end; a function of the sizes alone, so results do not depend on the device.
int norm_bwd_groups(int64_t N, int H);

}  // namespace plp
