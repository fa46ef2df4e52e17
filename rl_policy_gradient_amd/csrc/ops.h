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
// norm_bwd_groups(N, H) x H floats when gw or gb is asked for, else NULL.
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

// One tensor of the AdamW step (a plp_adamw_tensor, checked).
struct AdamTensor {
  void* param;
  const void* grad;
  float* master;       // or NULL: the step works on param
  void* m;             // fp32, or e4m3 codes
  void* v;             // fp32 second moment, or e4m3 codes of its root
  float *ms, *vs;      // 8-bit states: one scale per kAdamBlock elements
  int64_t n;
  float decay;         // lr weight_decay (weight_decay when the rate is read on the device)
  uint8_t param_bf16, grad_bf16, bits8;
};
constexpr int kAdamBlock = 256;   // elements of one scale
constexpr int kAdamTile = 1024;   // elements a workgroup takes
// Tensors of one launch: the table goes by value in the kernel's arguments,
// which hold 4 KB.
constexpr int kAdamMaxTensors = 52;
struct AdamLaunch {
  AdamTensor t[kAdamMaxTensors];
  uint32_t first[kAdamMaxTensors + 1];  // the workgroup each tensor begins at
  int count;
  float b1, c1, b2, c2;      // beta and 1 - beta
  float eps;
  float step_size, inv_root; // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), unless step_dev or lr_dev
  double lr, ln_b1, ln_b2;
  const int64_t* step_dev;
  int64_t step;
  const float *lr_dev, *grad_scale;
};
static_assert(sizeof(AdamLaunch) <= 4096, "kernel arguments");
hipError_t launch_adamw(const AdamLaunch& a, hipStream_t st);

// Sampling one token a row of logits; block_max and block_sum are workspace,
// sample_blocks(V) of each a row.
struct SampleArgs {
  const void* logits;
  const float* uniforms;
  float tau, top_p, min_p;
  int top_k;
  const float *tau_rows, *top_p_rows, *min_p_rows;  // instead of the scalars, or NULL
  const int32_t* top_k_rows;
  int64_t* token;
  float *logp, *kept_logp;
  double* block_sum;
  float* block_max;
  int64_t N, stride;
  int V, dtype;
};
constexpr int kSampleBlock = 256;  // logits of one block
// Blocks of a row of V logits, the first of which may begin up to seven
// elements before the row (at a multiple of 16 bytes).
inline int sample_blocks(int V) { return (V + 7 + kSampleBlock - 1) / kSampleBlock; }
constexpr int kSampleMaxV = 1 << 20;
hipError_t launch_sample(const SampleArgs& a, hipStream_t st);

}  // namespace plp
