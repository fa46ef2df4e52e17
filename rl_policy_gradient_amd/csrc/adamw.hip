// AdamW over a list of tensors in one launch:
//
//   g' = grad_scale g, m' = b1 m + (1 - b1) g', v' = b2 v + (1 - b2) g'^2,
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// with m and v in fp32, or in 8 bits: e4m3 codes of m and of r = sqrt(v), one
// fp32 scale (largest magnitude / 448) for each 256 consecutive elements.
// The root is kept rather than v because a code spans 2^18 of whatever it
// holds: that is 2^18 of gradient magnitudes this way, 2^9 the other. A root
// above zero keeps a code above zero, else an element whose m outlives its v
// would step by m / eps.
//
// Every element is read once and written once; nothing is reused, so the
// step is bound by HBM.
#include "ops.h"

#include <math.h>

namespace plp {

namespace {

constexpr int NT = 256;
constexpr float kCodeMax = 448.f;      // largest e4m3 value
constexpr float kCodeMin = 0x1p-9f;    // smallest above zero
constexpr float kScaleMin = 0x1p-126f; // a smaller scale's inverse would overflow

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

__device__ __forceinline__ float from_e4m3(uint8_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }
__device__ __forceinline__ uint8_t to_e4m3(float x) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.f, 0, false) & 0xff);
}

// The scalars of one step.
struct Scalars {
  float b1, c1, b2, c2, eps, step_size, inv_root, gscale, lr;
};

// With the step or the rate in device memory the corrections are formed here,
// in fp64 (1 - b^t as -expm1(t ln b), which does not cancel for small t).
__device__ Scalars scalars(const AdamLaunch& a) {
  Scalars s{a.b1, a.c1, a.b2, a.c2, a.eps, a.step_size, a.inv_root, 1.f, (float)a.lr};
  if (a.step_dev || a.lr_dev) {
    const int64_t t = a.step_dev ? (*a.step_dev < 1 ? 1 : *a.step_dev) : a.step;
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    s.step_size = (float)(lr / -expm1((double)t * a.ln_b1));
    s.inv_root = (float)(1.0 / sqrt(-expm1((double)t * a.ln_b2)));
    s.lr = (float)lr;
  }
  if (a.grad_scale) s.gscale = *a.grad_scale;
  return s;
}

struct Updated {
  float p, m, r, v;
};

// One element. Products and sums are rounded one by one: with a contraction
// the 8-bit code of a value at a tie would depend on the compiler's choice.
__device__ __forceinline__ Updated update(float p, float g, float m, float v, float keep, const Scalars& s) {
#pragma clang fp contract(off)
  g = g * s.gscale;
  Updated u;
  u.m = m * s.b1 + g * s.c1;
  u.v = v * s.b2 + g * g * s.c2;
  u.r = sqrtf(u.v);
  u.p = p * keep - u.m / (u.r * s.inv_root + s.eps) * s.step_size;
  return u;
}

__device__ __forceinline__ float load(const void* p, int64_t i, bool bf16) {
  return bf16 ? (float)((const __bf16*)p)[i] : ((const float*)p)[i];
}

// Largest finite magnitude over the block of 256 threads.
__device__ float block_absmax(float x, float* red) {
  x = finite(x) ? fabsf(x) : 0.f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  const float r = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  return r;
}

__device__ __forceinline__ uint8_t encode(float x, float scale, bool positive) {
  if (!finite(x)) return 0x7f;  // NaN, in its own place only
  float y = scale > 0.f ? x / scale : 0.f;
  y = fminf(fmaxf(y, -kCodeMax), kCodeMax);
  if (positive && x > 0.f && scale > 0.f) y = fmaxf(y, kCodeMin);
  return to_e4m3(y);
}

__device__ __forceinline__ float scale_of(float absmax) {
  const float s = absmax / kCodeMax;
  return s < kScaleMin ? 0.f : s;
}

// The tensor of this workgroup: one comparison a lane (the table holds fewer
// tensors than a wave has lanes).
static_assert(kAdamMaxTensors <= 64, "a lane per tensor");
__device__ __forceinline__ int tensor_of(const AdamLaunch& a) {
  const int l = threadIdx.x & 63;
  const bool after = l > 0 && l < a.count && blockIdx.x >= a.first[l];
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(after)));
}

__global__ __launch_bounds__(NT) void adamw_kernel(AdamLaunch a) {
  __shared__ float red[NT / 64];
  const int k = tensor_of(a);
  const AdamTensor t = a.t[k];
  const Scalars s = scalars(a);
  if (!finite(s.gscale)) return;  // the whole step is left out
  const float keep = a.lr_dev ? 1.f - s.lr * t.decay : t.decay;
  const int64_t begin = (int64_t)(blockIdx.x - a.first[k]) * kAdamTile;
  for (int64_t i0 = begin; i0 < begin + kAdamTile && i0 < t.n; i0 += NT) {
    const int64_t i = i0 + threadIdx.x;
    const bool in = i < t.n;
    Updated u{0.f, 0.f, 0.f, 0.f};
    if (in) {
      const float p = t.master ? t.master[i] : load(t.param, i, t.param_bf16);
      const float g = load(t.grad, i, t.grad_bf16);
      float m, v;
      if (t.bits8) {
        const int64_t b = i / kAdamBlock;
        const float r = from_e4m3(((const uint8_t*)t.v)[i]) * t.vs[b];
        m = from_e4m3(((const uint8_t*)t.m)[i]) * t.ms[b];
        v = r * r;
      } else {
        m = ((const float*)t.m)[i];
        v = ((const float*)t.v)[i];
      }
      u = update(p, g, m, v, keep, s);
      if (t.master) t.master[i] = u.p;
      if (t.param_bf16)
        ((__bf16*)t.param)[i] = (__bf16)u.p;
      else
        ((float*)t.param)[i] = u.p;
      if (!t.bits8) {
        ((float*)t.m)[i] = u.m;
        ((float*)t.v)[i] = u.v;
      }
    }
    if (t.bits8) {  // uniform: one block of 256 elements
      const float sm = scale_of(block_absmax(u.m, red)), sr = scale_of(block_absmax(u.r, red));
      if (in) {
        ((uint8_t*)t.m)[i] = encode(u.m, sm, false);
        ((uint8_t*)t.v)[i] = encode(u.r, sr, true);
      }
      if (threadIdx.x == 0) {
        t.ms[i0 / kAdamBlock] = sm;
        t.vs[i0 / kAdamBlock] = sr;
      }
    }
  }
}

}  // namespace

hipError_t launch_adamw(const AdamLaunch& a, hipStream_t st) {
  adamw_kernel<<<a.first[a.count], NT, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace plp
