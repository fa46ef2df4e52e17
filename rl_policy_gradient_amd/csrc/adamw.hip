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
// Codes are 6 to 12 % apart. A moment of which a step changes less than half
// of that would go back to where it was at every step if it were rounded to
// the nearest code: at b2 = 0.999 the roots of elements whose gradients fall
// to 0.03 of their blocks' others stay 14 times too large (5999 steps, mean),
// at 0.99 13 times (599). With b above kNearestBeta a moment is therefore
// rounded up or down, up as often as its distance from the lower code asks
// for: at step t, where that share of the spacing and the fraction of
// t golden + (a constant of the element's place in its block) reach one
// together. No random numbers, no state, and the mean over the steps is the
// value's own; the same roots come to 0.98 of the fp32 ones in the mean, 5 to
// 95 % of them to 0.59 to 1.57 (0.999) and 0.62 to 1.49 (0.99). Up to
// kNearestBeta a gradient's own noise carries a moment over the half codes
// and the nearest code is the better one: root mean square error 0.076
// against 0.089 at b2 = 0.95 (3000 steps), 0.060 against 0.067 of m at b1 =
// 0.9, 0.084 against 0.090 at 0.95. It is late after a fall: at 0.95 by 80
// steps or so, at 0.97 the roots are still 3.3 times too large after 199.
// (Measured: 151936 x 896 bf16, 399 us with the nearest codes, 417 with these.)
//
// Every element is read once and written once; nothing is reused, so the
// step is bound by HBM: at 151936 x 896 bf16 with a master copy 384 to 413 us
// with 8-bit states (16 bytes an element, 5.3 to 5.7 TB/s; 363 to 488 under
// the profiler) and 705 to 720 us with fp32 ones (28 bytes, 5.3 to 5.4 TB/s),
// where a plain copy of 2.2 GB takes 422 us. 145 tensors of a small model (27
// million elements, 8-bit states) take 97 to 101 us in three launches; a copy
// of their 435 MB 84.
#include "ops.h"

#include <math.h>

namespace plp {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int NT = 256;
constexpr float kCodeMax = 448.f;      // largest e4m3 value
constexpr float kCodeMin = 0x1p-9f;    // smallest above zero
constexpr float kNormalMin = 0x1p-6f;  // codes below it are kCodeMin apart
constexpr float kScaleMin = 0x1p-126f; // a smaller scale's inverse would overflow
constexpr float kNearestBeta = 0.95f;  // a moment with a larger beta is not rounded to the nearest code

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The scalars of one step.
struct Scalars {
  float b1, c1, b2, c2, eps, step_size, inv_root, gscale, lr;
  uint32_t t;  // the step's number
};

// With the step or the rate in device memory the corrections are formed here,
// in fp64 (1 - b^t as -expm1(t ln b), which does not cancel for small t).
__device__ Scalars scalars(const AdamLaunch& a) {
  const int64_t t = a.step_dev ? (*a.step_dev < 1 ? 1 : *a.step_dev) : a.step;
  Scalars s{a.b1, a.c1, a.b2, a.c2, a.eps, a.step_size, a.inv_root, 1.f, (float)a.lr, (uint32_t)t};
  if (a.step_dev || a.lr_dev) {
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
// decay: lr wd, which meets the parameter in the step's own subtraction; a
// factor 1 - lr wd in fp32 has steps of 2^-24, so that a rate of 1e-6 would
// decay 19 % too much at wd 0.1 and nothing at 0.01. (An infinite parameter
// stays what it is.)
__device__ __forceinline__ Updated update(float p, float g, float m, float v, float decay, const Scalars& s) {
#pragma clang fp contract(off)
  g = g * s.gscale;
  Updated u;
  u.m = m * s.b1 + g * s.c1;
  u.v = v * s.b2 + g * g * s.c2;
  u.r = sqrtf(u.v);
  u.p = p - ((finite(p) ? p * decay : 0.f) + u.m / (u.r * s.inv_root + s.eps) * s.step_size);
  return u;
}

// Four consecutive elements i .. i+3 of an array of n, those at or past n as
// 0. One load or store whatever the array's alignment: global memory asks
// only for that of the elements.
template <typename T>
struct Four;
template <>
struct Four<float> {
  typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Four<__bf16> {
  typedef __bf16 raw __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Four<uint8_t> {
  typedef uint8_t raw __attribute__((ext_vector_type(4), aligned(1)));
};
template <typename T>
__device__ __forceinline__ typename Four<T>::raw load4(const T* p, int64_t i, int64_t n) {
  typedef typename Four<T>::raw raw;
  if (i + 4 <= n) return *reinterpret_cast<const raw*>(p + i);
  raw x = {};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (i + k < n) x[k] = p[i + k];
  return x;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t i, int64_t n, typename Four<T>::raw x) {
  if (i + 4 <= n) {
    *reinterpret_cast<typename Four<T>::raw*>(p + i) = x;
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (i + k < n) p[i + k] = x[k];
}
template <typename T>
__device__ __forceinline__ f32x4 load4f(const T* p, int64_t i, int64_t n) {
  return __builtin_convertvector(load4(p, i, n), f32x4);
}
template <typename T>
__device__ __forceinline__ void store4f(T* p, int64_t i, int64_t n, f32x4 x) {
  typename Four<T>::raw y;
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = (T)x[k];
  store4(p, i, n, y);
}
__device__ __forceinline__ uint32_t load_codes(const void* p, int64_t i, int64_t n) {
  return __builtin_bit_cast(uint32_t, load4((const uint8_t*)p, i, n));
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t n, uint32_t c) {
  store4((uint8_t*)p, i, n, __builtin_bit_cast(Four<uint8_t>::raw, c));
}

__device__ __forceinline__ f32x4 from_e4m3(uint32_t c) {
  return f32x4{__builtin_amdgcn_cvt_f32_fp8(c, 0), __builtin_amdgcn_cvt_f32_fp8(c, 1),
               __builtin_amdgcn_cvt_f32_fp8(c, 2), __builtin_amdgcn_cvt_f32_fp8(c, 3)};
}

// Largest of 64 lanes' values, none negative, in every lane: within quads,
// half rows and rows of 16 by lane permutations, then across the rows.
__device__ __forceinline__ float wave_max(float v) {
#define PLP_DPP_MAX(ctrl, rows) \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false)))
  PLP_DPP_MAX(0xb1, 0xf);   // lanes 1 0 3 2 of each quad
  PLP_DPP_MAX(0x4e, 0xf);   // lanes 2 3 0 1
  PLP_DPP_MAX(0x141, 0xf);  // mirrored in each half row
  PLP_DPP_MAX(0x140, 0xf);  // mirrored in each row
  PLP_DPP_MAX(0x142, 0xa);  // the row before into rows 1 and 3
  PLP_DPP_MAX(0x143, 0xc);  // row 1 into rows 2 and 3
#undef PLP_DPP_MAX
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float finite_max(f32x4 x) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = fmaxf(m, finite(x[k]) ? fabsf(x[k]) : 0.f);
  return m;
}

// The block's scale and its reciprocal (both 0 for a block whose largest value
// is too small for a scale).
struct Scale {
  float s, inv;
  // x / s, correctly rounded: the reciprocal is, so one residual step makes
  // the quotient so too (Markstein 1990). Three operations instead of a
  // division's eleven, and the same code for a value at a tie however the
  // quotient is formed.
  __device__ __forceinline__ float divide(float x) const {
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
  }
};
__device__ __forceinline__ Scale scale_of(float absmax) {
  const float s = absmax * (1.f / kCodeMax);
  return s < kScaleMin ? Scale{0.f, 0.f} : Scale{s, 1.f / s};
}

// One of the two e4m3 values around y, |y| at most the largest of them, the
// one further from zero if y's distance from the other and phase / 2^20 of
// their spacing together reach it: a code has three of a float's 23 fraction
// bits, so the phase is added below them. (Below kNormalMin the codes are
// spaced as above it, and y is moved there and back.)
__device__ __forceinline__ float either_code(float y, uint32_t phase) {
  const float a = fabsf(y), lift = a < kNormalMin ? kNormalMin : 0.f;
  const uint32_t z = (__float_as_uint(a + lift) + phase) & ~0xfffffu;
  return copysignf(__uint_as_float(z) - lift, y);
}

// Step t's phase of the lane's first element, of 2^32: a turn of the golden
// ratio a step, and a start of each element's own.
constexpr uint32_t kPhaseStep = 0x9e3779b9u, kPhaseElement = 0x85ebca6bu;
__device__ __forceinline__ uint32_t phase_of(uint32_t t) {
  return t * kPhaseStep + (threadIdx.x & 63) * 4 * kPhaseElement;
}

// Four codes: the nearest e4m3 values (ties to even, as the hardware rounds),
// or with `either` those of either_code. What is not finite becomes NaN in
// its own place only.
__device__ __forceinline__ uint32_t encode(f32x4 x, Scale sc, bool positive, bool either, uint32_t phase) {
  f32x4 y;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    y[k] = fminf(fmaxf(sc.divide(x[k]), -kCodeMax), kCodeMax);
    if (either) y[k] = either_code(y[k], (phase + k * kPhaseElement) >> 12);  // uniform
    if (positive && x[k] > 0.f && sc.inv > 0.f) y[k] = fmaxf(y[k], kCodeMin);
  }
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (!finite(x[k])) c = (c & ~(0xff << 8 * k)) | (0x7f << 8 * k);
  return (uint32_t)c;
}

// A workgroup's tile: a block of 256 elements a wave, four a lane, so that a
// scale's maximum never leaves the wave. One block a wave and nothing
// unrolled: with 38 registers eight waves run on a SIMD, and it is their
// number that keeps the bytes in flight. At 151936 x 896 bf16 with 8-bit
// states, 390 to 400 us; with two blocks a wave (65 registers) 465 us, with
// four (113) 475 us; with fp32 states 694, 709 and 710 us.
static_assert(kAdamBlock == 4 * 64 && kAdamTile == 4 * NT, "one block of a scale a wave, one tile a workgroup");

template <typename P, typename G, bool MASTER, bool BITS8>
__device__ __forceinline__ void tile(const AdamTensor& t, const Scalars& s, float decay, int64_t begin) {
  const int64_t n = t.n, i = begin + threadIdx.x * 4, b = i / kAdamBlock;
  f32x4 p, g, m, v, r;
  if (MASTER)
    p = load4f((const float*)t.master, i, n);
  else
    p = load4f((const P*)t.param, i, n);
  g = load4f((const G*)t.grad, i, n);
  if (BITS8) {
    const uint32_t mc = load_codes(t.m, i, n), vc = load_codes(t.v, i, n);
    const float ms = i < n ? t.ms[b] : 0.f, vs = i < n ? t.vs[b] : 0.f;
    m = from_e4m3(mc) * ms;
    r = from_e4m3(vc) * vs;
    v = r * r;
  } else {
    m = load4f((const float*)t.m, i, n);
    v = load4f((const float*)t.v, i, n);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const Updated x = update(p[k], g[k], m[k], v[k], decay, s);
    p[k] = x.p;
    m[k] = x.m;
    v[k] = x.v;
    r[k] = x.r;
  }
  if (MASTER) store4f(t.master, i, n, p);
  store4f((P*)t.param, i, n, p);
  if (BITS8) {  // elements past the end are all zero and do not count
    const Scale sm = scale_of(wave_max(finite_max(m))), sr = scale_of(wave_max(finite_max(r)));
    const uint32_t phase = phase_of(s.t);
    store_codes(t.m, i, n, encode(m, sm, false, s.b1 > kNearestBeta, phase + 0x80000000u));  // half a turn from r's
    store_codes(t.v, i, n, encode(r, sr, true, s.b2 > kNearestBeta, phase));
    if ((threadIdx.x & 63) == 0 && i < n) {
      t.ms[b] = sm.s;
      t.vs[b] = sr.s;
    }
  } else {
    store4f((float*)t.m, i, n, m);
    store4f((float*)t.v, i, n, v);
  }
}

template <typename P, bool MASTER>
__device__ __forceinline__ void tile(const AdamTensor& t, const Scalars& s, float decay, int64_t begin) {
  if (t.grad_bf16) {
    if (t.bits8)
      tile<P, __bf16, MASTER, true>(t, s, decay, begin);
    else
      tile<P, __bf16, MASTER, false>(t, s, decay, begin);
  } else {
    if (t.bits8)
      tile<P, float, MASTER, true>(t, s, decay, begin);
    else
      tile<P, float, MASTER, false>(t, s, decay, begin);
  }
}

// The tensor of this workgroup: one comparison a lane (the table holds fewer
// tensors than a wave has lanes).
static_assert(kAdamMaxTensors <= 64, "a lane per tensor");
__device__ __forceinline__ int tensor_of(const AdamLaunch& a) {
  const int l = threadIdx.x & 63;
  const bool after = l > 0 && l < a.count && blockIdx.x >= a.first[l];
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(after)));
}

__global__ __launch_bounds__(NT) void adamw_kernel(AdamLaunch) {
  // the arguments where they lie, in constant memory: an index that varies by
  // workgroup into a by-value argument makes the compiler copy all of it to
  // scratch memory first (measured: the step eight times slower)
  const AdamLaunch& a = *(const AdamLaunch*)(const __attribute__((address_space(4))) AdamLaunch*)
                            __builtin_amdgcn_kernarg_segment_ptr();
  const int k = tensor_of(a);
  const AdamTensor t = a.t[k];
  const Scalars s = scalars(a);
  if (!finite(s.gscale)) return;  // the whole step is left out
  const float decay = a.lr_dev ? s.lr * t.decay : t.decay;
  const int64_t begin = (int64_t)(blockIdx.x - a.first[k]) * kAdamTile;
  if (!t.param_bf16)
    tile<float, false>(t, s, decay, begin);
  else if (t.master)
    tile<__bf16, true>(t, s, decay, begin);
  else
    tile<__bf16, false>(t, s, decay, begin);
}

}  // namespace

hipError_t launch_adamw(const AdamLaunch& a, hipStream_t st) {
  adamw_kernel<<<a.first[a.count], NT, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace plp
