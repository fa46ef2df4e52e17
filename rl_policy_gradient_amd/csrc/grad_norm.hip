// The global norm of a list of gradients and the factor that clips them:
//
//   norm = |s| sqrt(sum over all tensors of g^2),
//   scale = s min(1, max_norm / (norm + eps))         (NaN if norm is not finite)
//
// with s a given factor (1 without one), and the pass that applies a scale.
//
// Squares are formed and added in fp64: a square of an fp32 or bf16 value is
// exact there (24 + 24 bits of 53) and neither over- nor underflows, so a norm
// is good to half a step of fp32 whatever the gradients' size. Two launches: a
// workgroup a tile (each tensor's last may be short, an empty one's is empty: at
// most 4096 and the list's length in all) leaves the tile's sum, then one
// workgroup adds the tiles' sums in a fixed order, and others those of a tensor
// each, where asked for. A short list takes one launch of one workgroup.
//
// Bound by HBM: 145 tensors of 367 million bf16 elements take 126 us (5.8 TB/s,
// two operations in fp64 an element are 20 us of that at their rate) and 4 to
// finish; 27 million, which the caches after the L2 hold, 12.4 (4.4 TB/s) and 4,
// and their clipping in place 18.6 (5.8 TB/s, read and written). Finishing took
// 10 where a wave added up a tensor, the head's 2000 tiles among them.
#include "training_ops.h"

#include <math.h>

namespace plp {

namespace {

constexpr int NT = 256;

template <typename T>
constexpr int vec_of = 16 / (int)sizeof(T);
// 16 bytes of T at any element's address.
template <typename T>
struct Vec {
  typedef T type __attribute__((ext_vector_type(vec_of<T>), aligned(sizeof(T))));
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The entry that workgroup b belongs to: the last that begins at or before it.
__device__ __forceinline__ int entry_of(const GradLaunch& a, uint32_t b) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < (kGradMaxTensors + 63) / 64; ++i) {
    const uint32_t e = i * 64 + (threadIdx.x & 63);
    n += __popcll(__ballot(e < a.count && a.t[e < a.count ? e : 0].first <= b));
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// A workgroup's tile: elements [begin, begin + n) of entry e.
struct Tile {
  int e;
  bool bf16;
  int64_t begin, n;
};
__device__ __forceinline__ Tile tile_of(const GradLaunch& a, uint32_t b) {
  Tile t;
  t.e = entry_of(a, b);
  const uint32_t first = a.t[t.e].first, tb = a.t[t.e].tail_bf16;
  const uint32_t next = t.e + 1 < (int)a.count ? a.t[t.e + 1].first : a.groups;
  t.bf16 = tb & 1;
  t.begin = (int64_t)(b - first) << a.tile_shift;
  t.n = b + 1 == next ? (int64_t)(tb >> 1) : (int64_t)1 << a.tile_shift;
  return t;
}

// The squares of n elements that thread `thread` of `threads` takes, `deep`
// loads of it in flight.
template <int deep, typename T>
__device__ __forceinline__ double squares(const T* p, int64_t n, int thread, int threads) {
  typedef typename Vec<T>::type TV;
  constexpr int V = vec_of<T>;
  const int64_t step = (int64_t)threads * V;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const auto add = [&](const TV& x) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const double g = (double)(float)x[k];
      s[k % 4] = fma(g, g, s[k % 4]);
    }
  };
  int64_t i = (int64_t)thread * V;
  for (; i + (deep - 1) * step + V <= n; i += deep * step) {
    TV x[deep];
#pragma unroll
    for (int c = 0; c < deep; ++c) x[c] = *reinterpret_cast<const TV*>(p + i + c * step);
#pragma unroll
    for (int c = 0; c < deep; ++c) add(x[c]);
  }
  for (; i + V <= n; i += step) add(*reinterpret_cast<const TV*>(p + i));
  for (; i < n; ++i) {  // fewer than V, of one thread
    const double g = (double)(float)p[i];
    s[0] = fma(g, g, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}
template <int deep>
__device__ __forceinline__ double squares_of(const GradLaunch& a, const Tile& t, int thread, int threads) {
  return t.bf16 ? squares<deep>((const __bf16*)a.t[t.e].p + t.begin, t.n, thread, threads)
                : squares<deep>((const float*)a.t[t.e].p + t.begin, t.n, thread, threads);
}

__global__ __launch_bounds__(NT) void grad_squares_kernel(const GradLaunch a, double* __restrict__ part,
                                                          uint32_t* __restrict__ start) {
  __shared__ double red[NT / 64];
  const uint32_t b = blockIdx.x;
  const Tile t = tile_of(a, b);
  const double s = wave_sum(squares_of<4>(a, t, threadIdx.x, NT));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    part[a.first_tile + b] = (red[0] + red[1]) + (red[2] + red[3]);
    if (t.begin == 0) start[a.first_tensor + t.e] = a.first_tile + b;
  }
}

// The norm of a sum of squares, and the factor that goes with it.
__device__ __forceinline__ void say_norm(const GradFinish& a, double given, double sum) {
  const double norm = fabs(given) * sqrt(sum);
  const float n32 = (float)norm;
  a.norm[0] = n32;
  a.scale[0] = fabsf(n32) < INFINITY ? (float)(given * fmin(1.0, a.max_norm / (norm + a.eps))) : NAN;
}

// Workgroup 0 the whole norm, the others a tensor's each.
__global__ __launch_bounds__(NT) void grad_finish_kernel(const GradFinish a) {
  __shared__ double red[NT / 64];
  const double given = a.grad_scale ? (double)*a.grad_scale : 1.0;
  const uint32_t i = blockIdx.x - 1;  // not of workgroup 0
  uint32_t from = 0, to = a.tiles;
  if (blockIdx.x > 0) {
    from = a.start[i];
    if (i + 1 < a.count) to = a.start[i + 1];
  }
  double s = 0.0;
#pragma unroll 8
  for (uint32_t k = from + threadIdx.x; k < to; k += NT) s += a.part[k];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x > 0) return;
  s = (red[0] + red[1]) + (red[2] + red[3]);
  if (blockIdx.x > 0)
    a.norms[i] = (float)(fabs(given) * sqrt(s));
  else
    say_norm(a, given, s);
}

// A short list at once: one workgroup, a wave a tile at a time (a dozen tensors
// of 98 000 fp32 elements: 6.8 us).
constexpr int kSmallThreads = 1024;
__global__ __launch_bounds__(kSmallThreads) void grad_small_kernel(const GradLaunch a, const GradFinish f) {
  __shared__ double part[kGradSmallTiles];
  __shared__ uint32_t start[kGradMaxTensors + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t b = wave; b < a.groups; b += kSmallThreads / 64) {
    const Tile t = tile_of(a, b);
    const double s = wave_sum(squares_of<8>(a, t, lane, 64));
    if (lane == 0) {
      part[b] = s;
      if (t.begin == 0) start[t.e] = b;
    }
  }
  if (threadIdx.x == 0) start[a.count] = a.groups;
  __syncthreads();
  const double given = f.grad_scale ? (double)*f.grad_scale : 1.0;
  if (f.norms && threadIdx.x < a.count) {
    double s = 0.0;
    for (uint32_t k = start[threadIdx.x]; k < start[threadIdx.x + 1]; ++k) s += part[k];
    f.norms[threadIdx.x] = (float)(fabs(given) * sqrt(s));
  }
  if (wave == kSmallThreads / 64 - 1) {
    double s = 0.0;
    for (uint32_t k = lane; k < a.groups; k += 64) s += part[k];
    s = wave_sum(s);
    if (lane == 0) say_norm(f, given, s);
  }
}

template <typename T>
__device__ __forceinline__ void clip(T* p, int64_t n, float f) {
  typedef typename Vec<T>::type TV;
  constexpr int V = vec_of<T>;
  constexpr int64_t step = (int64_t)NT * V;
  const auto scaled = [&](TV x) {
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = (T)((float)x[k] * f);
    return x;
  };
  int64_t i = (int64_t)threadIdx.x * V;
  for (; i + 3 * step + V <= n; i += 4 * step) {
    TV x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const TV*>(p + i + c * step);
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<TV*>(p + i + c * step) = scaled(x[c]);
  }
  for (; i + V <= n; i += step) *reinterpret_cast<TV*>(p + i) = scaled(*reinterpret_cast<const TV*>(p + i));
  for (; i < n; ++i) p[i] = (T)((float)p[i] * f);
}

__global__ __launch_bounds__(NT) void grad_clip_kernel(const GradLaunch a, const float* __restrict__ scale) {
  const float f = *scale;
  if (f == 1.f || !(fabsf(f) < INFINITY)) return;
  const Tile t = tile_of(a, blockIdx.x);
  if (t.bf16)
    clip((__bf16*)a.t[t.e].p + t.begin, t.n, f);
  else
    clip((float*)a.t[t.e].p + t.begin, t.n, f);
}

}  // namespace

hipError_t launch_grad_squares(const GradLaunch& a, double* part, uint32_t* start, hipStream_t st) {
  grad_squares_kernel<<<a.groups, NT, 0, st>>>(a, part, start);
  return hipGetLastError();
}

hipError_t launch_grad_finish(const GradFinish& a, hipStream_t st) {
  grad_finish_kernel<<<1 + (a.norms ? a.count : 0), NT, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_small(const GradLaunch& a, const GradFinish& f, hipStream_t st) {
  grad_small_kernel<<<1, kSmallThreads, 0, st>>>(a, f);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradLaunch& a, const float* scale, hipStream_t st) {
  grad_clip_kernel<<<a.groups, NT, 0, st>>>(a, scale);
  return hipGetLastError();
}

}  // namespace plp
