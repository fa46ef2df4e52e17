// Layer norm (and its form without the mean) over rows of H, forward and
// backward, bf16 or fp32, statistics and sums in fp32.
//
//   forward   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) rstd w + b                       (rms: mu = 0)
//   backward  xh = (x - mu) rstd, c = dy w,
//             dx = rstd (c - mean(c) - xh mean(c xh))       (rms: no mean(c))
//             dw = sum over rows of dy xh, db = sum over rows of dy
//
// The deviations are taken from the mean in a second pass over the row, so a
// mean that is large beside them costs no precision.
#include "ops.h"

#include <algorithm>

namespace plp {

namespace {

constexpr int NT = 256;

template <typename T>
__device__ __forceinline__ float ldf(const T* p, int64_t i) {
  return (float)p[i];
}

// Sum over the block's NT threads in a fixed order.
__device__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const float r = (red[0] + red[1]) + (red[2] + red[3]);
  __syncthreads();
  return r;
}

// Any H and alignment: one workgroup a row, the row read again for each pass.
template <typename T>
__global__ __launch_bounds__(NT) void norm_fwd_any_kernel(NormFwd a) {
  __shared__ float red[NT / 64];
  const int H = a.H;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const T* x = (const T*)a.x + row * H;
    float mu = 0.f;
    if (!a.rms) {
      float s = 0.f;
      for (int d = threadIdx.x; d < H; d += NT) s += ldf(x, d);
      mu = block_sum(s, red) / (float)H;
    }
    float q = 0.f;
    for (int d = threadIdx.x; d < H; d += NT) {
      const float e = ldf(x, d) - mu;
      q += e * e;
    }
    const float rstd = 1.f / sqrtf(block_sum(q, red) / (float)H + a.eps);
    T* y = (T*)a.y + row * H;
    for (int d = threadIdx.x; d < H; d += NT)
      y[d] = (T)((ldf(x, d) - mu) * rstd * ldf((const T*)a.w, d) + (a.b ? ldf((const T*)a.b, d) : 0.f));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(NT) void norm_bwd_x_any_kernel(NormBwd a) {
  __shared__ float red[NT / 64];
  const int H = a.H;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const T *x = (const T*)a.x + row * H, *gy = (const T*)a.gy + row * H;
    const float mu = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
    float s = 0.f, q = 0.f;
    for (int d = threadIdx.x; d < H; d += NT) {
      const float c = ldf(gy, d) * ldf((const T*)a.w, d);
      s += c;
      q += c * ((ldf(x, d) - mu) * rstd);
    }
    const float mc = a.rms ? 0.f : block_sum(s, red) / (float)H;
    const float mq = block_sum(q, red) / (float)H;
    T* gx = (T*)a.gx + row * H;
    for (int d = threadIdx.x; d < H; d += NT) {
      const float c = ldf(gy, d) * ldf((const T*)a.w, d), xh = (ldf(x, d) - mu) * rstd;
      gx[d] = (T)(rstd * (c - mc - xh * mq));
    }
  }
}

// Partial sums of dw and db: thread per column, one row group per blockIdx.y.
template <typename T>
__global__ __launch_bounds__(NT) void norm_bwd_w_any_kernel(NormBwd a, int groups) {
  const int d = blockIdx.x * NT + threadIdx.x;
  if (d >= a.H) return;
  const int H = a.H;
  const int64_t per = (a.N + groups - 1) / groups;
  const int64_t r0 = (int64_t)blockIdx.y * per, r1 = min(a.N, r0 + per);
  float gw = 0.f, gb = 0.f;
  for (int64_t row = r0; row < r1; ++row) {
    const float gy = ldf((const T*)a.gy, row * H + d);
    const float mu = a.rms ? 0.f : a.mean[row];
    gw += gy * ((ldf((const T*)a.x, row * H + d) - mu) * a.rstd[row]);
    gb += gy;
  }
  a.part[(int64_t)blockIdx.y * H + d] = gw;
  a.part[((int64_t)groups + blockIdx.y) * H + d] = gb;
}

// dw and db: the groups' partial sums added in a fixed order, 64 columns a
// workgroup, four groups of partials at a time.
template <typename T>
__global__ __launch_bounds__(NT) void norm_bwd_reduce_kernel(const float* part, int groups, int H, T* gw, T* gb) {
  __shared__ float red[NT];
  const int d = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6;
  T* out = blockIdx.y ? gb : gw;
  if (!out) return;
  const float* p = part + (int64_t)blockIdx.y * groups * H;
  float s = 0.f;
  if (d < H)
    for (int g = k; g < groups; g += 4) s += p[(int64_t)g * H + d];
  red[threadIdx.x] = s;
  __syncthreads();
  if (k == 0 && d < H)
    out[d] = (T)((red[threadIdx.x] + red[64 + threadIdx.x]) + (red[128 + threadIdx.x] + red[192 + threadIdx.x]));
}

}  // namespace

int norm_bwd_groups(int64_t N, int H) { return (int)std::max<int64_t>(1, std::min<int64_t>(256, (N + 15) / 16)); }

namespace {

template <typename T>
hipError_t norm_fwd(const NormFwd& a, hipStream_t st) {
  norm_fwd_any_kernel<T><<<(unsigned)std::min<int64_t>(a.N, 65536), NT, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd(const NormBwd& a, hipStream_t st) {
  if (a.gx && a.N > 0) {
    norm_bwd_x_any_kernel<T><<<(unsigned)std::min<int64_t>(a.N, 65536), NT, 0, st>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.gw || a.gb) {
    const int groups = norm_bwd_groups(a.N, a.H);
    norm_bwd_w_any_kernel<T><<<dim3((a.H + NT - 1) / NT, groups), NT, 0, st>>>(a, groups);
    if (hipError_t e = hipGetLastError()) return e;
    norm_bwd_reduce_kernel<T><<<dim3((a.H + 63) / 64, 2), NT, 0, st>>>(a.part, groups, a.H, (T*)a.gw, (T*)a.gb);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwd& a, hipStream_t st) {
  return a.dtype == 0 ? norm_fwd<float>(a, st) : norm_fwd<__bf16>(a, st);
}

hipError_t launch_norm_bwd(const NormBwd& a, hipStream_t st) {
  return a.dtype == 0 ? norm_bwd<float>(a, st) : norm_bwd<__bf16>(a, st);
}

}  // namespace plp
