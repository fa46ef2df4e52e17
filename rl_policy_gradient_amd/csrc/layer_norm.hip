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
//
// Bound by HBM: x is read once and y written once forward; x and dy are read
// and dx written once backward, dw and db adding their partial rows. Measured:
// forward of 65536 x 896 bf16 36 to 41 us (5.7 to 6.5 TB/s, cached in part; a
// copy of as many bytes 33), of 16384 x 4096 fp32 101 us (5.3 TB/s); backward
// of 16384 x 4096 fp32 150 to 154 us (5.2 to 5.4 TB/s; a copy of as many bytes
// 163), of 65536 x 896 bf16 72 us (4.9 TB/s), of 512 x 896 bf16 8 us, two
// launches of 5 and 3. Rows that are no whole number of 16 bytes cost a third
// more or worse: 65536 x 897 bf16 47 and 100 us, backward of 16384 x 4099 fp32
// 249; the widest of them (640 lanes and more) spill registers backward: 8192
// x 12001 bf16 285 us, 4096 x 16383 153 where 16384 takes 92.
#include "ops.h"

#include <algorithm>
#include <type_traits>

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

// ---------------------------------------------------------------------------
// Rows of up to 16384: the row stays in registers, 16 elements a lane, and
// LPR lanes share a row: 8 .. 128, powers of two, in a workgroup of 256 that
// takes 256 / LPR rows at a time, or a workgroup of 192 .. 1024 a row (the
// least that hold it), so that no row leaves many lanes idle. A lane loads 16
// bytes at a time, whatever the row's alignment (global loads and stores need
// only that of their elements); the row's last few elements are the end of its
// last 16 bytes, and are stored 8, 4 and 2 bytes at a time (65536 x 897 bf16:
// 47 us forward and 101 backward, where an element at a time took 96 and 449).
// ---------------------------------------------------------------------------
constexpr int kPerLane = 16;
constexpr int kMaxLanes = 1024;

// Sum over the LPR lanes of a row (aligned groups of lanes), in every one of
// them, in a fixed order: lane permutations up to 16 lanes, exchanges up to a
// wave, then the waves' sums through LDS (`red`: a float per wave; all threads
// of the workgroup call).
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#define PLP_DPP_ADD(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, false))
  PLP_DPP_ADD(0xb1);   // lanes 1 0 3 2 of each quad
  PLP_DPP_ADD(0x4e);   // lanes 2 3 0 1
  PLP_DPP_ADD(0x141);  // mirrored in each half row of 16
  if constexpr (LPR >= 16) PLP_DPP_ADD(0x140);  // mirrored in each row
#undef PLP_DPP_ADD
  if constexpr (LPR >= 32) v += __shfl_xor(v, 16, 64);
  if constexpr (LPR >= 64) v += __shfl_xor(v, 32, 64);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = threadIdx.x >> 6, first = wave / W * W;
    __syncthreads();  // the sums before this have been read
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[first + w];
  }
  return v;
}

typedef unsigned __int128 Bits;
// 16 bytes of T at any element's address.
template <typename T>
constexpr int vec_of = 16 / (int)sizeof(T);
template <typename T>
struct Vec {
  typedef T type __attribute__((ext_vector_type(vec_of<T>), aligned(sizeof(T))));
};

// The 16 elements of a lane as they lie in memory: V consecutive ones, then V
// more LPR V further on. Those at or past H are 0. TAIL: H is no multiple of V.
template <typename T>
struct Raw {
  static constexpr int V = vec_of<T>, C = kPerLane / V;
  T x[kPerLane];
  template <int LPR, bool TAIL>
  __device__ __forceinline__ void load(const T* p, int lane, int H) {
    typedef typename Vec<T>::type TV;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int d = (c * LPR + lane) * V;
      TV t = {};
      if (TAIL ? d + V <= H : d < H) {
        t = *reinterpret_cast<const TV*>(p + d);
      } else if (TAIL && d < H) {
        if (H >= V) {
          const Bits b = __builtin_bit_cast(Bits, *reinterpret_cast<const TV*>(p + H - V));
          t = __builtin_bit_cast(TV, (Bits)(b >> 8 * (int)sizeof(T) * (d + V - H)));
        } else {
#pragma unroll
          for (int k = 0; k < V - 1; ++k)
            if (d + k < H) t[k] = p[d + k];
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) x[c * V + k] = t[k];
    }
  }
};
template <typename T, int LPR, bool TAIL>
__device__ __forceinline__ void load_row(const T* p, int lane, int H, float (&x)[kPerLane]) {
  Raw<T> r;
  r.template load<LPR, TAIL>(p, lane, H);
#pragma unroll
  for (int e = 0; e < kPerLane; ++e) x[e] = (float)r.x[e];
}

// Stores the low bits of b as a U and drops them.
template <typename U, typename T>
__device__ __forceinline__ T* put(T* p, Bits& b) {
  typedef U Any __attribute__((aligned(sizeof(T)), may_alias));
  *reinterpret_cast<Any*>(p) = (U)b;
  b >>= 8 * sizeof(U);
  return p + sizeof(U) / sizeof(T);
}

// V: elements a lane holds side by side, which the loads of the row's type set.
template <typename T, int V, int LPR, bool TAIL>
__device__ __forceinline__ void store_row(T* p, int lane, int H, const float (&x)[kPerLane]) {
  typedef T TV __attribute__((ext_vector_type(V), aligned(sizeof(T))));
#pragma unroll
  for (int c = 0; c < kPerLane / V; ++c) {
    const int d = (c * LPR + lane) * V;
    TV t;
#pragma unroll
    for (int k = 0; k < V; ++k) t[k] = (T)x[c * V + k];
    if (TAIL ? d + V <= H : d < H) {
      *reinterpret_cast<TV*>(p + d) = t;
    } else if (TAIL && d < H) {
      if constexpr (sizeof(TV) == sizeof(Bits)) {
        Bits b = __builtin_bit_cast(Bits, t);
        T* q = p + d;
        const int left = (H - d) * (int)sizeof(T);  // bytes; the same for every row
        if (left & 8) q = put<uint64_t>(q, b);
        if (left & 4) q = put<uint32_t>(q, b);
        if (left & 2) put<uint16_t>(q, b);
      } else {
#pragma unroll
        for (int k = 0; k < V - 1; ++k)
          if (d + k < H) p[d + k] = t[k];
      }
    }
  }
}

// Whether element e of the lane's 16 lies in the row.
template <int V, int LPR>
__device__ __forceinline__ bool inside(int e, int lane, int H) {
  return (e / V * LPR + lane) * V + e % V < H;
}

template <int LPR>
constexpr int threads_of = LPR > NT / 2 ? LPR : NT;

template <typename T, int LPR, bool TAIL>
__global__ __launch_bounds__(threads_of<LPR>) void norm_fwd_kernel(NormFwd a) {
  constexpr int slots = threads_of<LPR> / LPR, V = vec_of<T>;
  __shared__ float red[threads_of<LPR> / 64];
  const int H = a.H, lane = threadIdx.x % LPR;
  const float inv = 1.f / (float)H;
  const int64_t row = (int64_t)blockIdx.x * slots + threadIdx.x / LPR;
  const bool in = row < a.N;
  float x[kPerLane], w[kPerLane];
  load_row<T, LPR, TAIL>((const T*)a.x + (in ? row : 0) * H, lane, H, x);
  load_row<T, LPR, TAIL>((const T*)a.w, lane, H, w);
  float mu = 0.f;
  if (!a.rms) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) s += x[e];
    mu = row_sum<LPR>(s, red) * inv;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) x[e] = inside<V, LPR>(e, lane, H) ? x[e] - mu : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int e = 0; e < kPerLane; ++e) q += x[e] * x[e];
  const float rstd = 1.f / sqrtf(row_sum<LPR>(q, red) * inv + a.eps);
  if (!in) return;
#pragma unroll
  for (int e = 0; e < kPerLane; ++e) x[e] = x[e] * rstd * w[e];
  if (a.b) {
    load_row<T, LPR, TAIL>((const T*)a.b, lane, H, w);
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) x[e] += w[e];
  }
  store_row<T, V, LPR, TAIL>((T*)a.y + row * H, lane, H, x);
  if (lane == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Each workgroup takes every gridDim.x-th set of rows and adds up its part of
// dw and db in registers, then over its rows in LDS: one partial row each a
// workgroup, added up by norm_bwd_reduce_kernel. What lies past H has x, dy and
// w of 0 and adds nothing.
// (bf16 rows are half as many bytes, so it takes four waves a SIMD to keep
// enough in flight where their tail costs registers: 16384 x 4100, 128 us
// against 191; 65536 x 896 is at 72 either way.)
template <typename T, int LPR, bool TAIL>
__global__ __launch_bounds__(threads_of<LPR>, sizeof(T) == 4 ? 1 : 4) void norm_bwd_kernel(NormBwd a) {
  constexpr int slots = threads_of<LPR> / LPR, V = vec_of<T>;
  __shared__ float red[threads_of<LPR> / 64];
  __shared__ alignas(32) float sums[slots > 1 ? NT * kPerLane : 1];
  const int H = a.H, lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const float inv = 1.f / (float)H;
  float w[kPerLane], gw[kPerLane], gb[kPerLane];
  load_row<T, LPR, TAIL>((const T*)a.w, lane, H, w);
#pragma unroll
  for (int e = 0; e < kPerLane; ++e) gw[e] = gb[e] = 0.f;
  const int64_t stride = (int64_t)gridDim.x * slots;
  for (int64_t r0 = (int64_t)blockIdx.x * slots; r0 < a.N; r0 += stride) {  // uniform
    const int64_t row = r0 + slot, at = row < a.N ? row : 0;
    const int h = row < a.N ? H : 0;
    float x[kPerLane], gy[kPerLane];
    load_row<T, LPR, TAIL>((const T*)a.x + at * H, lane, h, x);
    load_row<T, LPR, TAIL>((const T*)a.gy + at * H, lane, h, gy);
    const float rstd = h ? a.rstd[at] : 0.f, mu = a.rms || !h ? 0.f : a.mean[at];
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) x[e] = (x[e] - mu) * rstd;
    // past the row's end c is 0, but (0 - mu) rstd may be infinite where no
    // element of the row's is (a row of one huge value)
    if (!(fabsf(mu * rstd) < INFINITY)) {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) x[e] = inside<V, LPR>(e, lane, H) ? x[e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const float c = gy[e] * w[e];
      s += c;
      q += c * x[e];
      gw[e] += gy[e] * x[e];
      gb[e] += gy[e];
    }
    if (!a.gx) continue;
    const float mc = a.rms ? 0.f : row_sum<LPR>(s, red) * inv;
    const float mq = row_sum<LPR>(q, red) * inv;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) x[e] = rstd * (gy[e] * w[e] - mc - x[e] * mq);
    if (row < a.N) store_row<T, V, LPR, TAIL>((T*)a.gx + row * H, lane, H, x);
  }
  if (!a.part) return;
  float* out = a.part + (int64_t)blockIdx.x * H;
#pragma unroll
  for (int k = 0; k < 2; ++k) {  // dw, then db
    if (slots == 1) {
      store_row<float, V, LPR, TAIL>(out, lane, H, k ? gb : gw);
    } else {
      __syncthreads();
      store_row<float, V, LPR, TAIL>(sums + slot * H, lane, H, k ? gb : gw);
      __syncthreads();
      for (int d = threadIdx.x; d < H; d += NT) {
        float t = 0.f;
#pragma unroll 4
        for (int i = 0; i < slots; ++i) t += sums[i * H + d];
        out[d] = t;
      }
    }
    out += (int64_t)gridDim.x * H;
  }
}

// Longer rows: one workgroup a row, the row read again for each pass.
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

// dw and db: the groups' partial sums added in a fixed order, 32 columns a
// workgroup, 32 groups of partials side by side.
constexpr int kReduceCols = 32, kReduceRows = 32;
template <typename T>
__global__ __launch_bounds__(kReduceCols* kReduceRows) void norm_bwd_reduce_kernel(const float* part, int groups, int H,
                                                                                   T* gw, T* gb) {
  __shared__ float red[kReduceRows][kReduceCols + 1];
  const int col = threadIdx.x % kReduceCols, k = threadIdx.x / kReduceCols;
  const int d = blockIdx.x * kReduceCols + col;
  T* out = blockIdx.y ? gb : gw;
  if (!out) return;
  const float* p = part + (int64_t)blockIdx.y * groups * H;
  float s = 0.f;
  if (d < H) {
#pragma unroll 8
    for (int g = k; g < groups; g += kReduceRows) s += p[(int64_t)g * H + d];
  }
  red[k][col] = s;
  __syncthreads();
  if (threadIdx.x < kReduceCols && d < H) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kReduceRows; ++i) s += red[i][col];
    out[d] = (T)s;
  }
}

// Lanes that share a row of H.
int lanes_of(int H) {
  const int need = (H + kPerLane - 1) / kPerLane;
  for (int l : {8, 16, 32, 64, 128, 192, 256, 320, 384, 512, 640, 768})
    if (l >= need) return l;
  return kMaxLanes;
}

// f(std::integral_constant<int, LPR>) for the row's lanes.
template <typename F>
hipError_t with_lanes(int H, F f) {
  switch (lanes_of(H)) {
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    case 192: return f(std::integral_constant<int, 192>());
    case 256: return f(std::integral_constant<int, 256>());
    case 320: return f(std::integral_constant<int, 320>());
    case 384: return f(std::integral_constant<int, 384>());
    case 512: return f(std::integral_constant<int, 512>());
    case 640: return f(std::integral_constant<int, 640>());
    case 768: return f(std::integral_constant<int, 768>());
    default: return f(std::integral_constant<int, kMaxLanes>());
  }
}

template <typename T>
hipError_t norm_fwd_rows(const NormFwd& a, hipStream_t st) {
  return with_lanes(a.H, [&](auto lanes) {
    constexpr int LPR = decltype(lanes)::value, slots = threads_of<LPR> / LPR;
    // a launch holds fewer than 2^32 threads
    constexpr int64_t most = ((int64_t)1 << 31) / threads_of<LPR> * slots;
    NormFwd b = a;
    for (int64_t left = a.N; left > 0; left -= most) {
      b.N = std::min(left, most);
      const unsigned grid = (unsigned)((b.N + slots - 1) / slots);
      if (a.H % vec_of<T>)
        norm_fwd_kernel<T, LPR, true><<<grid, threads_of<LPR>, 0, st>>>(b);
      else
        norm_fwd_kernel<T, LPR, false><<<grid, threads_of<LPR>, 0, st>>>(b);
      if (hipError_t e = hipGetLastError()) return e;
      b.x = (const T*)b.x + b.N * a.H;
      b.y = (T*)b.y + b.N * a.H;
      if (b.mean) b.mean += b.N;
      if (b.rstd) b.rstd += b.N;
    }
    return hipSuccess;
  });
}

template <typename T>
hipError_t norm_bwd_rows(const NormBwd& a, int groups, hipStream_t st) {
  return with_lanes(a.H, [&](auto lanes) {
    constexpr int LPR = decltype(lanes)::value;
    if (a.H % vec_of<T>)
      norm_bwd_kernel<T, LPR, true><<<groups, threads_of<LPR>, 0, st>>>(a);
    else
      norm_bwd_kernel<T, LPR, false><<<groups, threads_of<LPR>, 0, st>>>(a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t norm_fwd(const NormFwd& a, hipStream_t st) {
  if (a.H > kMaxLanes * kPerLane) {
    norm_fwd_any_kernel<T><<<(unsigned)std::min<int64_t>(a.N, 65536), NT, 0, st>>>(a);
    return hipGetLastError();
  }
  return norm_fwd_rows<T>(a, st);
}

template <typename T>
hipError_t norm_bwd(const NormBwd& a, hipStream_t st) {
  const int groups = norm_bwd_groups(a.N, a.H);
  if (a.H > kMaxLanes * kPerLane) {
    if (a.gx && a.N > 0) {
      norm_bwd_x_any_kernel<T><<<(unsigned)std::min<int64_t>(a.N, 65536), NT, 0, st>>>(a);
      if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.part) {
      norm_bwd_w_any_kernel<T><<<dim3((a.H + NT - 1) / NT, groups), NT, 0, st>>>(a, groups);
      if (hipError_t e = hipGetLastError()) return e;
    }
  } else if (a.N > 0 || a.part) {
    if (hipError_t e = norm_bwd_rows<T>(a, groups, st)) return e;
  }
  if (a.part)
    norm_bwd_reduce_kernel<T><<<dim3((a.H + kReduceCols - 1) / kReduceCols, 2), kReduceCols * kReduceRows, 0, st>>>(
        a.part, groups, a.H, (T*)a.gw, (T*)a.gb);
  return hipGetLastError();
}

}  // namespace

// More groups hide more latency, fewer leave less to add up at the end: 768
// where several rows share a workgroup, else 512 (65536 x 896 bf16: 79 us with
// 512, 72 with 768, 76 with 1024; 16384 x 4096 fp32: 155, 162 and 165 us).
// The partial sums stay below 32 MB however long the row.
int norm_bwd_groups(int64_t N, int H) {
  const int lanes = lanes_of(H), slots = lanes < NT ? NT / lanes : 1;
  const int most = std::min(slots > 1 ? 768 : 512, std::max(64, (4 << 20) / H));
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, (N + slots - 1) / slots));
}

hipError_t launch_norm_fwd(const NormFwd& a, hipStream_t st) {
  return a.dtype == 0 ? norm_fwd<float>(a, st) : norm_fwd<__bf16>(a, st);
}

hipError_t launch_norm_bwd(const NormBwd& a, hipStream_t st) {
  return a.dtype == 0 ? norm_bwd<float>(a, st) : norm_bwd<__bf16>(a, st);
}

}  // namespace plp
