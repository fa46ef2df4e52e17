// One token per row of logits, with temperature, top-k, top-p and min-p, from
// one given uniform number a row.
//
// With m the row's largest logit, w_i = exp((z_i - m) / tau) and the order
// "value descending, index ascending", each of the three limits keeps a first
// part of the order (top-p: those before which the mass, among the top-k, is
// below p times it; min-p: those with w_i >= min_p), so together they keep a
// prefix: all values above a cut value and the first few, by index, of those
// equal to it. The token is the first index at which the kept weights' running
// sum exceeds u times their sum.
//
// Every decision (which value is the cut, how many of it are kept, at which
// index the sum is exceeded) is taken on whole numbers q_i = round(w_i 2^F),
// F chosen so that they add up below 2^62: their sums are exact, so the
// result does not depend on the order of additions or on the launch's shape.
// w_i is formed in fp64 (2^x by its own polynomial, to 4e-16): at a vocabulary's
// length an fp32 weight's rounding moves the running sum across a token of
// the tail too often.
//
// Two launches: the first reads the logits once and leaves each block of 256
// its maximum and sum; the second, a workgroup a row, finds the cut and the
// token from those and from the blocks that matter.
#include "ops.h"

#include <math.h>

#include <algorithm>

namespace plp {

namespace {

constexpr int kChunk = 8;                       // consecutive logits a lane takes
constexpr int kLanes = kSampleBlock / kChunk;   // lanes of one block: 32
static_assert(kLanes == 32, "half a wave a block");

// 2^y for y <= 0 (and a little above): a polynomial of degree 10 through the
// Chebyshev points of [-1/2, 1/2] (relative error 3.2e-16) times 2^round(y).
// Below -1100 the result is 0; not for NaN.
__device__ __forceinline__ double exp2_neg(double y) {
  y = fmax(y, -1100.0);
  const double n = rint(y), f = y - n;
  double p = 0x1.e6063f7217bc6p-28;
  p = fma(p, f, 0x1.b675bca4eeebbp-24);
  p = fma(p, f, 0x1.62bfd47773353p-20);
  p = fma(p, f, 0x1.ffcb54062e698p-17);
  p = fma(p, f, 0x1.430913096fd9fp-13);
  p = fma(p, f, 0x1.5d87fe9d7a584p-10);
  p = fma(p, f, 0x1.3b2ab6fba1ddap-7);
  p = fma(p, f, 0x1.c6b08d703ce49p-5);
  p = fma(p, f, 0x1.ebfbdff82c598p-3);
  p = fma(p, f, 0x1.62e42fefa3a19p-1);
  p = fma(p, f, 1.0);
  return ldexp(p, (int)n);
}

// Monotone whole-number keys of the logits (no NaN): -inf is the least that
// occurs. bf16 logits need 16 bits, fp32 ones 32.
template <typename T>
struct Key;
template <>
struct Key<float> {
  static constexpr int bits = 32;
  __device__ static uint32_t of(float z) {
    const uint32_t b = __float_as_uint(z);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  }
  __device__ static float value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  }
};
template <>
struct Key<__bf16> {
  static constexpr int bits = 16;
  __device__ static uint32_t of(float z) { return Key<float>::of(z) >> 16; }
  __device__ static float value(uint32_t k) {
    return Key<float>::value(k & 0x8000u ? k << 16 : (k << 16) | 0xffffu);
  }
};

// Row `row` of the logits as chunks of 8 that begin at multiples of 16 bytes
// of the address: chunk c holds the elements 8c - lead .. 8c - lead + 7 of the
// row, those outside [0, V) as -inf. (A bf16 chunk is one 16-byte load, an
// fp32 one two.) -0 becomes +0, which it ties with.
template <typename T>
struct Row {
  const T* p;
  int V, lead;
  __device__ Row(const SampleArgs& a, int64_t row) : p((const T*)a.logits + row * a.stride), V(a.V) {
    constexpr int per16 = 16 / sizeof(T);
    lead = (int)(((uintptr_t)p / sizeof(T)) % per16);
  }
  __device__ int chunks() const { return (V + lead + kChunk - 1) / kChunk; }
  __device__ int blocks() const { return (V + lead + kSampleBlock - 1) / kSampleBlock; }
  __device__ int first(int c) const { return c * kChunk - lead; }
  __device__ void load(int c, float (&z)[kChunk]) const {
    const int e0 = first(c);
    if (e0 >= 0 && e0 + kChunk <= V) {
      if constexpr (sizeof(T) == 4) {
        const float4 u = *(const float4*)(p + e0), v = *(const float4*)(p + e0 + 4);
        z[0] = u.x, z[1] = u.y, z[2] = u.z, z[3] = u.w, z[4] = v.x, z[5] = v.y, z[6] = v.z, z[7] = v.w;
      } else {
        const uint4 u = *(const uint4*)(p + e0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[2 * k] = __uint_as_float(w[k] << 16);
          z[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) z[k] = e0 + k >= 0 && e0 + k < V ? (float)p[e0 + k] : -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kChunk; ++k) z[k] += 0.f;
  }
};

__device__ __forceinline__ float temperature_of(const SampleArgs& a, int64_t row) {
  return a.tau_rows ? a.tau_rows[row] : a.tau;
}
// log2(e) / tau; 1 for the greedy row, whose weights are not used.
__device__ __forceinline__ double rate_of(float tau) { return tau == 0.f ? 1.0 : 1.4426950408889634 / (double)tau; }

// ---------------------------------------------------------------------------
// First launch: per block of 256 its maximum (NaN if it holds one) and
// sum exp((z - maximum) / tau), one block per half wave.
// ---------------------------------------------------------------------------
constexpr int kStatThreads = 256;
constexpr int kStatBlocks = kStatThreads / kLanes;

template <typename T>
__global__ __launch_bounds__(kStatThreads) void sample_stats_kernel(SampleArgs a, int G) {
  const int64_t row = blockIdx.y;
  const Row<T> r(a, row);
  const int b = blockIdx.x * kStatBlocks + threadIdx.x / kLanes;
  if (b >= r.blocks()) return;  // uniform over the half wave
  const int c = b * kLanes + threadIdx.x % kLanes;
  float z[kChunk];
  r.load(c, z);
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < kChunk; ++k) {
    nan |= z[k] != z[k];
    m = fmaxf(m, z[k]);
  }
  int any = nan;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o, kLanes));
    any |= __shfl_xor(any, o, kLanes);
  }
  const double rate = rate_of(temperature_of(a, row));
  const double ref = m == -INFINITY ? 0.0 : (double)m;
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kChunk; ++k) s += exp2_neg(((double)z[k] - ref) * rate);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor(s, o, kLanes);
  if (threadIdx.x % kLanes == 0) {
    a.block_max[row * G + b] = any ? NAN : m;
    a.block_sum[row * G + b] = s;
  }
}

// ---------------------------------------------------------------------------
// Second launch: one workgroup a row.
// ---------------------------------------------------------------------------
constexpr int NT = 512;
constexpr int kWaves = NT / 64;
constexpr int kBins = 2048;
constexpr int kBinsPer = kBins / NT;

template <typename V_>
__device__ __forceinline__ V_ wave_scan(V_ v) {  // inclusive
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const V_ u = __shfl_up(v, o, 64);
    if ((int)(threadIdx.x & 63) >= o) v += u;
  }
  return v;
}

// Sum over the threads before this one, and over all of them. `tmp` holds a
// value per wave.
template <typename V_>
__device__ V_ block_scan(V_ v, V_* tmp, V_& total) {
  const V_ inc = wave_scan(v);
  if ((threadIdx.x & 63) == 63) tmp[threadIdx.x >> 6] = inc;
  __syncthreads();
  V_ before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < (int)(threadIdx.x >> 6)) before += tmp[w];
    total += tmp[w];
  }
  __syncthreads();
  return before + inc - v;
}

// What part of the order is kept: keys above `key`, and the first `ties` by
// index of those equal to it.
struct Cut {
  uint32_t key;
  uint32_t ties;
};

struct Shared {
  unsigned long long mass[kBins];
  uint32_t count[kBins];
  unsigned long long scan64[kWaves];
  uint32_t scan32[kWaves];
  double scand[kWaves];
  float maxw[kWaves];
  int nanw[kWaves];
  // what one thread found for all
  uint32_t bin;
  unsigned long long before;
  uint32_t bin_count;
  unsigned long long bin_mass;
  int block;
  unsigned long long block_target, block_ties;
};

template <typename T>
struct RowSampler {
  const Row<T> r;
  Shared& sh;
  const double m, rate;
  const double unit;  // 2^F
  __device__ double weight(float z) const { return exp2_neg(((double)z - m) * rate); }
  __device__ unsigned long long quant(float z) const { return (unsigned long long)rint(weight(z) * unit); }

  // The cut at which, from the top of the order, `target` is first reached by
  // the count (by_mass false) or by the mass. lo: the least key that takes
  // part. above_mass: the mass above the cut's key. If the target is never
  // reached, everything from lo on.
  __device__ Cut find(bool by_mass, unsigned long long target, uint32_t lo, uint32_t hi,
                      unsigned long long& above_mass) {
    unsigned long long above = 0, am = 0;
    uint32_t bin_count = 0;
    for (;;) {
      const uint32_t range = hi - lo;
      const int bits = 32 - __clz(range | 1);
      const int shift = bits > 11 ? bits - 11 : 0;
      const int nbins = (int)(range >> shift) + 1;
      for (int i = threadIdx.x; i < kBins; i += NT) sh.mass[i] = 0, sh.count[i] = 0;
      __syncthreads();
      for (int c = threadIdx.x; c < r.chunks(); c += NT) {
        float z[kChunk];
        r.load(c, z);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const uint32_t key = Key<T>::of(z[k]);
          if (key >= lo && key <= hi) {
            atomicAdd(&sh.count[(key - lo) >> shift], 1u);
            if (shift) atomicAdd(&sh.mass[(key - lo) >> shift], quant(z[k]));
          }
        }
      }
      __syncthreads();
      if (!shift)  // one key a bin: its mass is its count times its weight
        for (int i = threadIdx.x; i < nbins; i += NT)
          sh.mass[i] = sh.count[i] * quant(Key<T>::value(lo + i));
      __syncthreads();
      unsigned long long cnt = 0, mas = 0;
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        const int bin = nbins - 1 - ((int)threadIdx.x * kBinsPer + i);
        if (bin >= 0) cnt += sh.count[bin], mas += sh.mass[bin];
      }
      unsigned long long tc, tm;
      unsigned long long c0 = block_scan(cnt, sh.scan64, tc), m0 = block_scan(mas, sh.scan64, tm);
      if (by_mass ? am + tm < target : above + tc < target) {  // never reached
        above_mass = am + tm;
        return Cut{lo, 0xffffffffu};
      }
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        const int bin = nbins - 1 - ((int)threadIdx.x * kBinsPer + i);
        if (bin < 0) continue;
        const unsigned long long c1 = c0 + sh.count[bin], m1 = m0 + sh.mass[bin];
        const unsigned long long x0 = by_mass ? am + m0 : above + c0, x1 = by_mass ? am + m1 : above + c1;
        if (x0 < target && x1 >= target) {  // one thread, one bin
          sh.bin = bin;
          sh.before = c0;
          sh.block_target = m0;
          sh.bin_count = sh.count[bin];
          sh.bin_mass = sh.mass[bin];
        }
        c0 = c1;
        m0 = m1;
      }
      __syncthreads();
      above += sh.before;
      am += sh.block_target;
      bin_count = sh.bin_count;
      const uint32_t bin = sh.bin;
      __syncthreads();
      const uint32_t last = (bin << shift) | ((1u << shift) - 1);  // within the bracket, which may end at 2^32 - 1
      hi = lo + (last < range ? last : range);
      lo += bin << shift;
      if (!shift) break;
    }
    above_mass = am;
    const unsigned long long need = target - (by_mass ? am : above);  // >= 1
    unsigned long long ties = need;
    if (by_mass) {
      const unsigned long long q = quant(Key<T>::value(lo));
      ties = q ? (need + q - 1) / q : bin_count;
    }
    return Cut{lo, (uint32_t)(ties < bin_count ? ties : bin_count)};
  }
};

template <typename T>
__global__ __launch_bounds__(NT) void sample_row_kernel(SampleArgs a, int G) {
  extern __shared__ char lds[];
  Shared& sh = *reinterpret_cast<Shared*>(lds);
  unsigned long long* bq = reinterpret_cast<unsigned long long*>(lds + sizeof(Shared));  // [G] kept mass
  uint32_t* bt = reinterpret_cast<uint32_t*>(bq + G);                                    // [G] ties
  const int64_t row = blockIdx.x;
  const Row<T> r(a, row);
  const int nb = r.blocks();
  const float* bmax = a.block_max + row * G;
  const double* bsum = a.block_sum + row * G;

  const float tau = temperature_of(a, row);
  const float top_p = a.top_p_rows ? a.top_p_rows[row] : a.top_p;
  const float min_p = a.min_p_rows ? a.min_p_rows[row] : a.min_p;
  const int top_k = a.top_k_rows ? a.top_k_rows[row] : a.top_k;
  float u = a.uniforms[row];

  float mf = -INFINITY;
  int nan = 0;
  for (int b = threadIdx.x; b < nb; b += NT) {
    const float v = bmax[b];
    nan |= v != v;
    mf = fmaxf(mf, v);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    mf = fmaxf(mf, __shfl_xor(mf, o, 64));
    nan |= __shfl_xor(nan, o, 64);
  }
  if ((threadIdx.x & 63) == 0) sh.maxw[threadIdx.x >> 6] = mf, sh.nanw[threadIdx.x >> 6] = nan;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mf = fmaxf(mf, sh.maxw[w]), nan |= sh.nanw[w];
  __syncthreads();
  // no distribution: a NaN, nothing above -inf, +inf, or a setting that is none
  if (nan || !(fabsf(mf) < INFINITY) || !(tau >= 0.f && tau < INFINITY) || top_p != top_p || min_p != min_p ||
      u != u) {
    if (threadIdx.x == 0) {
      a.token[row] = -1;
      if (a.logp) a.logp[row] = NAN;
      if (a.kept_logp) a.kept_logp[row] = NAN;
    }
    return;
  }
  if (tau == 0.f) {  // the first of the largest
    if (threadIdx.x == 0) sh.block = 0x7fffffff;
    __syncthreads();
    for (int b = threadIdx.x; b < nb; b += NT)
      if (bmax[b] == mf) {
        atomicMin(&sh.block, b);
        break;
      }
    __syncthreads();
    if (threadIdx.x < kLanes) {
      const int c = sh.block * kLanes + threadIdx.x;
      float z[kChunk];
      r.load(c, z);
      int at = 0x7fffffff;
#pragma unroll
      for (int k = kChunk - 1; k >= 0; --k)
        if (z[k] == mf) at = r.first(c) + k;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) at = min(at, __shfl_xor(at, o, kLanes));
      if (threadIdx.x == 0) {
        a.token[row] = at;
        if (a.logp) a.logp[row] = 0.f;
        if (a.kept_logp) a.kept_logp[row] = 0.f;
      }
    }
    return;
  }

  const double rate = rate_of(tau);
  const int per = (nb + NT - 1) / NT;  // blocks a thread takes, one after the other
  const int b0 = min(nb, (int)threadIdx.x * per), b1 = min(nb, b0 + per);
  double sum = 0.0;
  for (int b = b0; b < b1; ++b) sum += bsum[b] * exp2_neg(((double)bmax[b] - (double)mf) * rate);
  double S;
  block_scan(sum, sh.scand, S);
  // q_i = round(w_i 2^F) add up to less than 2^62: S < 2^(e+1), and the
  // roundings add at most half of V <= 2^20
  const int F = 60 - ilogb(S);
  RowSampler<T> s{r, sh, (double)mf, rate, ldexp(1.0, F)};

  const uint32_t lowest = Key<T>::of(-INFINITY) + 1, highest = Key<T>::of(mf);
  Cut cut{lowest, 0xffffffffu};
  const bool k_on = top_k > 0 && top_k < a.V, p_on = top_p < 1.f, m_on = min_p > 0.f;
  unsigned long long above = 0;
  if (k_on) cut = s.find(false, top_k, lowest, highest, above);
  if (p_on) {
    double mass;
    if (k_on) {
      const unsigned long long q = s.quant(Key<T>::value(cut.key));
      mass = cut.ties == 0xffffffffu ? (double)above : (double)above + (double)cut.ties * (double)q;
    } else {
      mass = S * s.unit;
    }
    const double t = ceil(fmax((double)top_p, 0.0) * mass);
    unsigned long long ap;
    const Cut c = s.find(true, t < 1.0 ? 1ull : (unsigned long long)t, k_on ? cut.key : lowest, highest, ap);
    if (!k_on || c.key > cut.key || (c.key == cut.key && c.ties < cut.ties)) cut = c;
  }
  const bool limited = k_on || p_on || m_on;
  const double least = fmin((double)min_p, 1.0);

  // the kept mass of each block, and its ties with the cut
  if (limited) {
    for (int b = threadIdx.x / kLanes; b < nb; b += NT / kLanes) {
      float z[kChunk];
      r.load(b * kLanes + threadIdx.x % kLanes, z);
      unsigned long long q = 0;
      uint32_t t = 0;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        const uint32_t key = Key<T>::of(z[k]);
        if (key < cut.key) continue;
        if (key == cut.key && cut.ties != 0xffffffffu)
          ++t;
        else if (s.weight(z[k]) >= least)
          q += s.quant(z[k]);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) q += __shfl_xor(q, o, kLanes), t += __shfl_xor(t, o, kLanes);
      if (threadIdx.x % kLanes == 0) bq[b] = q, bt[b] = t;
    }
    __syncthreads();
    uint32_t ties = 0, all;
    for (int b = b0; b < b1; ++b) ties += bt[b];
    uint32_t before = block_scan(ties, sh.scan32, all);
    const float zc = Key<T>::value(cut.key);
    const unsigned long long qc = s.weight(zc) >= least ? s.quant(zc) : 0;
    for (int b = b0; b < b1; ++b) {
      const uint32_t mine = bt[b], left = before < cut.ties ? cut.ties - before : 0;
      bq[b] += (unsigned long long)(mine < left ? mine : left) * qc;
      bt[b] = left;  // ties this block may still keep
      before += mine;
    }
  } else {
    // a block whose largest logit weighs nothing is left out, so that the
    // block taken holds a token to take
    for (int b = b0; b < b1; ++b)
      bq[b] = s.quant(bmax[b]) ? (unsigned long long)rint(bsum[b] * s.weight(bmax[b]) * s.unit) : 0ull;
  }
  unsigned long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += bq[b];
  unsigned long long before = block_scan(mine, sh.scan64, total);
  u = fminf(fmaxf(u, 0.f), 0x1.fffffep-1f);
  const unsigned long long target = (unsigned long long)((double)u * (double)total);  // the sum to exceed
  for (int b = b0; b < b1; ++b) {
    if (before <= target && before + bq[b] > target) sh.block = b, sh.block_target = target - before;
    before += bq[b];
  }
  __syncthreads();

  // the index within the block
  if (threadIdx.x < 64) {
    const int l = threadIdx.x;
    const int c = sh.block * kLanes + l;
    float z[kChunk];
    unsigned long long q[kChunk], chunk = 0;
    uint32_t t = 0;
    if (l < kLanes) r.load(c, z);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (l >= kLanes) z[k] = -INFINITY;
      t += Key<T>::of(z[k]) == cut.key;
    }
    uint32_t rank = wave_scan(t) - t;
    const uint32_t left = limited ? bt[sh.block] : 0;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      const uint32_t key = Key<T>::of(z[k]);
      bool keep = z[k] != -INFINITY;
      if (limited) {
        keep = keep && key >= cut.key && s.weight(z[k]) >= least;
        if (key == cut.key && cut.ties != 0xffffffffu) keep = keep && rank++ < left;
      }
      q[k] = keep ? s.quant(z[k]) : 0;
      chunk += q[k];
    }
    unsigned long long run = wave_scan(chunk) - chunk;
    // the first index at which the sum exceeds the target; if roundings of
    // the block's own sum leave none, the last that weighs anything
    int hit = 0x7fffffff, last = -1;
    float zh = 0.f, zl = 0.f;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      run += q[k];
      if (q[k]) {
        last = r.first(c) + k, zl = z[k];
        if (run > sh.block_target && hit == 0x7fffffff) hit = r.first(c) + k, zh = z[k];
      }
    }
    const int first = [&] {
      int x = hit;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) x = min(x, __shfl_xor(x, o, 64));
      return x;
    }();
    int end = last;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) end = max(end, __shfl_xor(end, o, 64));
    const int tok = first != 0x7fffffff ? first : end;
    if (hit == tok || (first == 0x7fffffff && last == tok)) {
      const float zt = hit == tok ? zh : zl;
      const double x = ((double)zt - (double)mf) / (double)tau;
      a.token[row] = tok;
      if (a.logp) a.logp[row] = (float)(x - log(S));
      if (a.kept_logp) a.kept_logp[row] = (float)(x - log((double)total / s.unit));
    }
  }
}

template <typename T>
hipError_t sample(const SampleArgs& a, hipStream_t st) {
  const int G = sample_blocks(a.V);
  const size_t lds = sizeof(Shared) + (size_t)G * 12;
  for (int64_t r0 = 0; r0 < a.N; r0 += 32768) {  // the grid's second dimension holds 65535
    SampleArgs b = a;
    b.N = std::min<int64_t>(32768, a.N - r0);
    b.logits = (const T*)a.logits + r0 * a.stride;
    b.uniforms = a.uniforms + r0;
    if (a.tau_rows) b.tau_rows = a.tau_rows + r0;
    if (a.top_p_rows) b.top_p_rows = a.top_p_rows + r0;
    if (a.min_p_rows) b.min_p_rows = a.min_p_rows + r0;
    if (a.top_k_rows) b.top_k_rows = a.top_k_rows + r0;
    b.token = a.token + r0;
    if (a.logp) b.logp = a.logp + r0;
    if (a.kept_logp) b.kept_logp = a.kept_logp + r0;
    b.block_max = a.block_max + r0 * G;
    b.block_sum = a.block_sum + r0 * G;
    sample_stats_kernel<T><<<dim3((G + kStatBlocks - 1) / kStatBlocks, (unsigned)b.N), kStatThreads, 0, st>>>(b, G);
    if (hipError_t e = hipGetLastError()) return e;
    sample_row_kernel<T><<<(unsigned)b.N, NT, lds, st>>>(b, G);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t st) {
  return a.dtype == 0 ? sample<float>(a, st) : sample<__bf16>(a, st);
}

}  // namespace plp
