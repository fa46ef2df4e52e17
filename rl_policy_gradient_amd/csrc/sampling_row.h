// What sampling and the verification of drafted tokens share: a row of logits,
// its blocks' statistics, and the search for the cut that the row's limits set,
// on whole-number masses (sampling.hip says what the cut is and why so).
#pragma once

#include "ops.h"

#include <math.h>

#include <algorithm>

namespace plp {

namespace {

typedef unsigned long long u64;

constexpr int kChunk = 8;                       // consecutive logits a lane takes
constexpr int kLanes = kSampleBlock / kChunk;   // lanes of one block: 32
static_assert(kLanes == 32, "half a wave a block");

// 2^(d rate) for d rate between -1000 and a little above 0 (the callers hold
// d at or above -1000 / rate): a polynomial of degree 9 through the Chebyshev
// points of [-1/2, 1/2] (relative error 1.9e-14) on the distance
// to the nearest whole number, which is added to the result's exponent.
// Adding 1.5 x 2^52 rounds to that number and leaves it in the sum's low
// bits: no conversion, and 14 operations in all.
__device__ __forceinline__ double exp2_of(double d, double rate) {
  constexpr double magic = 0x1.8p52;
  const double t = fma(d, rate, magic);
  const double f = fma(d, rate, magic - t);
  double p = 0x1.b6571de2f2351p-24;
  p = fma(p, f, 0x1.63ef969a64d3cp-20);
  p = fma(p, f, 0x1.ffcb76789860fp-17);
  p = fma(p, f, 0x1.43088e257f341p-13);
  p = fma(p, f, 0x1.5d87fe908f88ap-10);
  p = fma(p, f, 0x1.3b2ab72b175eep-7);
  p = fma(p, f, 0x1.c6b08d7044119p-5);
  p = fma(p, f, 0x1.ebfbdff8149f2p-3);
  p = fma(p, f, 0x1.62e42fefa39f7p-1);
  p = fma(p, f, 1.0);
  const int n = (int)(uint32_t)__double_as_longlong(t);
  return __hiloint2double(__double2hiint(p) + (n << 20), __double2loint(p));
}
// The least d that exp2_of takes: -1000 / rate.
__device__ __forceinline__ double least_of(float tau) { return tau == 0.f ? -1000.0 : (double)tau * -693.147180559945; }

// A value that is the same in every lane, kept in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) { return __int_as_float(uniform(__float_as_int(v))); }
__device__ __forceinline__ u64 uniform(u64 v) {
  return (u64)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v);
}
__device__ __forceinline__ double uniform(double v) {
  return __longlong_as_double((long long)uniform((u64)__double_as_longlong(v)));
}
// Lane `l`'s value, l the same in every lane.
__device__ __forceinline__ int lane_of(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) { return (uint32_t)lane_of((int)v, l); }
__device__ __forceinline__ float lane_of(float v, int l) { return __int_as_float(lane_of(__float_as_int(v), l)); }
__device__ __forceinline__ u64 lane_of(u64 v, int l) {
  return (u64)(uint32_t)lane_of((int)(v >> 32), l) << 32 | (uint32_t)lane_of((int)v, l);
}
__device__ __forceinline__ double lane_of(double v, int l) {
  return __longlong_as_double((long long)lane_of((u64)__double_as_longlong(v), l));
}
// The value of another lane by a lane permutation (no LDS round trip); 0 where
// it has no source or the row is not in ROWS (with all rows, the permutation
// itself fills in the 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ int permuted(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, ROWS == 0xf);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t permuted(uint32_t v) {
  return (uint32_t)permuted<CTRL, ROWS>((int)v);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float permuted(float v) {
  return __int_as_float(permuted<CTRL, ROWS>(__float_as_int(v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 permuted(u64 v) {
  return (u64)(uint32_t)permuted<CTRL, ROWS>((int)(v >> 32)) << 32 | (uint32_t)permuted<CTRL, ROWS>((int)v);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double permuted(double v) {
  return __longlong_as_double((long long)permuted<CTRL, ROWS>((u64)__double_as_longlong(v)));
}
// op over the 16 lanes of a row, in each of them.
template <typename V_, typename F>
__device__ __forceinline__ V_ row_reduce(V_ v, F op) {
  v = op(v, permuted<0xb1, 0xf>(v));   // lanes 1 0 3 2 of each quad
  v = op(v, permuted<0x4e, 0xf>(v));   // lanes 2 3 0 1
  v = op(v, permuted<0x141, 0xf>(v));  // mirrored in each half row
  return op(v, permuted<0x140, 0xf>(v));
}
// op over the 32 lanes of a half wave, in each of them, and over a wave.
template <typename V_, typename F>
__device__ __forceinline__ V_ half_reduce(V_ v, F op) {
  v = row_reduce(v, op);
  return op(v, __shfl_xor(v, 16, 64));
}
template <typename V_, typename F>
__device__ __forceinline__ V_ wave_reduce(V_ v, F op) {
  v = row_reduce(v, op);
  return op(op(lane_of(v, 0), lane_of(v, 16)), op(lane_of(v, 32), lane_of(v, 48)));
}
struct Add {
  template <typename V_>
  __device__ __forceinline__ V_ operator()(V_ a, V_ b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Min {
  __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};

// Monotone whole-number keys of the logits (no NaN): -inf is the least that
// occurs. bf16 logits need 16 bits, fp32 ones 32.
template <typename T>
struct Key;
template <>
struct Key<float> {
  static constexpr int bits = 32;
  __device__ static uint32_t of(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);  // -0 ties with +0
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
// fp32 one two.)
template <typename T>
struct Row {
  const T* p;
  int V, lead;
  __device__ Row(const T* logits, int length) : p(logits), V(length) {
    constexpr int per16 = 16 / sizeof(T);
    lead = (int)(((uintptr_t)p / sizeof(T)) % per16);
  }
  __device__ int chunks() const { return (V + lead + kChunk - 1) / kChunk; }
  __device__ int blocks() const { return (V + lead + kSampleBlock - 1) / kSampleBlock; }
  __device__ int first(int c) const { return c * kChunk - lead; }
  // A chunk as it lies in memory: nothing waits for the load before `values`.
  struct Raw {
    uint4 w[kChunk * sizeof(T) / 16];
  };
  __device__ __forceinline__ Raw fetch(int c) const {
    const int e0 = first(c);
    if (e0 >= 0 && e0 + kChunk <= V) return *(const Raw*)(p + e0);
    T t[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) t[k] = e0 + k >= 0 && e0 + k < V ? p[e0 + k] : (T)-INFINITY;
    return __builtin_bit_cast(Raw, t);
  }
  __device__ static __forceinline__ void values(const Raw& raw, float (&z)[kChunk]) {
    const T(&t)[kChunk] = reinterpret_cast<const T(&)[kChunk]>(raw);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) z[k] = (float)t[k];
  }
  __device__ __forceinline__ void load(int c, float (&z)[kChunk]) const { values(fetch(c), z); }
};

// log2(e) / tau; 1 for the greedy row, whose weights are not used.
__host__ __device__ inline double rate_of(float tau) { return tau == 0.f ? 1.0 : 1.4426950408889634 / (double)tau; }

// ---------------------------------------------------------------------------
// First launch: per block of 256 its maximum (NaN if it holds one) and
// sum exp((z - maximum) / tau), one block per 16 lanes.
// ---------------------------------------------------------------------------
constexpr int kStatThreads = 256;
constexpr int kStatLanes = 16;                     // a row of lanes a block
constexpr int kStatChunks = kLanes / kStatLanes;   // chunks a lane takes
constexpr int kStatBlocks = kStatThreads / kStatLanes;

// The larger, NaN if either is.
struct MaxOrNan {
  __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_elementwise_maximum(a, b); }
};

// Block b of a row, by its 16 lanes (`lane` of them).
template <typename T>
__device__ __forceinline__ void fetch_block(const Row<T>& r, int b, int lane, typename Row<T>::Raw (&raw)[kStatChunks]) {
#pragma unroll
  for (int c = 0; c < kStatChunks; ++c) raw[c] = r.fetch(b * kLanes + c * kStatLanes + lane);
}
// Eight logits of 16 or 32 bytes. The wider type's bits are put together, as the
// compiler takes a maximum of converted bf16 values in bf16, in three
// instructions for each (576 rows of 151936: 77 us so, 72 as it is).
template <typename T, typename R>
__device__ __forceinline__ void widen(const R& raw, float (&z)[kChunk]) {
  static_assert(sizeof(R) == kChunk * sizeof(T), "a chunk");
  if constexpr (sizeof(T) == 2) {
    const auto w = __builtin_bit_cast(uint4, raw);
    const uint32_t pairs[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < kChunk; ++k)
      z[k] = __uint_as_float(k & 1 ? pairs[k / 2] & 0xffff0000u : pairs[k / 2] << 16);
  } else {
    const T(&t)[kChunk] = reinterpret_cast<const T(&)[kChunk]>(raw);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) z[k] = t[k];
  }
}
template <typename T>
__device__ __forceinline__ void block_stats(const typename Row<T>::Raw (&raw)[kStatChunks], float tau, double rate, float& m,
                                            double& s) {
  const double least = least_of(tau);
  float z[kStatChunks][kChunk];
#pragma unroll
  for (int c = 0; c < kStatChunks; ++c) widen<T>(raw[c], z[c]);
  m = z[0][0];
#pragma unroll
  for (int c = 0; c < kStatChunks; ++c)
#pragma unroll
    for (int k = 0; k < kChunk; k += 2) m = MaxOrNan()(MaxOrNan()(m, z[c][k]), z[c][k + 1]);
  m = row_reduce(m, MaxOrNan());
  const double ref = m == -INFINITY ? 0.0 : (double)m;
  s = 0.0;
#pragma unroll
  for (int c = 0; c < kStatChunks; ++c)
#pragma unroll
    for (int k = 0; k < kChunk; ++k) s += exp2_of(fmax((double)z[c][k] - ref, least), rate);
  s = row_reduce(s, Add());
}

// ---------------------------------------------------------------------------
// Second launch: one workgroup a row. What it reads again is decided by the
// blocks' maxima and sums:
//
//  1. From them alone, a value that the cut cannot lie below: one that at
//     least k block maxima reach, or above which the blocks that reach it hold
//     a mass of top_p even if all their other logits were as large as it. Only
//     the blocks that reach it (the active ones) are read.
//  2. The logits at or above it are listed in LDS; each one's rank and the mass
//     before it give the cut (a few), or a radix search over their places in
//     the order does (many).
//  3. Where the maxima give no bound (fewer blocks than k) or the candidates
//     are too many to list (top_p on a flat row, or many active blocks), a
//     histogram of at least 16384 logits of the row tells near which value the
//     cut lies; one pass adds up what is above that neighbourhood and lists
//     what is in it.
//  4. Where that fails too (a large k, thousands of equal logits at the cut),
//     the neighbourhood is narrowed by exact histograms over places, 11 bits
//     a pass, until it can be listed.
//
// In each case the decision is the same whole-number one. The kernel runs once
// through most of its code, so that its size counts (36 KB): loops over a
// lane's eight logits are not unrolled where it can be helped and each step has
// one place in the code (unrolled and inlined where used it was 91 KB, and a
// row took two to three times as long, fetching it).
// ---------------------------------------------------------------------------
// Threads of a row's workgroup: NT of them, one workgroup a CU, or where there
// are more rows than CUs half as many and two a CU (verify.hip); no result
// depends on which (TH, in what follows).
constexpr int NT = 1024;
constexpr int kHalfNT = NT / 2;
constexpr int kWaves = NT / 64;  // at most
constexpr int kBins = 2048;
constexpr int kList = 4096;        // logits that can be listed
// Up to so many, every listed logit is compared with every other, else the
// cut is searched for by histograms (51 listed: 18 us a call against 22).
template <int TH>
constexpr int kRanked = TH / 4;
// Logits up to which a whole row is listed for top_k, when the maxima do not
// bound it, instead of an estimate (64 rows, k = 50 to 400: of 300, 24 us
// against 26; of 1000, 21 to 25 against 18 to 33; of 1500, 24 against 20).
constexpr int kAll = 1024;
// Active blocks up to which top_p's candidates are listed without an estimate
// in rows that are not flat (64 peaked rows of 32000 bf16 at top_p 0.9, 125
// blocks: 25 us against 30; of 151936 with some 200 active, 35 against 40,
// with nearly all 594 active 85 against 58).
constexpr int kDirect = 256;
// Logits of the estimate, at least (64 flat rows of 151936 in fp32: 94 us;
// 8192 of them miss the cut too often, 210; 32768 cost what they save, 97).
constexpr int kEstimate = 16384;
// Logits listed on either side of the estimated cut: a margin for the bins'
// own error, and kAround sqrt(V (step - 1)) for that of a sample of every
// step-th, about three times its usual one (1250 of 151936; rows of 32000 are
// sampled whole: 37 us instead of 42 with a list of 1250 either side).
constexpr float kMargin = 32.f, kAround = 1.09f;

// A logit's place in the order, the larger the earlier: its key, then its
// index from the end.
constexpr int kIndexBits = 20;
static_assert(kSampleMaxV <= 1 << kIndexBits, "an index fits its bits");
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
__device__ __forceinline__ u64 place_of(uint32_t key, int index) {
  return (u64)key << kIndexBits | (kIndexMask - (uint32_t)index);
}
__device__ __forceinline__ u64 last_place(uint32_t key) { return (u64)key << kIndexBits; }
__device__ __forceinline__ int index_at(u64 place) { return (int)(kIndexMask - ((uint32_t)place & kIndexMask)); }

// Inclusive scan over the wave by lane permutations within rows of 16, then
// across rows.
template <typename V_>
__device__ __forceinline__ V_ wave_scan(V_ v) {
  v += permuted<0x111, 0xf>(v);  // one lane up within the row, two, four, eight
  v += permuted<0x112, 0xf>(v);
  v += permuted<0x114, 0xf>(v);
  v += permuted<0x118, 0xf>(v);
  v += permuted<0x142, 0xa>(v);  // the row before's last into rows 1 and 3
  v += permuted<0x143, 0xc>(v);  // row 1's last into rows 2 and 3
  return v;
}

// Sum over the threads before this one, and over all of them. `tmp` holds a
// value per wave.
template <int TH = NT, typename V_>
__device__ __forceinline__ V_ block_scan(V_ v, V_* tmp, V_& total) {
  constexpr int waves_of = TH / 64;
  const V_ inc = wave_scan(v);
  const int wave = uniform((int)threadIdx.x >> 6);
  if ((threadIdx.x & 63) == 63) tmp[wave] = inc;
  __syncthreads();
  const V_ waves = wave_scan(tmp[threadIdx.x & (waves_of - 1)]);  // the first lanes' count
  total = lane_of(waves, waves_of - 1);
  const V_ before = wave ? lane_of(waves, wave - 1) : (V_)0;
  __syncthreads();
  return before + (inc - v);
}

// f(k, z[k]) for the chunk's eight, one copy of f in the code: the registers
// move on instead of the index.
template <typename F>
__device__ __forceinline__ void for_chunk(float (&z)[kChunk], F f) {
#pragma unroll 1
  for (int k = 0; k < kChunk; ++k) {
    f(k, z[0]);
    const float first = z[0];
#pragma unroll
    for (int i = 0; i + 1 < kChunk; ++i) z[i] = z[i + 1];
    z[kChunk - 1] = first;  // as they were after the last
  }
}

// For rows with limits only.
template <int TH = NT>
struct Lists {
  u64 list[kList];  // places
  u64 q[kList];     // their masses
  u64 mass[kBins];
  uint32_t count[kBins];
  __device__ __forceinline__ u64* masses() { return q; }
};
// Two workgroups a CU have 80 KB of LDS each, up to some 440000 logits: the
// masses of a short list, and what a pass puts side by side, are where the
// histograms are at other times; a longer list's are formed again.
template <>
struct Lists<kHalfNT> {
  u64 list[kList];
  u64 mass[kBins];
  uint32_t count[kBins];
  __device__ __forceinline__ u64* masses() { return mass; }
};
static_assert(sizeof(Lists<kHalfNT>::mass) >= kHalfNT / kLanes * kSampleBlock * sizeof(float) &&
                  sizeof(Lists<NT>::q) >= NT / kLanes * kSampleBlock * sizeof(float),
              "a block's logits for each half wave");
static_assert(kRanked<kHalfNT> <= kBins, "the masses of a short list");
struct Shared {
  u64 scan64[kWaves];
  double scand[kWaves];
  uint32_t scan32[kWaves];
  float maxw[kWaves], minw[kWaves];
  int flag[kWaves];
  float low;
  // what one thread found for all
  int block, bin, edge_lo, edge_hi;
  uint32_t n, few, bin_count;
  u64 place, a, b, bin_mass, above;
};

template <typename T, int TH = NT>
struct RowSampler {
  static constexpr int kBinsPer = kBins / TH;
  static constexpr bool kMasses = TH == NT;  // whether a list's masses are kept
  const Row<T> r;
  Shared& sh;
  Lists<TH>& ls;
  float* const bmax;    // [blocks] maxima
  u64* const bq;        // [blocks] the bits of the blocks' sums (doubles), later their kept masses
  uint16_t* const act;  // active blocks, by index
  const int nb;
  const float mf;
  const double m, rate, least_d;
  double S, unit;       // sum of the weights; 2^F
  double least;         // min_p, or -1

  // A logit of -inf weighs 2^-1000, which is nothing beside the largest's 1
  // and a mass of 0.
  __device__ __forceinline__ double weight(float z) const {
    return exp2_of(fmax((double)z - m, least_d), rate);
  }
  // round(w 2^F), below 2^52: the low bits of the sum with 2^52
  __device__ __forceinline__ u64 quant(double w) const {
    return (u64)__double_as_longlong(fma(w, unit, 0x1p52)) & 0xfffffffffffffull;
  }
  // The mass of entry j of the list, which is `place`.
  __device__ __forceinline__ u64 mass_of(int j, u64 place) const {
    if constexpr (kMasses)
      return ls.masses()[j];
    else
      return quant(weight(value_at(place)));
  }
  __device__ __forceinline__ float value_at(u64 place) const {
    return Key<T>::value((uint32_t)(place >> kIndexBits));
  }

  // The highest of 2048 values between lowest_max and mf that at least k block
  // maxima reach, or above which the blocks that reach it hold `goal` even if
  // all their logits below it were as large as it; `none` if there is none. A
  // histogram of the maxima, with the blocks' masses.
  __device__ __forceinline__ float bound(float lowest_max, bool by_count, int k, double goal, float none) {
    const float scale = (float)kBins / (mf - lowest_max);
    if (threadIdx.x == 0) sh.bin = -1;
    clear_bins();
    for (int b = threadIdx.x; b < nb; b += TH) {
      if (bmax[b] == -INFINITY) continue;
      const int bin = max(0, min(kBins - 1, (int)((bmax[b] - lowest_max) * scale)));
      atomicAdd(&ls.count[bin], 1u);
      if (!by_count) atomicAdd(&ls.mass[bin], quant(__longlong_as_double((long long)bq[b])));
    }
    __syncthreads();
    uint32_t c = 0, tc;
    u64 q = 0, tq;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int bin = kBins - 1 - ((int)threadIdx.x * kBinsPer + i);
      c += ls.count[bin], q += ls.mass[bin];
    }
    c = block_scan<TH>(c, sh.scan32, tc);
    if (!by_count) q = block_scan<TH>(q, sh.scan64, tq);
    // a hundredth of a bin lower, so that a bin's rounding does not matter
    const auto value = [&](int bin) { return lowest_max + ((float)bin - 0.01f) / scale; };
    int best = -1;  // bins fall with the thread: the first to say yes has the highest
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int bin = kBins - 1 - ((int)threadIdx.x * kBinsPer + i);
      c += ls.count[bin], q += ls.mass[bin];
      const bool yes = by_count ? (int)c >= k
                                : c > 0 && (double)q >= goal + (double)c * kSampleBlock * weight(value(bin)) * unit;
      if (yes && best < 0) best = bin;
    }
    const u64 said = __ballot(best >= 0);
    if (said && (threadIdx.x & 63) == (unsigned)__ffsll(said) - 1) atomicMax(&sh.bin, best);
    __syncthreads();
    const int bin = uniform(sh.bin);
    return bin < 0 ? none : value(bin);
  }

  // Whether a block holds a 32nd of the row's mass, and four times its even
  // share or half of everything.
  __device__ __forceinline__ bool peaked() {
    bool yes = false;
    const double most = S * fmax(1.0 / 32.0, fmin(4.0 / (double)nb, 0.5));
    for (int b = threadIdx.x; b < nb; b += TH) yes |= __longlong_as_double((long long)bq[b]) >= most;
    return __syncthreads_or(yes ? 1 : 0) != 0;
  }

  // Lists the active blocks: those whose maximum is at least z.
  __device__ __forceinline__ int activate(float z) {
    const int per = (nb + TH - 1) / TH, b0 = min(nb, (int)threadIdx.x * per), b1 = min(nb, b0 + per);
    uint32_t n = 0, total;
    for (int b = b0; b < b1; ++b) n += bmax[b] >= z;
    uint32_t at = block_scan<TH>(n, sh.scan32, total);
    for (int b = b0; b < b1; ++b)
      if (bmax[b] >= z) act[at++] = (uint16_t)b;
    __syncthreads();
    return uniform((int)total);
  }

  __device__ __forceinline__ void begin_pass() {
    for (int b = threadIdx.x; b < nb; b += TH) bq[b] = 0;
    if (threadIdx.x == 0) sh.n = 0, sh.above = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void end_pass(u64 above) {
    above = wave_reduce(above, Add());
    if ((threadIdx.x & 63) == 0 && above) atomicAdd(&sh.above, above);
    __syncthreads();
  }

  // Over the active blocks: the mass of the logits at or above zh (in
  // sh.above), into bq what of it min_p keeps, and into the list the places of
  // those from zl on (sh.n of them; those past kList are only counted).
  __device__ __forceinline__ void pass(int nact, float zl, float zh) {
    constexpr int step = TH / kLanes;
    begin_pass();
    u64 above = 0;
    const int lane = threadIdx.x % kLanes;
    // the half wave's logits above, in the place of the list's masses, which come later
    float* const some = reinterpret_cast<float*>(ls.masses()) + threadIdx.x / kLanes * kSampleBlock;
    typename Row<T>::Raw next;
    int i = (int)threadIdx.x / kLanes;
    if (i < nact) next = r.fetch(act[i] * kLanes + lane);
#pragma unroll 1
    for (; i < nact; i += step) {
      const int b = act[i];
      float z[kChunk];
      r.values(next, z);
      if (i + step < nact) next = r.fetch(act[i + step] * kLanes + lane);  // on the way meanwhile
      uint32_t listed = 0, over = 0;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        listed |= (z[k] >= zl) & (z[k] < zh) ? 1u << k : 0u;
        over |= z[k] >= zh ? 1u << k : 0u;
      }
      // both counts in one scan
      const uint32_t mine = (uint32_t)__popc(listed) | (uint32_t)__popc(over) << 16, upto = wave_scan(mine);
      if (__ballot(listed != 0)) {  // one addition to the count a wave (a half at the end)
        const int e0 = r.first(b * kLanes + lane);
        const int last = 63 - __clzll((long long)__ballot(1));
        uint32_t at = 0;
        if ((int)(threadIdx.x & 63) == last) at = atomicAdd(&sh.n, upto & 0xffff);
        at = lane_of(at, last) + ((upto - mine) & 0xffff);
#pragma unroll
        for (int k = 0; k < kChunk; ++k)
          if (listed >> k & 1) {
            if (at < kList) ls.list[at] = place_of(Key<T>::of(z[k]), e0 + k);
            ++at;
          }
      }
      if (zh < INFINITY) {  // uniform
        // A weight costs some 20 operations in fp64 and few of the logits are
        // above, so the block's are first put side by side: 64 rows of 151936
        // bf16 at top_p 0.9 and temperature 1.2, 93 us with all eight weights
        // of a lane, 75 so (fp32 rows so flat that most are above: 86 and 94).
        const uint32_t lower = lane_of(upto, 31) >> 16, both = lane_of(upto, 63) >> 16;
        const bool second = threadIdx.x & 32;
        const int n = (int)(second ? both - lower : lower);
        uint32_t at = ((upto - mine) >> 16) - (second ? lower : 0);
#pragma unroll
        for (int k = 0; k < kChunk; ++k)
          if (over >> k & 1) some[at++] = z[k];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");  // read by other lanes of the wave
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        u64 kept = 0;
#pragma unroll 1
        for (int j = lane; j < n; j += kLanes) {
          const double w = weight(some[j]);
          const u64 q = quant(w);
          above += q;
          kept += w >= least ? q : 0;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        kept = half_reduce(kept, Add());
        if (lane == 0) bq[b] = kept;
      }
    }
    end_pass(above);
  }

  // The same over the whole row with bounds at places: above hi, and from hi
  // to lo.
  __device__ __forceinline__ void pass_places(u64 lo, u64 hi) {
    begin_pass();
    u64 above = 0;
    const int lane = threadIdx.x % kLanes;
#pragma unroll 1
    for (int b = threadIdx.x / kLanes; b < nb; b += TH / kLanes) {
      const int c = b * kLanes + lane, e0 = r.first(c);
      float z[kChunk];
      r.load(c, z);
      u64 kept = 0;
      for_chunk(z, [&](int k, float x) {
        const u64 place = place_of(Key<T>::of(x), e0 + k);
        if (place > hi) {
          const double w = weight(x);
          above += quant(w);
          kept += w >= least ? quant(w) : 0;
        } else if (place >= lo) {
          const uint32_t at = atomicAdd(&sh.n, 1u);
          if (at < kList) ls.list[at] = place;
        }
      });
      kept = half_reduce(kept, Add());
      if (lane == 0) bq[b] = kept;
    }
    end_pass(above);
  }

  // The least whole mass at or above p times `mass`, and at least 1.
  __device__ static __forceinline__ u64 needed(float p, double mass) {
    const double t = ceil(fmax((double)p, 0.0) * mass);
    return t < 1.0 ? 1ull : (u64)t;
  }

  // The cut within the list of n places from hi to lo, above which lies the
  // mass `above`: kept are the first k (k >= n: no limit) of those the mass
  // before which is below p times the mass of the first k with k_on, else of
  // everything. False if the cut is not in the list, unless `whole`: then all
  // of it is kept. Adds the kept ones to bq; through: the mass up to and with
  // the cut.
  __device__ __forceinline__ bool cut_in_list(int n, u64 lo, u64 hi, u64 above, u64 k, bool k_on, float p, double mass,
                                              bool whole, u64& cut, u64& through) {
    u64 mine = 0, total;
#pragma unroll 1
    for (int j = threadIdx.x; j < n; j += TH) {
      const u64 q = quant(weight(value_at(ls.list[j])));
      if (kMasses || n <= kRanked<TH>) ls.masses()[j] = q;
      mine += q;
    }
    u64 t = ~0ull;
    if (n <= kRanked<TH>) {
      // every place against every other: four threads share one, each with a
      // quarter of the list
      const int e = threadIdx.x >> 2;
      const bool in = e < n;
      __syncthreads();
      const u64 place = in ? ls.list[e] : 0, q = in ? ls.masses()[e] : 0;
      uint32_t rank = 0;
      u64 before = 0;
      if (in)
#pragma unroll 4
        for (int j = threadIdx.x & 3; j < n; j += 4) {
          const bool first = ls.list[j] > place;
          rank += first;
          before += first ? ls.masses()[j] : 0;
        }
      rank += permuted<0xb1, 0xf>(rank);
      rank += permuted<0x4e, 0xf>(rank);
      before += permuted<0xb1, 0xf>(before);
      before += permuted<0x4e, 0xf>(before);
      before += above;
      const bool one = in && (threadIdx.x & 3) == 0;
      if (one && (rank == k - 1 || (k >= (u64)n && rank == (uint32_t)n - 1))) sh.a = before + q;
      if (one && rank == (uint32_t)n - 1) sh.bin_mass = before + q;
      __syncthreads();
      if (p < 1.f) {
        t = uniform(needed(p, k_on ? (double)sh.a : mass));
        if (above >= t || (!whole && t > uniform(sh.bin_mass))) return false;  // uniform
      }
      if (one && rank < k && before < t && (rank + 1 == (uint32_t)n || rank + 1 >= k || before + q >= t)) {
        sh.place = place;
        sh.b = before + q;
      }
      __syncthreads();
      cut = uniform(sh.place);
      through = uniform(sh.b);
    } else {
      block_scan<TH>(mine, sh.scan64, total);
      total = uniform(total);
      u64 at = lo;  // the earliest cut so far
      through = above + total;
#pragma unroll 1
      for (int by_mass = 0; by_mass < 2; ++by_mass) {
        u64 target = k, got;
        if (by_mass) {
          if (p >= 1.f) break;
          t = uniform(needed(p, k_on ? (double)through : mass));
          if (above >= t || (!whole && t > above + total)) return false;  // uniform
          if (t > above + total) break;
          target = t - above;
        } else if (k >= (u64)n) {
          continue;
        }
        at = radix(by_mass, target, at, hi, got);
        through = above + got;
      }
      cut = at;  // or lo, the last place there can be: all of it
    }
#pragma unroll 1
    for (int j = threadIdx.x; j < n; j += TH) {
      const u64 place = ls.list[j];
      if (place >= cut && (least <= 0.0 || weight(value_at(place)) >= least))
        atomicAdd(&bq[(index_at(place) + r.lead) / kSampleBlock], mass_of(j, place));
    }
    __syncthreads();
    return true;
  }

  // One step of a search for the place at which, from the top of the order, a
  // target is first reached: the histogram of [lo, hi] (bins of 2^shift
  // places) is in sh.mass and sh.count. reached: the count or mass above hi.
  // Narrows lo and hi to the bin; `am` and `an`: the mass and the count above
  // it. False if the target is not reached.
  __device__ __forceinline__ bool step(bool by_mass, u64 target, u64& lo, u64& hi, int shift, u64& am, u64& an) {
    u64 c0 = 0, m0 = 0, tc, tm;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int bin = kBins - 1 - ((int)threadIdx.x * kBinsPer + i);
      c0 += ls.count[bin], m0 += ls.mass[bin];
    }
    // by mass, the count above is not needed
    tc = 0;
    if (!by_mass) c0 = an + block_scan<TH>(c0, sh.scan64, tc);
    m0 = am + block_scan<TH>(m0, sh.scan64, tm);
    if (uniform(target > (by_mass ? am + tm : an + tc) ? 1 : 0)) return false;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int bin = kBins - 1 - ((int)threadIdx.x * kBinsPer + i);
      const u64 c1 = c0 + ls.count[bin], m1 = m0 + ls.mass[bin];
      if ((by_mass ? m0 : c0) < target && (by_mass ? m1 : c1) >= target) {  // one thread, one bin
        sh.bin = bin;
        sh.a = c0;
        sh.b = m0;
        sh.bin_count = ls.count[bin];
        sh.bin_mass = ls.mass[bin];
      }
      c0 = c1;
      m0 = m1;
    }
    __syncthreads();
    an = uniform(sh.a);
    am = uniform(sh.b);
    const u64 range = hi - lo, bin = (u64)uniform(sh.bin), last = (bin << shift) | ((1ull << shift) - 1);
    hi = lo + (last < range ? last : range);
    lo += bin << shift;
    return true;
  }

  __device__ __forceinline__ void clear_bins() {
    for (int i = threadIdx.x; i < kBins; i += TH) ls.mass[i] = 0, ls.count[i] = 0;
    __syncthreads();
  }
  static __device__ __forceinline__ int shift_of(u64 range) {
    const int bits = 64 - __clzll((long long)(range | 1));
    return bits > 11 ? bits - 11 : 0;
  }

  // Among the listed places from hi to lo the one at which `target` is first
  // reached, which it is; through: the mass up to and with it.
  __device__ __forceinline__ u64 radix(bool by_mass, u64 target, u64 lo, u64 hi, u64& through) {
    u64 am = 0, an = 0;
    const int n = uniform((int)sh.n);
#pragma unroll 1
    for (;;) {
      const int shift = shift_of(hi - lo);
      clear_bins();
#pragma unroll 1
      for (int j = threadIdx.x; j < n; j += TH) {
        const u64 place = ls.list[j];
        if (place >= lo && place <= hi) {
          atomicAdd(&ls.mass[(place - lo) >> shift], mass_of(j, place));
          atomicAdd(&ls.count[(place - lo) >> shift], 1u);
        }
      }
      __syncthreads();
      if (!step(by_mass, target, lo, hi, shift, am, an)) break;
      const int left = uniform((int)sh.bin_count);
      if (threadIdx.x == 0) sh.few = 0;
      __syncthreads();
      if (left <= 64 || !shift) break;
    }
    // the few that are left, each against the others
#pragma unroll 1
    for (int j = threadIdx.x; j < n; j += TH) {
      const u64 place = ls.list[j];
      if (place >= lo && place <= hi) {
        const uint32_t at = atomicAdd(&sh.few, 1u);
        ls.mass[at] = place;
        ls.mass[64 + at] = mass_of(j, place);
      }
    }
    __syncthreads();
    const int few = uniform((int)sh.few);
    if ((int)threadIdx.x < few) {
      const u64 place = ls.mass[threadIdx.x], q = ls.mass[64 + threadIdx.x];
      u64 before = by_mass ? am : an, mass = am;
      for (int j = 0; j < few; ++j)
        if (ls.mass[j] > place) {
          const u64 qj = ls.mass[64 + j];
          before += by_mass ? qj : 1;
          mass += qj;
        }
      if (before < target && before + (by_mass ? q : 1) >= target) sh.place = place, sh.b = mass + q;
    }
    __syncthreads();
    through = uniform(sh.b);
    return uniform(sh.place);
  }

  // Narrows [lo, hi] around the place at which the count or the mass of the
  // row first reaches the target until it can be listed; an: the logits above
  // it. If the target is never reached, to nothing below everything.
  __device__ __forceinline__ void narrow(bool by_mass, u64 target, u64& lo, u64& hi, u64& an) {
    const u64 bottom = lo;
    u64 am = 0;
#pragma unroll 1
    for (;;) {
      const int shift = shift_of(hi - lo);
      clear_bins();
      const int chunks = r.chunks();
#pragma unroll 1
      for (int c = threadIdx.x; c < chunks; c += TH) {
        float z[kChunk];
        r.load(c, z);
        const int e0 = r.first(c);
        for_chunk(z, [&](int k, float x) {
          const u64 place = place_of(Key<T>::of(x), e0 + k);
          if (place >= lo && place <= hi) {
            atomicAdd(&ls.mass[(place - lo) >> shift], quant(weight(x)));
            atomicAdd(&ls.count[(place - lo) >> shift], 1u);
          }
        });
      }
      __syncthreads();
      if (!step(by_mass, target, lo, hi, shift, am, an)) {
        lo = bottom;
        hi = bottom - 1;
        an = 0;
        return;
      }
      const int left = uniform((int)sh.bin_count);
      __syncthreads();
      if (left <= kList) return;
    }
  }

  // Bounds zl (raised) and zh of a neighbourhood of the cut. By count: a zl
  // that t logits reach, give or take four standard deviations of the sample
  // (the list's count tells whether they do). Else of the cut above which a
  // mass of `t` of the row's lies, from a sample of the row in which the mass
  // below the cut is counted from the bottom, where no single logit weighs
  // much. Logits below zl on entry are surely below the cut.
  __device__ __forceinline__ void estimate(bool by_count, u64 t, float& zl, float& zh) {
    const float scale = (float)kBins / (mf - zl), ratef = (float)rate;
    const int chunks = r.chunks(), step = max(1, chunks * kChunk / kEstimate);
    const float rest = 1.f / scale;
    if (threadIdx.x == 0) sh.bin = kBins - 1, sh.bin_count = 0, sh.edge_lo = 0, sh.edge_hi = kBins, sh.low = 0.f;
    clear_bins();
    float low = 0.f;
#pragma unroll 1
    for (int c = threadIdx.x * step; c < chunks; c += TH * step) {
      float z[kChunk];
      r.load(c, z);
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (z[k] >= zl)
          atomicAdd(&ls.count[min(kBins - 1, (int)((z[k] - zl) * scale))], 1u);
        else
          low += __builtin_amdgcn_exp2f((z[k] - mf) * ratef);
    }
    // in any order: the estimate only says where to look
    low = wave_reduce(low, Add());
    if ((threadIdx.x & 63) == 0 && low > 0.f) atomicAdd(&sh.low, low);
    __syncthreads();
    double mass[kBinsPer];
    uint32_t cnt[kBinsPer];
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int bin = threadIdx.x * kBinsPer + i;
      cnt[i] = ls.count[bin];
      mass[i] = (double)cnt[i] * (double)__builtin_amdgcn_exp2f((zl + ((float)bin + 0.5f) * rest - mf) * ratef);
    }
    // counts and masses in one scan: the count in the low 20 bits, the mass
    // above them in units that make the mass sought 2^30 of them, a bin's at
    // most 2^32
    const double lows = (double)sh.low;
    const double below = (S - (double)t / unit) / step - lows;  // of the sample, from zl on
    const double fine = 0x1p30 / fmax(below, 1e-300);
    u64 both[kBinsPer], mine = 0, all;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      both[i] = (u64)fmin(mass[i] * fine, 0x1p32) << 20 | cnt[i];
      mine += both[i];
    }
    u64 run = block_scan<TH>(mine, sh.scan64, all);
    const uint32_t c0 = (uint32_t)run & 0xfffff;
    if (by_count) {
      const float aim = ((float)t + (step > 1 ? 4.f * sqrtf((float)t * (float)step) : 0.f)) / (float)step;
      float left = (float)(((uint32_t)all & 0xfffff) - c0);
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        if (left >= aim && left - (float)cnt[i] < aim) sh.edge_lo = threadIdx.x * kBinsPer + i;
        left -= (float)cnt[i];
      }
      __syncthreads();
      zl += (float)uniform(sh.edge_lo) * rest;
      return;
    }
    if (below > 0.0) {
#pragma unroll
      for (int i = 0; i < kBinsPer; ++i) {
        if ((run >> 20) < 1u << 30 && ((run + both[i]) >> 20) >= 1u << 30) {
          sh.bin = threadIdx.x * kBinsPer + i;
          sh.bin_count = (uint32_t)run & 0xfffff;
        }
        run += both[i];
      }
    } else if (threadIdx.x == 0) {
      sh.bin = 0;
    }
    if (threadIdx.x == 0 && (all >> 20) < 1u << 30) sh.bin_count = (uint32_t)all & 0xfffff;
    uint32_t at;
    __syncthreads();
    // edges: so many of the sample below the cut's bin and above it
    const int around = (int)((kMargin + kAround * sqrtf((float)r.V * (float)(step - 1))) / (float)step);
    const int lo_at = (int)sh.bin_count - around, hi_at = (int)(sh.bin_count + ls.count[sh.bin]) + around;
    at = c0;
#pragma unroll
    for (int i = 0; i < kBinsPer; ++i) {
      const int bin = threadIdx.x * kBinsPer + i;
      if ((int)at <= lo_at && (int)(at + cnt[i]) > lo_at) sh.edge_lo = bin;
      if ((int)at < hi_at && (int)(at + cnt[i]) >= hi_at) sh.edge_hi = bin + 1;
      at += cnt[i];
    }
    __syncthreads();
    const int edge_lo = uniform(sh.edge_lo), edge_hi = uniform(sh.edge_hi);
    if (edge_hi < kBins) zh = zl + (float)edge_hi / scale;
    if (edge_lo > 0) zl += (float)edge_lo / scale;
  }

  // The cut's place, and the blocks' kept masses in bq, which holds the
  // blocks' sums (relative to m) on entry.
  __device__ __forceinline__ u64 cut(int top_k, float top_p, float lowest_max) {
    const bool k_on = top_k > 0 && top_k < r.V, p_on = top_p < 1.f;
    const uint32_t lowest = Key<T>::of(-INFINITY) + 1;  // the least finite key
    const float all = Key<T>::value(lowest);
    float L = all, from = all;
    double goal = 0.0;
    if (!k_on && p_on) {
      goal = (double)top_p * S * unit * (1.0 + 1e-9);
      // with every other logit at most (1 - p) S / (2 x their number), it holds
      from = fmaxf(all, (float)(m + log2((1.0 - (double)fmaxf(top_p, 0.f)) * S / (512.0 * nb)) / rate));
    }
    // In a flat row the bound would not be far above `from`, and the list too
    // long (64 flat rows of 32000 bf16: 37 us against 39 with a bound; of 4000,
    // 21 against 30 when listed; peaked ones pay 0.5 us for the look).
    const bool flat = !k_on && p_on && !peaked();
    if (flat) L = from;
    else if (k_on ? top_k <= nb : p_on) L = bound(lowest_max, k_on, top_k, goal, k_on ? all : from);
    bool whole = false;  // whether what lies below L is cut by min_p, whatever the mass above it
    if (!k_on && least > 0.0) {
      const double z = m + (log2(least) - 1e-6) / rate;  // below it, w < min_p for certain
      uint32_t key = Key<float>::of((float)z);
      if ((double)Key<float>::value(key) > z) --key;
      const float zm = Key<float>::value(key);
      whole = zm >= L;
      L = fmaxf(L, zm);
    }
    L = fmaxf(uniform(L), all);
    int nact = activate(L);
    bool known = !k_on || nact >= top_k;  // a bound for k from the maxima alone
    if (!known && r.V <= kAll) {
      nact = activate(L = all);
      known = true;
    }
    const u64 top = last_place(Key<T>::of(mf)) | kIndexMask;
    u64 place = last_place(lowest), through = 0;
    double mass = S * unit;
    u64 k = k_on ? (u64)top_k : ~0ull;
    bool count = k_on;  // the first k are still to be found
    const bool limits = k_on || p_on;
    // 0: list all candidates; 1: those around an estimate of the cut; 2: narrow
#pragma unroll 1
    for (int method = known && (k_on || !limits || (nact <= kDirect && !flat) || !(L < mf)) ? 0 : 1; method < 3; ++method) {
      if (method == 1 && (k_on ? top_k > kList / 2 : !(L < mf))) continue;
      u64 lo = place, hi = top, an = 0;
      bool one_limit = false;  // k's cut first, then top_p's
      if (method < 2) {
        float zl = L, zh = limits ? INFINITY : L;
        if (method == 1) {
          if (k_on) zl = fmaxf(all, lowest_max - 3.f * (mf - lowest_max));  // where the sample's histogram begins
          estimate(k_on, k_on ? k : needed(top_p, mass), zl, zh);
          if (k_on) nact = activate(zl);
        }
        pass(nact, zl, zh);
        if (!limits) return place;
        // the last place of what is listed: of the least value that is not below zl
        const uint32_t key = Key<T>::of(zl);
        lo = last_place(max(lowest, key + (Key<T>::value(key) < zl)));
        if (zh < INFINITY) hi = last_place(Key<T>::of(zh)) | kIndexMask;  // at or above
        whole = whole && zl == L;
      } else {
        whole = false;
        lo = last_place(lowest);
        one_limit = count && p_on;
        narrow(!count, count ? k : needed(top_p, mass), lo, hi, an);
        pass_places(lo, hi);
      }
      const int n = uniform((int)sh.n);
      const u64 above = uniform(sh.above);
      if (method == 2 && hi < lo) {  // never reached: everything
        if (!one_limit) return lo;
        through = above;
      } else {
        if (n == 0 || n > kList || (method == 1 && k_on && n < top_k)) continue;
        if (!cut_in_list(n, lo, hi, above, k == ~0ull ? k : k - an, count, one_limit ? 1.f : top_p, mass, whole, place,
                         through))
          continue;
        if (!one_limit) return place;
      }
      mass = (double)through;
      count = false;
      method = 1;
      k = ~0ull;
    }
    return place;
  }
};

// Bytes of LDS before the lists. Every part begins at a multiple of its
// elements' size: the lists at one of 16, the blocks' 8-byte sums after Shared.
static_assert(alignof(Lists<>) <= 16 && alignof(Shared) <= 16 && sizeof(Shared) % sizeof(u64) == 0, "LDS alignment");
__host__ __device__ inline size_t shared_bytes(int G) {
  return (sizeof(Shared) + (size_t)G * (sizeof(u64) + sizeof(float) + sizeof(uint16_t)) + 15) / 16 * 16;
}

// The row's blocks from their statistics into LDS, and over them the largest
// logit, the least finite maximum and whether any is NaN.
template <int TH = NT>
__device__ __forceinline__ void load_blocks(Shared& sh, float* bmax, u64* bq, const float* block_max,
                                            const double* block_sum, int nb, float& most, float& lowest_max, int& nan) {
  most = -INFINITY;
  lowest_max = INFINITY;
  nan = 0;
#pragma unroll 1
  for (int b = threadIdx.x; b < nb; b += TH) {
    const float v = block_max[b];
    bmax[b] = v;
    bq[b] = (u64)__double_as_longlong(block_sum[b]);
    nan |= v != v;
    most = fmaxf(most, v);
    if (v > -INFINITY) lowest_max = fminf(lowest_max, v);
  }
  most = wave_reduce(most, Max());
  lowest_max = wave_reduce(lowest_max, Min());
  nan = __ballot(nan) != 0;
  if ((threadIdx.x & 63) == 0) {
    sh.maxw[threadIdx.x >> 6] = most;
    sh.minw[threadIdx.x >> 6] = lowest_max;
    sh.flag[threadIdx.x >> 6] = nan;
  }
  if (threadIdx.x == 0) sh.block = 0x7fffffff, sh.bin = 0x7fffffff;
  __syncthreads();
  constexpr int waves = TH / 64;
  static_assert(waves <= 16, "a row of lanes holds the waves' values");
  most = uniform(row_reduce(sh.maxw[threadIdx.x & (waves - 1)], Max()));
  lowest_max = uniform(row_reduce(sh.minw[threadIdx.x & (waves - 1)], Min()));
  nan = __ballot(sh.flag[threadIdx.x & (waves - 1)]) != 0;
  __syncthreads();
}

// Whether the row has a distribution: no NaN, something above -inf, no +inf,
// and settings that are some.
__device__ __forceinline__ bool has_distribution(float most, int nan, float tau, float top_p, float min_p) {
  return !(nan || !(fabsf(most) < INFINITY) || !(tau >= 0.f && tau < INFINITY) || top_p != top_p || min_p != min_p);
}

// The first of the largest logits: what it is is in sh.bin for every thread.
template <int TH = NT, typename T>
__device__ __forceinline__ void find_first(Shared& sh, const Row<T>& r, const float* bmax, float mf, int nb) {
  for (int b = threadIdx.x; b < nb; b += TH)
    if (bmax[b] == mf) atomicMin(&sh.block, b);
  __syncthreads();
  const int e = sh.block * kSampleBlock - r.lead + (int)threadIdx.x;
  if (threadIdx.x < kSampleBlock && e >= 0 && e < r.V && (float)r.p[e] == mf) atomicMin(&sh.bin, e);
  __syncthreads();
}

// The blocks' sums relative to the row's largest logit, in bq, and over all
// (s.S). NT threads take some blocks each, which lie side by side, or TH the
// parts of several of those: the sum is the same to the last bit.
template <typename T, int TH>
__device__ __forceinline__ void weigh_blocks(RowSampler<T, TH>& s) {
  const int each = (s.nb + NT - 1) / NT;
#pragma unroll 1
  for (int t0 = 0; t0 < NT; t0 += TH) {
    const int b0 = min(s.nb, (t0 + (int)threadIdx.x) * each), b1 = min(s.nb, b0 + each);
    double sum = 0.0, all;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const double w = __longlong_as_double((long long)s.bq[b]) * s.weight(s.bmax[b]);
      s.bq[b] = (u64)__double_as_longlong(w);
      sum += w;
    }
    block_scan<TH>(sum, s.sh.scand, all);
    s.S = t0 ? all + s.S : all;
  }
  s.S = uniform(s.S);
  // q = round(w 2^F) add up to less than 2^52: S < 2^(e+1), and the roundings
  // add at most half of V <= 2^20
  s.unit = uniform(ldexp(1.0, 50 - ilogb(s.S)));
}

}  // namespace

}  // namespace plp
