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
// What limits a row (which value is the cut, how many of it are kept) and at
// which index the sum is exceeded is decided on whole numbers q_i =
// round(w_i 2^F), F chosen so that they add up below 2^52: their sums are
// exact, in whatever order. Two masses are sums in fp64 instead: a block's
// where nothing limits the row, and the whole row's, of which top-p without
// top-k keeps its part. They are added in a fixed order, which with the
// blocks' bounds goes by the row's length and its address modulo 16 bytes, and
// are good to 1e-13 of themselves (twice the exponential's 2e-14, and the
// roundings of some 40 additions): a border that close to u or p times the
// sum is all that a row's address can move.
// w_i is formed in fp64 (2^x by its own polynomial, to 2e-14): at a vocabulary's
// length an fp32 weight's rounding moves the running sum across a token of
// the tail too often.
//
// Two launches: the first reads the logits once and leaves each block of 256
// its maximum and sum; the second, a workgroup a row, finds the cut and the
// token from those and from the blocks that matter.
//
// What bounds them. The first: 16 operations in fp64 a logit, which one SIMD
// issues at 2.2 ns a wave (fp32: 1.3), and the bytes, about evenly: 512 rows
// of 151936 in fp32 take 68 us, of which the fp64 alone would be 42 and a copy
// of their 311 MB takes 58. (64 rows of 151936 bf16 take 12, of which the fp64
// is 5: their 9728 waves, a sixth more than run at once, have four blocks
// each, taken together, and nothing to do while the loads are on the way.)
// The second: the length of one row's chain of steps on one CU, 6 us without
// limits, 14 where the maxima bound the cut (1 row of 151936 bf16, top_k 50),
// 30 to 70 where the row is flat and read twice more; with limits it needs
// all of a CU (128 registers, of which it spills 10 in fp32 and 8 in bf16, and
// 16 waves that meet at every step). Both together: 1 row 17.6 to 18.1 us, 64
// unlimited rows of 151936 bf16 15.7 to 16.6, 128 flat rows of 32000 at top_p
// 0.9 39, 512 rows of 151936 fp32 with settings of their own 142 to 171 (two
// rounds of rows on 256 CUs).
#include "sampling_row.h"

#include <algorithm>

namespace plp {

namespace {

__device__ __forceinline__ float temperature_of(const SampleArgs& a, int64_t row) {
  return a.tau_rows ? a.tau_rows[row] : a.tau;
}

template <typename T>
__global__ __launch_bounds__(kStatThreads) void sample_stats_kernel(SampleArgs a, int G) {
  const int64_t row = blockIdx.y;
  const Row<T> r((const T*)a.logits + row * a.stride, a.V);
  const int lane = threadIdx.x % kStatLanes;
  const int b = blockIdx.x * kStatBlocks + threadIdx.x / kStatLanes;
  if (b >= r.blocks()) return;  // the same for the 16 lanes
  typename Row<T>::Raw raw[kStatChunks];
  fetch_block(r, b, lane, raw);
  float m;
  double s;
  const float tau = temperature_of(a, row);
  block_stats<T>(raw, tau, rate_of(tau), m, s);
  if (lane == 0) {
    a.block_max[row * G + b] = m;
    a.block_sum[row * G + b] = s;
  }
}

template <typename T, bool LIMITS>  // whether there may be any
__global__ __launch_bounds__(NT) void sample_row_kernel(SampleArgs a, int G) {
  extern __shared__ __attribute__((aligned(16))) char lds[];  // 8-byte members and atomics lie in it
  Shared& sh = *reinterpret_cast<Shared*>(lds);
  u64* bq = reinterpret_cast<u64*>(lds + sizeof(Shared));
  float* bmax = reinterpret_cast<float*>(bq + G);
  uint16_t* act = reinterpret_cast<uint16_t*>(bmax + G);
  Lists<>& ls = *reinterpret_cast<Lists<>*>(lds + shared_bytes(G));
  const int64_t row = blockIdx.x;
  const Row<T> r((const T*)a.logits + row * a.stride, a.V);
  const int nb = r.blocks();

  const float tau = temperature_of(a, row);
  const float top_p = a.top_p_rows ? a.top_p_rows[row] : a.top_p;
  const float min_p = a.min_p_rows ? a.min_p_rows[row] : a.min_p;
  const int top_k = a.top_k_rows ? a.top_k_rows[row] : a.top_k;
  float u = a.uniforms[row];

  float mf, lowest_max;
  int nan;
  load_blocks(sh, bmax, bq, a.block_max + row * G, a.block_sum + row * G, nb, mf, lowest_max, nan);
  if (!has_distribution(mf, nan, tau, top_p, min_p) || u != u) {
    if (threadIdx.x == 0) {
      a.token[row] = -1;
      if (a.logp) a.logp[row] = NAN;
      if (a.kept_logp) a.kept_logp[row] = NAN;
    }
    return;
  }
  if (tau == 0.f) {
    find_first(sh, r, bmax, mf, nb);
    if (threadIdx.x == 0) {
      a.token[row] = sh.bin;
      if (a.logp) a.logp[row] = 0.f;
      if (a.kept_logp) a.kept_logp[row] = 0.f;
    }
    return;
  }

  RowSampler<T> s{r, sh, ls, bmax, bq, act, nb, mf, uniform((double)mf), uniform(rate_of(tau)),
                  uniform(least_of(tau)), 0.0, 0.0,
                  uniform(min_p > 0.f ? fmin((double)min_p, 1.0) : -1.0)};
  const int per = (nb + NT - 1) / NT;  // blocks a thread takes, one after the other
  const int b0 = min(nb, (int)threadIdx.x * per), b1 = min(nb, b0 + per);
  weigh_blocks(s);
  u64 cut = 0;
  const bool limited = LIMITS && ((top_k > 0 && top_k < a.V) || top_p < 1.f || min_p > 0.f);
  if (limited) cut = s.cut(top_k, top_p, lowest_max);
  u64 mine = 0, total;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    // a block whose largest logit weighs nothing is left out, so that the
    // block taken holds a token to take
    if (!limited) bq[b] = s.quant(s.weight(bmax[b])) ? s.quant(__longlong_as_double((long long)bq[b])) : 0ull;
    mine += bq[b];
  }
  u64 before = block_scan(mine, sh.scan64, total);
  u = fminf(fmaxf(u, 0.f), 0x1.fffffep-1f);
  const u64 target = (u64)((double)u * (double)total);  // the sum to exceed
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    if (before <= target && before + bq[b] > target) sh.block = b, sh.a = target - before;
    before += bq[b];
  }
  __syncthreads();

  // the index within the block, a thread a logit: the first at which the sum
  // exceeds the target, or, if roundings of the block's own sum leave none,
  // the last that weighs anything
  const int e = sh.block * kSampleBlock - r.lead + (int)threadIdx.x;
  float z = -INFINITY;
  u64 q = 0, all;
  if (threadIdx.x < kSampleBlock && e >= 0 && e < r.V) {
    z = (float)r.p[e] + 0.f;
    if (z > -INFINITY && place_of(Key<T>::of(z), e) >= cut) {
      const double w = s.weight(z);
      if (w >= s.least) q = s.quant(w);
    }
  }
  const u64 inside = sh.a, run = block_scan(q, sh.scan64, all);
  const u64 aim = inside < all ? inside : all - 1;  // all > 0: the block's largest logit weighs something
  if (q && run <= aim && run + q > aim) {
    const double x = ((double)z - (double)mf) / (double)tau;
    a.token[row] = e;
    if (a.logp) a.logp[row] = (float)(x - log(s.S));
    if (a.kept_logp) a.kept_logp[row] = (float)(x - log((double)total / s.unit));
  }
}

template <typename T>
hipError_t sample(const SampleArgs& a, hipStream_t st) {
  const int G = sample_blocks(a.V);
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
    sample_stats_kernel<T>
        <<<dim3((G + kStatBlocks - 1) / kStatBlocks, (unsigned)b.N), kStatThreads, 0, st>>>(b, G);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.top_k_rows || a.top_p_rows || a.min_p_rows || (a.top_k > 0 && a.top_k < a.V) || a.top_p < 1.f || a.min_p > 0.f)
      sample_row_kernel<T, true><<<(unsigned)b.N, NT, shared_bytes(G) + sizeof(Lists<>), st>>>(b, G);
    else
      sample_row_kernel<T, false><<<(unsigned)b.N, NT, shared_bytes(G), st>>>(b, G);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t st) {
  return a.dtype == 0 ? sample<float>(a, st) : sample<__bf16>(a, st);
}

}  // namespace plp
