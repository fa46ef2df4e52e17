// Verification of drafted tokens against the target's distribution, from given
// uniform numbers.
//
// p_k is the distribution that sampling draws from in target row k (its logits
// under temperature, top-k, top-p and min-p: sampling.hip), q_k the draft's in
// its row k, or 1 at a token that is certain. Draft d_k is accepted if
// u_k q_k(d_k) < p_k(d_k), as long as all before it are. The token after the
// last accepted one comes from max(0, p_k - q_k) where draft k was refused and
// from p_K where none was: the first index at which the running sum exceeds
// the last uniform number times the sum. So every token is distributed as if
// it had been drawn from p.
//
// Probabilities are weights in fp64 (to 2e-14, by sampling's exponential) over
// masses. A whole row's mass is a sum in fp64, good to 1e-13 of itself. A limited
// row's is sampling's sum of whole numbers, each within 2^-51 of the whole mass
// of its weight, equal logits all on the same side; k tokens of V are kept that
// hold k / V of the whole or more, so that it is good to V 2^-51 of itself (7e-11
// at 151936, where one token and 151935 equal ones are off by 4e-11). Weights of
// less than half a unit are none of that mass, but have their chance here, as
// all have down to 2^-1000 of the largest. What is left is added in fp64, in an
// order that goes by V alone, in blocks of 256 logits from the row's first. What
// is accepted and which token is drawn can so differ from the exact
// probabilities' only where a border lies that close to a uniform number, and
// with the row's place in memory only within 1e-13 of one.
//
// Four launches: the statistics of every row's blocks, as in sampling; the
// rows' cuts and masses, and from them the chances of the drafted token; the
// acceptance, which each workgroup decides for itself, and the blocks' sums of
// what is left of the sequence's last row; and one workgroup a sequence for the
// token.
//
// What bounds them: the first by operations in fp64, as in sampling (576 rows of
// 151936 bf16: 67 us, their bytes 30); the second by the length of a row's chain
// of steps on a CU, or half of one, where there are limits (15 us for 9 rows of
// 151936, 43 for some 400 of 32000 with settings of their own), 7 without; the
// third by fp64 again (64 x 2 rows of 151936: 24 us), and 5 for one sequence,
// three loads one after the other; the last by two of them, 5 to 6. 1 x 4 drafts
// at 151936 bf16 take 29 us, 64 x 4 93 to 106 without limits.
#include "sampling_row.h"
#include "verify_ops.h"

namespace plp {

namespace {

// Sequence, and the row's place among its own: targets 0 .. K, drafts from K + 1.
struct Place {
  int64_t seq;
  int j;
  int draft;
};
__device__ __forceinline__ Place place_of_row(const VerifyArgs& a, int64_t row, int per) {
  const int64_t seq = (int64_t)((uint32_t)row / (uint32_t)per);  // rows of one launch: below 2^31
  const int j = (int)(row - seq * per);
  return Place{seq, j > a.K ? j - a.K - 1 : j, j > a.K ? 1 : 0};
}
// The row of workgroup `group` of a launch over rows.
__device__ __forceinline__ Place place_of_group(const VerifyArgs& a, uint32_t group, int per) {
  if (!a.skip) return place_of_row(a, group, per);
  const int place = (int)(group / (uint32_t)a.B), slot = a.slot + place;
  const bool both = a.of[1].logits != nullptr;
  return Place{(int64_t)(group - place * (uint32_t)a.B), both ? slot / 2 : slot, both ? slot % 2 : 0};
}

__device__ __forceinline__ int64_t row_of(const VerifyArgs& a, const Place& p, int per) {
  return p.seq * per + (p.draft ? a.K + 1 : 0) + p.j;
}
__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int64_t seq) {
  return a.num_drafts ? min(max(a.num_drafts[seq], 0), a.K) : a.K;
}
template <typename T>
__device__ __forceinline__ const T* logits_of(const VerifyRows& r, int64_t seq, int j) {
  return (const T*)r.logits + seq * r.seq_stride + j * r.row_stride;
}
// Whether the row is looked at: a target row up to the one after the last draft.
__device__ __forceinline__ bool used(const VerifyArgs& a, const Place& p) {
  const int n = drafts_of(a, p.seq);
  return p.draft ? p.j < n : p.j <= n;
}

template <typename T>
__global__ __launch_bounds__(kStatThreads) void verify_stats_kernel(VerifyArgs a, int per, int G) {
  const Place at = place_of_group(a, blockIdx.y, per);
  if (!used(a, at)) return;
  if (a.slot > 0 && a.refused[at.seq] < at.j) return;  // as far as an earlier launch found
  const int64_t row = row_of(a, at, per);
  if (blockIdx.x == 0 && at.j == 0 && !at.draft) {  // what the next launch says of the sequence's drafts
    if (threadIdx.x == 0) a.refused[at.seq] = a.K;
    for (int k = threadIdx.x; k < 2 * a.K; k += kStatThreads) a.chance[at.seq * a.K * 2 + k] = -1.0;
  }
  const VerifyRows& src = a.of[at.draft];
  const Row<T> r(logits_of<T>(src, at.seq, at.j), a.V);
  const int b = blockIdx.x * kStatBlocks + threadIdx.x / kStatLanes, lane = threadIdx.x % kStatLanes;
  if (b >= r.blocks()) return;  // the same for the 16 lanes
  typename Row<T>::Raw raw[kStatChunks];
  fetch_block(r, b, lane, raw);
  float m;
  double s;
  float tau = src.tau;
  double rate = src.rate;  // (576 rows of 151936: a division in each thread took 4 us more)
  if (src.tau_seq) {
    tau = src.tau_seq[at.seq];
    rate = rate_of(tau);
  }
  block_stats<T>(raw, tau, rate, m, s);
  if (lane == 0) {
    a.block_max[row * G + b] = m;
    a.block_sum[row * G + b] = s;
  }
}

// The probabilities of a row's tokens. Nothing is contracted, so that a token's
// is the same wherever it is formed.
struct Chance {
  double m, rate, inv, least;
  float lowest;      // what weighs 2^-1000 of the largest
  float cut, above;  // kept is what is at or above them, up to index `upto` and past it
  int upto, state;
  __device__ explicit Chance(const VerifyRow& r)
      : m((double)r.most),
        rate(rate_of(r.tau)),
        inv(1.0 / r.mass),
        least((double)r.least),
        lowest(lowest_of(r)),
        cut(fmaxf(r.cut, lowest)),
        above(fmaxf(Key<float>::value(Key<float>::of(r.cut) + 1), lowest)),
        upto(r.upto),
        state(r.state) {}
  // The least value whose distance to the largest exp2_of takes.
  __device__ static __forceinline__ float lowest_of(const VerifyRow& r) {
    const double z = (double)r.most + least_of(r.tau);
    const float f = (float)z;
    return (double)f < z ? Key<float>::value(Key<float>::of(f) + 1) : f;
  }
  // Of N tokens with logits z from e0 on. (What weighs 2^-1000 of the largest,
  // or less, is nothing.) The decisions that are the same for all are made
  // outside the loops, so that these have no branches.
  template <int N>
  __device__ __forceinline__ void of(const float (&z)[N], int e0, double (&chance)[N]) const {
#pragma clang fp contract(off)
    if (state == kOneToken) {
#pragma unroll
      for (int k = 0; k < N; ++k) chance[k] = e0 + k == upto ? 1.0 : 0.0;
      return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) chance[k] = exp2_of((double)fmaxf(z[k], lowest) - m, rate);
    if (least > 0.0)
#pragma unroll
      for (int k = 0; k < N; ++k) chance[k] = chance[k] >= least ? chance[k] : 0.0;
#pragma unroll
    for (int k = 0; k < N; ++k) chance[k] = z[k] >= (e0 + k <= upto ? cut : above) ? chance[k] * inv : 0.0;
  }
  __device__ __forceinline__ double of(float z, int e) const {
    const float one[1] = {z};
    double chance[1];
    of(one, e, chance);
    return chance[0];
  }
  // Whether one of the tokens may have a chance.
  template <int N>
  __device__ __forceinline__ bool any(const float (&z)[N], int e0) const {
    if (state == kOneToken) return e0 <= upto && upto < e0 + N;
    float most = z[0];
#pragma unroll
    for (int k = 1; k < N; ++k) most = fmaxf(most, z[k]);
    return most >= cut;
  }
};

// A number that another workgroup of the launch may look at while this one runs.
__device__ __forceinline__ void publish(double* p, double v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V_>
__device__ __forceinline__ V_ seen(const V_* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether a draft is accepted, of a uniform and the chances of it. (False for NaN.)
__device__ __forceinline__ bool accepts(float u, double own, double chance) {
  return u == u && (double)fminf(fmaxf(u, 0.f), 0x1.fffffep-1f) * own < chance;
}

// The token whose chance is asked for, or -1, and its logit: in LDS, so that no
// registers hold them meanwhile.
struct Drafted {
  int token;
  float logit;
};

// One thread: the row as it was found, and the chance of its drafted token.
__device__ __forceinline__ void leave_row(const VerifyArgs& a, int per, const Drafted& drafted, const VerifyRow& r) {
  const Place at = place_of_group(a, blockIdx.x, per);
  a.rows[row_of(a, at, per)] = r;
  if (at.j >= a.K) return;
  const double mine = r.state == kNoRow ? (double)NAN : drafted.token < 0 ? 0.0 : Chance(r).of(drafted.logit, drafted.token);
  double* const both = a.chance + (at.seq * a.K + at.j) * 2;
  if (!a.skip) {
    both[at.draft] = mine;
    return;
  }
  publish(both + at.draft, mine);
  // the rows after a draft that is refused need not be looked at: an earlier
  // end of the launch, and nothing else, depends on who sees what when
  const double other = a.of[1].logits ? seen(both + (1 - at.draft)) : 1.0;
  if (other < 0.0) return;  // not known yet, or not to this workgroup
  if (!accepts(a.uniforms[at.seq * (a.K + 1) + at.j], at.draft ? mine : other, at.draft ? other : mine))
    __hip_atomic_fetch_min(a.refused + at.seq, at.j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What sampling's row kernel finds before it draws. With `skip` rows go by their
// place in the sequence, the first of all sequences first (a target's row, then
// the draft's): a launch of many more rows than run at once (two a CU, with
// limits) then meets many whose sequence has a draft refused before them, and
// leaves them out. Otherwise a sequence's rows follow each other.
template <typename T, bool LIMITS, int TH>
__global__ __launch_bounds__(TH, 4) void verify_row_kernel(VerifyArgs a, int per, int G) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Shared& sh = *reinterpret_cast<Shared*>(lds);
  u64* bq = reinterpret_cast<u64*>(lds + sizeof(Shared));
  float* bmax = reinterpret_cast<float*>(bq + G);
  uint16_t* act = reinterpret_cast<uint16_t*>(bmax + G);
  Lists<TH>& ls = *reinterpret_cast<Lists<TH>*>(lds + shared_bytes(G));
  __shared__ Drafted drafted;
  const Place at = place_of_group(a, blockIdx.x, per);
  if (!used(a, at)) return;
  const int64_t row = row_of(a, at, per);
  const VerifyRows& src = a.of[at.draft];
  const Row<T> r(logits_of<T>(src, at.seq, at.j), a.V);
  const int nb = r.blocks();
  int refused = a.K, token = -1;
  if (threadIdx.x == 0 && a.skip && at.j > 0) refused = seen(a.refused + at.seq);
  if (threadIdx.x == 0 && at.j < a.K) {
    const int64_t d = a.draft_tokens[at.seq * a.K + at.j];
    token = d >= 0 && d < a.V ? (int)d : -1;
  }
  const float tau = src.tau_seq ? src.tau_seq[at.seq] : src.tau;
  const float top_p = src.top_p_seq ? src.top_p_seq[at.seq] : src.top_p;
  const float min_p = src.min_p_seq ? src.min_p_seq[at.seq] : src.min_p;
  const int top_k = src.top_k_seq ? src.top_k_seq[at.seq] : src.top_k;

  float mf, lowest_max;
  int nan;
  if (a.skip && threadIdx.x == 0) sh.place = (u64)refused;
  load_blocks<TH>(sh, bmax, bq, a.block_max + row * G, a.block_sum + row * G, nb, mf, lowest_max, nan);
  if (a.skip && uniform(sh.place) < (u64)at.j) return;
  if (threadIdx.x == 0) drafted = Drafted{token, token >= 0 ? (float)r.p[token] : 0.f};
  if (!has_distribution(mf, nan, tau, top_p, min_p)) {
    if (threadIdx.x == 0) leave_row(a, per, drafted, VerifyRow{1.0, 1.0, 0.f, 1.f, -1.f, 0.f, -1, kNoRow});
    return;
  }
  if (tau == 0.f) {
    find_first<TH>(sh, r, bmax, mf, nb);
    if (threadIdx.x == 0)
      leave_row(a, per, drafted, VerifyRow{1.0, 1.0, mf, tau, -1.f, 0.f, sh.bin, kOneToken});
    return;
  }
  RowSampler<T, TH> s{r, sh, ls, bmax, bq, act, nb, mf, uniform((double)mf), uniform(rate_of(tau)),
                  uniform(least_of(tau)), 0.0, 0.0,
                  uniform(min_p > 0.f ? fmin((double)min_p, 1.0) : -1.0)};
  weigh_blocks(s);
  VerifyRow out{s.S, s.S, mf, tau, -1.f, -INFINITY, -1, kWeights};
  if (LIMITS && ((top_k > 0 && top_k < a.V) || top_p < 1.f || min_p > 0.f)) {
    const u64 cut = s.cut(top_k, top_p, lowest_max);
    u64 mine = 0, total;
#pragma unroll 1
    for (int b = threadIdx.x; b < nb; b += TH) mine += bq[b];
    block_scan<TH>(mine, sh.scan64, total);
    out = VerifyRow{(double)total / s.unit, s.S, mf, tau, (float)s.least, s.value_at(cut), index_at(cut), kWeights};
  }
  if (threadIdx.x == 0) leave_row(a, per, drafted, out);
}

// Lane l's value of a row.
__device__ __forceinline__ VerifyRow row_of_lane(const VerifyRow& r, int l) {
  return VerifyRow{lane_of(r.mass, l), lane_of(r.whole, l), lane_of(r.most, l), lane_of(r.tau, l),
                   lane_of(r.least, l), lane_of(r.cut, l), lane_of(r.upto, l), lane_of(r.state, l)};
}

// The same verdict in every wave: lane l looks at draft l, and everything that
// may be needed is loaded at once. More drafts than lanes go on in steps.
__device__ __forceinline__ Verdict judge(const VerifyArgs& a, int64_t seq, int per) {
  const int lane = threadIdx.x & 63, n = drafts_of(a, seq);
  const float* u = a.uniforms + seq * (a.K + 1);
  const bool logits = a.of[1].logits != nullptr;
  const float last = u[a.K];
  Verdict v;
  for (int k0 = 0;; k0 += 64) {
    const int k = min(k0 + lane, a.K), kd = min(k, a.K - 1);  // kd: -1 without drafts
    const VerifyRow p = a.rows[seq * per + k];
    VerifyRow q = p;
    double own = 1.0, chance = 0.0;
    int64_t d = -1;
    if (kd >= 0) {
      const double* both = a.chance + (seq * a.K + kd) * 2;
      chance = both[0];
      if (logits) {
        own = both[1];
        q = a.rows[seq * per + a.K + 1 + kd];
      } else {
        d = a.draft_tokens[seq * a.K + kd];
      }
    }
    const float mine = u[k];
    // the first that is refused, or is no draft. Past it rows and chances may
    // not be known, and do not matter.
    const u64 ends = __ballot(k0 + lane >= n || !accepts(mine, own, chance));
    if (!ends) continue;
    const int l = __builtin_ctzll(ends);
    v.count = k0 + l;
    v.refused = v.count < n ? 1 : 0;
    v.p = row_of_lane(p, l);
    v.q = row_of_lane(q, l);
    const int64_t drafted = (int64_t)lane_of((u64)d, l);
    v.certain = v.refused && !logits && drafted >= 0 && drafted < a.V ? (int)drafted : -1;
    const float at = lane_of(mine, l);
    v.state = last != last || (v.refused && (at != at || (logits && v.q.state == kNoRow))) ? kNoRow : v.p.state;
    return v;
  }
}

// What the last token is drawn from: max(0, p - q), or p.
template <typename T>
struct Rest {
  const T *zp, *zq;  // zq NULL: q is 1 at `certain`, or nothing (-1)
  Chance p, q;
  int certain;
  __device__ Rest(const VerifyArgs& a, int64_t seq, const Verdict& v)
      : zp(logits_of<T>(a.of[0], seq, v.count)),
        zq(v.refused && a.of[1].logits ? logits_of<T>(a.of[1], seq, v.count) : nullptr),
        p(v.p),
        q(v.q),
        certain(v.certain) {}
  // What is left of N tokens with logits z and y from e0 on.
  template <int N>
  __device__ __forceinline__ void of(const float (&z)[N], const float (&y)[N], int e0, double (&left)[N]) const {
#pragma clang fp contract(off)
    p.of(z, e0, left);
    if (zq) {
      double own[N];
      q.of(y, e0, own);
#pragma unroll
      for (int k = 0; k < N; ++k) left[k] = fmax(left[k] - own[k], 0.0);
    } else if (certain >= 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) left[k] = e0 + k == certain ? 0.0 : left[k];
    }
  }
};

constexpr int kRestThreads = 256;
constexpr int kRestBlocks = kRestThreads / 16;  // blocks at a time, 16 lanes each

// The logits of a block of both rows that one of its 16 lanes takes, as they lie
// in memory: nothing waits for the loads before they are used.
template <typename T>
struct RestBlock {
  typedef T TV __attribute__((ext_vector_type(kChunk), aligned(sizeof(T))));
  TV z[2], y[2];
  __device__ static __forceinline__ int first(int b, int lane, int c) { return b * kSampleBlock + (c * 16 + lane) * kChunk; }
  __device__ static __forceinline__ TV load8(const T* p, int e0, int V) {
    if (e0 + kChunk <= V) return *reinterpret_cast<const TV*>(p + e0);
    TV t;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) t[k] = e0 + k < V ? p[e0 + k] : (T)-INFINITY;
    return t;
  }
  __device__ __forceinline__ void load(const Rest<T>& rest, int b, int lane, int V) {
#pragma unroll
    for (int c = 0; c < 2; ++c) z[c] = load8(rest.zp, first(b, lane, c), V);
    if (rest.zq)  // uniform
#pragma unroll
      for (int c = 0; c < 2; ++c) y[c] = load8(rest.zq, first(b, lane, c), V);
  }
  // The sum of the block's chances, in each of its 16 lanes. (One copy of the
  // code for both halves: the registers move on.)
  __device__ __forceinline__ double sum(const Rest<T>& rest, int b, int lane) {
    double s = 0.0;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int e0 = first(b, lane, c);
      float zf[kChunk], yf[kChunk];
#pragma unroll
      for (int k = 0; k < kChunk; ++k) zf[k] = (float)z[0][k], yf[k] = (float)y[0][k];
      z[0] = z[1];
      y[0] = y[1];
      if (!__any(rest.p.any(zf, e0))) continue;  // most of a row with limits
      double left[kChunk];
      rest.of(zf, yf, e0, left);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) s += left[k];  // 0 past the row's end
    }
    return row_reduce(s, Add());
  }
};

// The verdict, and the outputs but for the last token.
template <typename T>
__device__ __forceinline__ void say(const VerifyArgs& a, int64_t seq, int per, const Verdict& v) {
  if (threadIdx.x == 0) {
    Verdict w = v;
    w.log_whole = log(v.p.whole);
    w.log_mass = log(v.p.mass);
    a.verdicts[seq] = w;
    a.accepted[seq] = v.count;
  }
  // the accepted drafts, and nothing after the last token
  for (int k = threadIdx.x; k <= a.K; k += kRestThreads) {
    if (k == v.count) continue;
    int64_t token = -1;
    float lp = 0.f, kp = 0.f;
    if (k < v.count) {
      token = a.draft_tokens[seq * a.K + k];
      const VerifyRow r = a.rows[seq * per + k];
      if (r.state == kWeights) {
        const double x = ((double)logits_of<T>(a.of[0], seq, k)[token] - (double)r.most) / (double)r.tau;
        lp = (float)(x - log(r.whole));
        kp = (float)(x - log(r.mass));
      }
    }
    const int64_t at = seq * (a.K + 1) + k;
    a.tokens[at] = token;
    if (a.logp) a.logp[at] = lp;
    if (a.kept_logp) a.kept_logp[at] = kp;
  }
}

template <typename T>
__global__ __launch_bounds__(kRestThreads) void verify_rest_kernel(VerifyArgs a, int per, int blocks, int each) {
  const int64_t seq = blockIdx.y;
  const Verdict v = judge(a, seq, per);
  if (blockIdx.x == gridDim.x - 1) return say<T>(a, seq, per, v);  // none of the blocks are its
  if (v.state == kNoRow) return;
  const Rest<T> rest(a, seq, v);
  const int lane = threadIdx.x & 15, end = min(blocks, ((int)blockIdx.x + 1) * each);
  int b = blockIdx.x * each + (int)(threadIdx.x >> 4);
  if (b >= end) return;  // the same for the 16 lanes
  RestBlock<T> next;
  next.load(rest, b, lane, a.V);
#pragma unroll 1
  for (;;) {
    RestBlock<T> now = next;
    const int then = b + kRestBlocks;
    if (then < end) next.load(rest, then, lane, a.V);
    const double s = now.sum(rest, b, lane);
    if (lane == 0) a.rest[seq * blocks + b] = s;
    if (then >= end) break;
    b = then;
  }
}

struct Pick {
  double scan[kWaves];
  int first, last;
  double before;
};

// The least `first` and the largest `last` of the threads, which both grow with
// the thread, from one lane a wave.
__device__ __forceinline__ void say_ends(Pick& sh, int first, int last) {
  const u64 a = __ballot(first < 0x7fffffff), b = __ballot(last >= 0);
  const int lane = threadIdx.x & 63;
  if (a && lane == __builtin_ctzll(a)) atomicMin(&sh.first, first);
  if (b && lane == 63 - __clzll((long long)b)) atomicMax(&sh.last, last);
}

template <typename T>
__global__ __launch_bounds__(NT) void verify_pick_kernel(VerifyArgs a, int blocks) {
  __shared__ Pick sh;
  const int64_t seq = blockIdx.x;
  const Verdict v = a.verdicts[seq];
  const int64_t at = seq * (a.K + 1) + v.count;
  if (threadIdx.x == 0) {
    sh.first = 0x7fffffff;
    sh.last = -1;
  }
  const auto none = [&] {
    if (threadIdx.x > 0) return;
    a.tokens[at] = -1;
    if (a.logp) a.logp[at] = NAN;
    if (a.kept_logp) a.kept_logp[at] = NAN;
  };
  if (v.state == kNoRow) return none();
  Rest<T> rest(a, seq, v);
  double* sums = a.rest + seq * blocks;
  const int each = (blocks + NT - 1) / NT;
  const int b0 = min(blocks, (int)threadIdx.x * each), b1 = min(blocks, b0 + each);
  double total, before;
  for (int again = 0;; ++again) {
    double mine = 0.0;
    for (int b = b0; b < b1; ++b) mine += sums[b];
    before = block_scan(mine, sh.scan, total);
    if (total > 0.0 || again) break;
    // p is nowhere above q (a draft that neither side could give): the token comes from p
    rest.zq = nullptr;
    rest.certain = -1;
    for (int b = threadIdx.x >> 4; b < blocks; b += NT / 16) {
      RestBlock<T> now;
      now.load(rest, b, threadIdx.x & 15, a.V);
      const double s = now.sum(rest, b, threadIdx.x & 15);
      if ((threadIdx.x & 15) == 0) sums[b] = s;
    }
    __threadfence_block();
    __syncthreads();
  }
  const float u = fminf(fmaxf(a.uniforms[seq * (a.K + 1) + a.K], 0.f), 0x1.fffffep-1f);
  const double target = (double)u * total;
  // the first block whose end exceeds the target; where the sums' roundings
  // leave none, the last that holds anything
  double run = before;
  int first = 0x7fffffff, last = -1;
  for (int b = b0; b < b1; ++b) {
    const double s = sums[b];
    run += s;
    if (s > 0.0) {
      last = b;
      if (run > target) first = min(first, b);
    }
  }
  say_ends(sh, first, last);
  __syncthreads();
  const int block = uniform(sh.first < 0x7fffffff ? sh.first : sh.last);
  if (block < 0) return none();  // no block holds anything: a row with a distribution has one that does
  if (block >= b0 && block < b1) {
    run = before;
    for (int b = b0; b < block; ++b) run += sums[b];
    sh.before = run;
  }
  __syncthreads();
  const double inside = target - sh.before;
  if (threadIdx.x == 0) sh.first = 0x7fffffff, sh.last = -1;
  const int e = block * kSampleBlock + (int)threadIdx.x;
  double r = 0.0;
  float z = 0.f;
  if (threadIdx.x < kSampleBlock && e < a.V) {
    z = (float)rest.zp[e];
    const float one[1] = {z}, other[1] = {rest.zq ? (float)rest.zq[e] : 0.f};
    double left[1];
    rest.of(one, other, e, left);
    r = left[0];
  }
  double all;
  const double upto = block_scan(r, sh.scan, all) + r;  // its barriers are after the resets
  say_ends(sh, r > 0.0 && upto > inside ? e : 0x7fffffff, r > 0.0 ? e : -1);
  __syncthreads();
  const int token = uniform(sh.first < 0x7fffffff ? sh.first : sh.last);
  if (token < 0) return none();
  if (e == token && threadIdx.x < kSampleBlock) {
    const VerifyRow& row = v.p;
    float lp = 0.f, kp = 0.f;
    if (row.state == kWeights) {
      const double x = ((double)z - (double)row.most) / (double)row.tau;
      lp = (float)(x - v.log_whole);
      kp = (float)(x - v.log_mass);
    }
    a.tokens[at] = e;
    if (a.logp) a.logp[at] = lp;
    if (a.kept_logp) a.kept_logp[at] = kp;
  }
}

// Rows with limits above which they look at what is refused before them: twice
// as many as run at once (certain drafts at 32000, top_p 0.95: 1280 rows of 256
// x 4 110 us, 123 without; 2000 of 400 x 4 150 and 184; with the draft's logits
// 1800 of 200 x 4 165 and 174; up to a thousand the same either way, but 672 of 96
// x 3 of ragged numbers 74 in their sequences' order and 80 by their place. Under
// settings of each sequence it pays less: 400 x 8 certain ones 206 and 281, 700 x 8
// with logits 634 and 799, but 256 x 4 of these at 151936 512 and 480).
constexpr unsigned kSkipRows = 1024;

// Launches over rows, so that the statistics of those after a refused draft are
// left out too: the sequences' first rows, then the others, or their first, the
// second and the others. It costs some 7 us a launch and pays by the logits, of
// which certain drafts, mostly refused at once, leave out more (without limits in
// one, two and three: 64 x 4 drafts at 151936 105, 109 and 116 us, 128 x 4 178,
// 172 and 177, 256 x 4 342, 308 and 293 to 304, 512 x 8 at 32000 277, 256 and 245;
// 256 x 4 certain ones at 32000 60, 56 and 63, 512 x 4 114, 90 and 91). With limits
// a launch ends with its last rows' cuts, beside which other rows had been at
// work. Under one setting for all it pays past twice as many logits (256 x 4 at
// 151936, top_p 0.95: 653, 641 and 624, with top_k 50 384, 350 and 337, 700 x 8 at
// 32000 766, 741 and 728; 200 x 4 certain ones at 151936 322, 243 and 275), before
// by the rows of certain drafts (at 32000: 1280 of 256 x 4 108 and 120, 2000 of 400 x
// 4 150 and 146, 2560 of 512 x 4 192 and 171, with top_k 50 155 and 135; of ragged
// numbers, on average half of the rows, 2304 of 256 x 8 117 and 122, 2700 138 and
// 137) and by both where the drafts have logits (at 32000: 2304 rows of 256 x 4 204
// and 212, 3600 294 and 307, but 4608 372 and 367, 7200 587 and 577; 120 x 4 at
// 151936 in fp32 375 and 383). Under settings of each sequence, whose cuts take
// more or less long, it does not where they have (256 x 4 drafts at 151936 534, 597
// and 674, in fp32 and ragged 395, 449 and 515, 100 x 4 180 and 232, 400 x 3 at
// 32000 174 and 199; 700 x 8 665, 652 and 648), and for certain ones by their rows
// alone (200 x 4 at 151936 270, 295 and 329, 512 x 4 at 32000 191, 190 and 205, 400 x
// 8 219, 205 and 218).
constexpr int64_t kStepRows = 2048, kStepLogits = (int64_t)1 << 27;
int steps_of(int64_t rows, int V, bool limits, bool each, bool certain) {
  const int64_t logits = rows * V * (certain ? 2 : 1);
  if (logits > 2 * kStepLogits && !(limits && each)) return certain ? 2 : 3;
  if (!limits) return logits > kStepLogits ? 2 : 1;
  return rows > kStepRows && (certain || (logits > kStepLogits && !each)) ? 2 : 1;
}

bool limited(const VerifyRows& r, int V) {
  return r.top_k_seq || r.top_p_seq || r.min_p_seq || (r.top_k > 0 && r.top_k < V) || r.top_p < 1.f || r.min_p > 0.f;
}
bool of_each(const VerifyRows& r) { return r.tau_seq || r.top_k_seq || r.top_p_seq || r.min_p_seq; }
VerifyRows from(const VerifyRows& r, int64_t seq, size_t esize) {
  VerifyRows o = r;
  o.rate = rate_of(r.tau);
  if (r.logits) o.logits = (const char*)r.logits + seq * r.seq_stride * (int64_t)esize;
  if (r.tau_seq) o.tau_seq = r.tau_seq + seq;
  if (r.top_p_seq) o.top_p_seq = r.top_p_seq + seq;
  if (r.min_p_seq) o.min_p_seq = r.min_p_seq + seq;
  if (r.top_k_seq) o.top_k_seq = r.top_k_seq + seq;
  return o;
}

// Rows up to which each has a CU and its workgroup all threads it can have;
// above, half of them, and two workgroups a CU. At 151936 bf16 and top_p 0.95
// 24 x 4 drafts (216 rows) take 102 us with all, 114 with half; 28 x 4 (252 rows)
// 111 and 121; 32 x 4 (288 rows) 160 and 143; at 32000 256 x 4 279 and 216. (A
// quarter of the threads, two a CU all the same for what their lists take of its
// LDS: 242.)
constexpr unsigned kFewRows = 256;

template <typename T, int TH>
hipError_t row_kernel(const VerifyArgs& a, int per, int G, unsigned rows, bool limits, hipStream_t st) {
  if (limits)
    verify_row_kernel<T, true, TH><<<rows, TH, shared_bytes(G) + sizeof(Lists<TH>), st>>>(a, per, G);
  else
    verify_row_kernel<T, false, TH><<<rows, TH, shared_bytes(G), st>>>(a, per, G);
  return hipGetLastError();
}

template <typename T>
hipError_t verify(const VerifyArgs& all, hipStream_t st) {
  const int G = sample_blocks(all.V), blocks = verify_blocks(all.V);
  const int per = verify_rows(all.K, all.of[1].logits != nullptr);
  const bool limits = limited(all.of[0], all.V) || (all.of[1].logits && limited(all.of[1], all.V));
  const bool each_own = of_each(all.of[0]) || (all.of[1].logits && of_each(all.of[1]));
  const int64_t most = std::max(1, 32768 / per);  // the grid's second dimension holds 65535
  for (int64_t s0 = 0; s0 < all.B; s0 += most) {
    VerifyArgs a = all;
    a.B = std::min(most, all.B - s0);
    a.of[0] = from(all.of[0], s0, sizeof(T));
    a.of[1] = from(all.of[1], s0, sizeof(T));
    a.draft_tokens = all.draft_tokens + s0 * all.K;
    if (all.num_drafts) a.num_drafts = all.num_drafts + s0;
    a.uniforms = all.uniforms + s0 * (all.K + 1);
    a.tokens = all.tokens + s0 * (all.K + 1);
    a.accepted = all.accepted + s0;
    if (all.logp) a.logp = all.logp + s0 * (all.K + 1);
    if (all.kept_logp) a.kept_logp = all.kept_logp + s0 * (all.K + 1);
    const int places = all.of[1].logits ? 2 : 1, steps = steps_of(a.B * per, a.V, limits, each_own, places == 1);
    a.skip = steps > 1 || (limits && a.B * per > kSkipRows);
    // all rows at once, or the first of each sequence, its second and so on and then the others
    for (int from = 0, to; from <= a.K; from = to + 1) {
      to = std::min(a.K, from < steps - 1 ? from : a.K);
      a.slot = from * places;
      const unsigned rows = (unsigned)(a.B * ((to - from + 1) * places - (places == 2 && to == a.K ? 1 : 0)));
      verify_stats_kernel<T><<<dim3((G + kStatBlocks - 1) / kStatBlocks, rows), kStatThreads, 0, st>>>(a, per, G);
      if (hipError_t e = hipGetLastError()) return e;
      hipError_t e = rows > kFewRows ? row_kernel<T, kHalfNT>(a, per, G, rows, limits, st)
                                     : row_kernel<T, NT>(a, per, G, rows, limits, st);
      if (e) return e;
    }
    // some 2048 workgroups, of whole sets of blocks
    const int sets = (blocks + kRestBlocks - 1) / kRestBlocks;
    const int splits = (int)std::min<int64_t>(sets, std::max<int64_t>(1, 2048 / a.B));
    const int each = (sets + splits - 1) / splits * kRestBlocks;
    verify_rest_kernel<T><<<dim3((blocks + each - 1) / each + 1, (unsigned)a.B), kRestThreads, 0, st>>>(a, per, blocks, each);
    if (hipError_t e = hipGetLastError()) return e;
    verify_pick_kernel<T><<<(unsigned)a.B, NT, 0, st>>>(a, blocks);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, hipStream_t st) {
  return a.dtype == 0 ? verify<float>(a, st) : verify<__bf16>(a, st);
}

}  // namespace plp
