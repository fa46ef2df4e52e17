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
// masses that are exact or good to 1e-13; sums are added in an order that goes
// by V alone, in blocks of 256 logits from the row's first. What is accepted
// and which token is drawn can so change only where a border lies within about
// 1e-13 of a uniform number.
//
// Four launches: the statistics of every row's blocks and the rows' cuts and
// masses, as in sampling; then the acceptance, which each workgroup decides for
// itself, and the blocks' sums of what is left of the sequence's last row; then
// one workgroup a sequence for the token.
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
  const int64_t row = blockIdx.y;
  const Place at = place_of_row(a, row, per);
  if (!used(a, at)) return;
  const VerifyRows& src = a.of[at.draft];
  const Row<T> r(logits_of<T>(src, at.seq, at.j), a.V);
  const int b = blockIdx.x * kStatBlocks + threadIdx.x / kStatLanes;
  if (b >= r.blocks()) return;  // the same for the 16 lanes
  float m;
  double s;
  block_stats(r, b, threadIdx.x % kStatLanes, src.tau_seq ? src.tau_seq[at.seq] : src.tau, m, s);
  if (threadIdx.x % kStatLanes == 0) {
    a.block_max[row * G + b] = m;
    a.block_sum[row * G + b] = s;
  }
}

// What sampling's row kernel finds before it draws.
template <typename T, bool LIMITS>
__global__ __launch_bounds__(NT) void verify_row_kernel(VerifyArgs a, int per, int G) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Shared& sh = *reinterpret_cast<Shared*>(lds);
  u64* bq = reinterpret_cast<u64*>(lds + sizeof(Shared));
  float* bmax = reinterpret_cast<float*>(bq + G);
  uint16_t* act = reinterpret_cast<uint16_t*>(bmax + G);
  Lists& ls = *reinterpret_cast<Lists*>(lds + shared_bytes(G));
  const int64_t row = blockIdx.x;
  const Place at = place_of_row(a, row, per);
  if (!used(a, at)) return;
  const VerifyRows& src = a.of[at.draft];
  const Row<T> r(logits_of<T>(src, at.seq, at.j), a.V);
  const int nb = r.blocks();
  const float tau = src.tau_seq ? src.tau_seq[at.seq] : src.tau;
  const float top_p = src.top_p_seq ? src.top_p_seq[at.seq] : src.top_p;
  const float min_p = src.min_p_seq ? src.min_p_seq[at.seq] : src.min_p;
  const int top_k = src.top_k_seq ? src.top_k_seq[at.seq] : src.top_k;

  float mf, lowest_max;
  int nan;
  load_blocks(sh, bmax, bq, a.block_max + row * G, a.block_sum + row * G, nb, mf, lowest_max, nan);
  if (!has_distribution(mf, nan, tau, top_p, min_p)) {
    if (threadIdx.x == 0) a.rows[row].state = kNoRow;
    return;
  }
  if (tau == 0.f) {
    find_first(sh, r, bmax, mf, nb);
    if (threadIdx.x == 0) a.rows[row] = VerifyRow{1.0, 1.0, mf, tau, -1.f, 0.f, sh.bin, kOneToken};
    return;
  }
  RowSampler<T> s{r, sh, ls, bmax, bq, act, nb, mf, uniform((double)mf), uniform(rate_of(tau)),
                  uniform(least_of(tau)), 0.0, 0.0,
                  uniform(min_p > 0.f ? fmin((double)min_p, 1.0) : -1.0)};
  const int each = (nb + NT - 1) / NT;
  const int b0 = min(nb, (int)threadIdx.x * each), b1 = min(nb, b0 + each);
  weigh_blocks(s, b0, b1);
  if (LIMITS && ((top_k > 0 && top_k < a.V) || top_p < 1.f || min_p > 0.f)) {
    const u64 cut = s.cut(top_k, top_p, lowest_max);
    u64 mine = 0, total;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += bq[b];
    block_scan(mine, sh.scan64, total);
    if (threadIdx.x == 0)
      a.rows[row] = VerifyRow{(double)total / s.unit, s.S, mf, tau, (float)s.least, s.value_at(cut), index_at(cut), kWeights};
  } else if (threadIdx.x == 0) {
    a.rows[row] = VerifyRow{s.S, s.S, mf, tau, -1.f, -INFINITY, -1, kWeights};
  }
}

// The probability of a row's token e with logit z. The same bits wherever it is
// formed: nothing is contracted.
struct Chance {
  double m, rate, least_d, inv, least;
  float cut;
  int upto, state;
  __device__ explicit Chance(const VerifyRow& r)
      : m((double)r.most),
        rate(rate_of(r.tau)),
        least_d(least_of(r.tau)),
        inv(1.0 / r.mass),
        least((double)r.least),
        cut(r.cut),
        upto(r.upto),
        state(r.state) {}
  __device__ __forceinline__ bool kept(float z, int e) const {
    return state == kOneToken ? e == upto : z > cut || (z == cut && e <= upto);
  }
  __device__ __forceinline__ double of(float z, int e) const {
#pragma clang fp contract(off)
    if (!kept(z, e)) return 0.0;
    if (state == kOneToken) return 1.0;
    const double d = (double)z - m;
    const double w = exp2_of(fmax(d, least_d), rate);
    return w >= least && d >= least_d ? w * inv : 0.0;  // 2^-1000 of the largest, or less, is nothing
  }
};

// Every thread of the workgroup gets the same verdict (`sh`: an int in LDS).
template <typename T>
__device__ __forceinline__ Verdict judge(const VerifyArgs& a, int64_t seq, int per, int* sh) {
  const int n = drafts_of(a, seq);
  const VerifyRow* rows = a.rows + seq * per;
  const float* u = a.uniforms + seq * (a.K + 1);
  if (threadIdx.x == 0) *sh = n;
  __syncthreads();
  for (int k = threadIdx.x; k < n; k += blockDim.x) {
    const int64_t d = a.draft_tokens[seq * a.K + k];
    const bool real = d >= 0 && d < a.V;
    const VerifyRow p = rows[k];
    bool yes = real && p.state != kNoRow && u[k] == u[k];
    if (yes) {
      const double chance = Chance(p).of((float)logits_of<T>(a.of[0], seq, k)[d], (int)d);
      double own = 1.0;
      if (a.of[1].logits) {
        const VerifyRow q = rows[a.K + 1 + k];
        yes = q.state != kNoRow;
        if (yes) own = Chance(q).of((float)logits_of<T>(a.of[1], seq, k)[d], (int)d);
      }
      yes = yes && (double)fminf(fmaxf(u[k], 0.f), 0x1.fffffep-1f) * own < chance;
    }
    if (!yes) atomicMin(sh, k);
  }
  __syncthreads();
  Verdict v;
  v.count = uniform(*sh);
  v.refused = v.count < n ? 1 : 0;
  v.state = rows[v.count].state;
  if (u[a.K] != u[a.K]) v.state = kNoRow;
  if (v.refused) {
    if (u[v.count] != u[v.count]) v.state = kNoRow;
    if (a.of[1].logits && rows[a.K + 1 + v.count].state == kNoRow) v.state = kNoRow;
  }
  return v;
}

// What the last token is drawn from: max(0, p - q), or p.
template <typename T>
struct Rest {
  const T *zp, *zq;  // zq NULL: q is 1 at `certain`, or nothing (-1)
  Chance p, q;
  int certain;
  __device__ Rest(const VerifyArgs& a, int64_t seq, int per, const Verdict& v)
      : zp(logits_of<T>(a.of[0], seq, v.count)),
        zq(v.refused && a.of[1].logits ? logits_of<T>(a.of[1], seq, v.count) : nullptr),
        p(a.rows[seq * per + v.count]),
        q(a.rows[seq * per + (zq ? a.K + 1 + v.count : v.count)]),
        certain(-1) {
    if (v.refused && !a.of[1].logits) {
      const int64_t d = a.draft_tokens[seq * a.K + v.count];
      certain = d >= 0 && d < a.V ? (int)d : -1;
    }
  }
  __device__ __forceinline__ double of(float z, float y, int e) const {
#pragma clang fp contract(off)
    const double chance = p.of(z, e);
    if (chance == 0.0) return 0.0;
    if (zq) return fmax(chance - q.of(y, e), 0.0);
    return e == certain ? 0.0 : chance;
  }
};

constexpr int kRestThreads = 256;
constexpr int kRestBlocks = kRestThreads / 16;  // blocks at a time, 16 lanes each

template <typename T>
__device__ __forceinline__ void load8(const T* p, int e0, int V, float (&z)[kChunk]) {
  typedef T TV __attribute__((ext_vector_type(kChunk), aligned(sizeof(T))));
  if (e0 + kChunk <= V) {
    const TV t = *reinterpret_cast<const TV*>(p + e0);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) z[k] = (float)t[k];
  } else {
#pragma unroll
    for (int k = 0; k < kChunk; ++k) z[k] = e0 + k < V ? (float)p[e0 + k] : -INFINITY;
  }
}

// The sum of a block's chances, in each of its 16 lanes.
template <typename T>
__device__ __forceinline__ double block_rest(const Rest<T>& rest, int b, int lane, int V) {
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = b * kSampleBlock + (c * 16 + lane) * kChunk;
    float z[kChunk], y[kChunk];
    load8(rest.zp, e0, V, z);
    bool any = false;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) any |= rest.p.kept(z[k], e0 + k);
    if (!any) continue;
    if (rest.zq) load8(rest.zq, e0, V, y);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) s += e0 + k < V ? rest.of(z[k], rest.zq ? y[k] : 0.f, e0 + k) : 0.0;
  }
  return row_reduce(s, Add());
}

// The verdict, and the outputs but for the last token.
template <typename T>
__device__ __forceinline__ void say(const VerifyArgs& a, int64_t seq, int per, const Verdict& v) {
  if (threadIdx.x == 0) {
    a.verdicts[seq] = v;
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
  __shared__ int sh;
  const int64_t seq = blockIdx.y;
  const Verdict v = judge<T>(a, seq, per, &sh);
  if (blockIdx.x == 0) say<T>(a, seq, per, v);
  if (v.state == kNoRow) return;
  const Rest<T> rest(a, seq, per, v);
  const int lane = threadIdx.x & 15, end = min(blocks, ((int)blockIdx.x + 1) * each);
  for (int b = blockIdx.x * each + (int)(threadIdx.x >> 4); b < end; b += kRestBlocks) {
    const double s = block_rest(rest, b, lane, a.V);
    if (lane == 0) a.rest[seq * blocks + b] = s;
  }
}

struct Pick {
  double scan[kWaves];
  int first, last;
  double before;
};

template <typename T>
__global__ __launch_bounds__(NT) void verify_pick_kernel(VerifyArgs a, int per, int blocks) {
  __shared__ Pick sh;
  const int64_t seq = blockIdx.x;
  const Verdict v = a.verdicts[seq];
  const int64_t at = seq * (a.K + 1) + v.count;
  if (threadIdx.x == 0) {
    sh.first = 0x7fffffff;
    sh.last = -1;
  }
  if (v.state == kNoRow) {
    if (threadIdx.x == 0) {
      a.tokens[at] = -1;
      if (a.logp) a.logp[at] = NAN;
      if (a.kept_logp) a.kept_logp[at] = NAN;
    }
    return;
  }
  Rest<T> rest(a, seq, per, v);
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
      const double s = block_rest(rest, b, threadIdx.x & 15, a.V);
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
  if (first < 0x7fffffff) atomicMin(&sh.first, first);
  if (last >= 0) atomicMax(&sh.last, last);
  __syncthreads();
  const int block = uniform(sh.first < 0x7fffffff ? sh.first : sh.last);
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
    r = rest.of(z, rest.zq ? (float)rest.zq[e] : 0.f, e);
  }
  double all;
  const double upto = block_scan(r, sh.scan, all) + r;  // its barriers are after the resets
  if (r > 0.0) {
    atomicMax(&sh.last, e);
    if (upto > inside) atomicMin(&sh.first, e);
  }
  __syncthreads();
  if (e == (sh.first < 0x7fffffff ? sh.first : sh.last) && threadIdx.x < kSampleBlock) {
    const VerifyRow row = a.rows[seq * per + v.count];
    float lp = 0.f, kp = 0.f;
    if (row.state == kWeights) {
      const double x = ((double)z - (double)row.most) / (double)row.tau;
      lp = (float)(x - log(row.whole));
      kp = (float)(x - log(row.mass));
    }
    a.tokens[at] = e;
    if (a.logp) a.logp[at] = lp;
    if (a.kept_logp) a.kept_logp[at] = kp;
  }
}

bool limited(const VerifyRows& r, int V) {
  return r.top_k_seq || r.top_p_seq || r.min_p_seq || (r.top_k > 0 && r.top_k < V) || r.top_p < 1.f || r.min_p > 0.f;
}
VerifyRows from(const VerifyRows& r, int64_t seq, size_t esize) {
  VerifyRows o = r;
  if (r.logits) o.logits = (const char*)r.logits + seq * r.seq_stride * (int64_t)esize;
  if (r.tau_seq) o.tau_seq = r.tau_seq + seq;
  if (r.top_p_seq) o.top_p_seq = r.top_p_seq + seq;
  if (r.min_p_seq) o.min_p_seq = r.min_p_seq + seq;
  if (r.top_k_seq) o.top_k_seq = r.top_k_seq + seq;
  return o;
}

template <typename T>
hipError_t verify(const VerifyArgs& all, hipStream_t st) {
  const int G = sample_blocks(all.V), blocks = verify_blocks(all.V);
  const int per = verify_rows(all.K, all.of[1].logits != nullptr);
  const bool limits = limited(all.of[0], all.V) || (all.of[1].logits && limited(all.of[1], all.V));
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
    const unsigned rows = (unsigned)(a.B * per);
    verify_stats_kernel<T><<<dim3((G + kStatBlocks - 1) / kStatBlocks, rows), kStatThreads, 0, st>>>(a, per, G);
    if (hipError_t e = hipGetLastError()) return e;
    if (limits)
      verify_row_kernel<T, true><<<rows, NT, shared_bytes(G) + sizeof(Lists), st>>>(a, per, G);
    else
      verify_row_kernel<T, false><<<rows, NT, shared_bytes(G), st>>>(a, per, G);
    if (hipError_t e = hipGetLastError()) return e;
    // some 2048 workgroups, of whole sets of blocks
    const int sets = (blocks + kRestBlocks - 1) / kRestBlocks;
    const int splits = (int)std::min<int64_t>(sets, std::max<int64_t>(1, 2048 / a.B));
    const int each = (sets + splits - 1) / splits * kRestBlocks;
    verify_rest_kernel<T><<<dim3((blocks + each - 1) / each, (unsigned)a.B), kRestThreads, 0, st>>>(a, per, blocks, each);
    if (hipError_t e = hipGetLastError()) return e;
    verify_pick_kernel<T><<<(unsigned)a.B, NT, 0, st>>>(a, per, blocks);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, hipStream_t st) {
  return a.dtype == 0 ? verify<float>(a, st) : verify<__bf16>(a, st);
}

}  // namespace plp
