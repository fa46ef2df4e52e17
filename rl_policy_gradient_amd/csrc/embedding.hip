// Embedding lookup and its gradient.
//
//   forward   y_n = round(scale weight[t_n]), zeros where t_n is no row
//   backward  grad_weight_v = round((old +) scale sum over t_n = v of grad_y_n)
//
// The backward pass sorts the tokens (stably, so that equal ones keep their
// order) and then adds rows that lie side by side in the sorted order: sums in
// fp32 in the order of n, no atomics on them, one rounding.
//
// Sorting: up to kCountingN tokens by counting, for each, the tokens before
// it; more by passes of a radix sort, least digit first, with at most 256
// workgroups a pass.
//
// Adding: the work is a merge of V row ends (each writes a row of grad_weight)
// with N sorted tokens (each reads a row of grad_y); a wave takes an equal
// range of the merged order, for 64 lanes' columns, whatever the tokens'
// frequencies. With `accumulate` rows without tokens are left alone and only
// the tokens are cut into ranges. A row whose tokens lie in several ranges is
// added up by a last kernel from their partial sums, in their order.
#include "training_ops.h"

#include <algorithm>

namespace plp {

namespace {

// ---- rows --------------------------------------------------------------------

// N consecutive elements at any element's address.
template <typename T, int N>
struct VecOf {
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// Elements d .. d + V - 1 of a row of H, those past its end as 0.
template <typename T, int V>
__device__ __forceinline__ typename VecOf<T, V>::type load_raw(const T* row, int d, int H) {
  typedef typename VecOf<T, V>::type TV;
  if (d + V <= H) return *reinterpret_cast<const TV*>(row + d);
  TV t = {};
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (d + k < H) t[k] = row[d + k];
  return t;
}
template <typename T, int V>
__device__ __forceinline__ void load_part(const T* row, int d, int H, float (&x)[V]) {
  const auto t = load_raw<T, V>(row, d, H);
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] = (float)t[k];
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T* row, int d, int H, const float (&x)[V]) {
  typedef typename VecOf<T, V>::type TV;
  if (d + V <= H) {
    TV t;
#pragma unroll
    for (int k = 0; k < V; ++k) t[k] = (T)x[k];
    *reinterpret_cast<TV*>(row + d) = t;
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (d + k < H) row[d + k] = (T)x[k];
  }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- forward -----------------------------------------------------------------

constexpr int kFwdRows = 4;  // rows a wave has in flight

template <typename T>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedFwd a, uint32_t slices, uint32_t units) {
  constexpr int V = 16 / (int)sizeof(T);
  const uint32_t unit = blockIdx.x * 4 + uniform(threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t n0 = (int64_t)(unit / slices) * kFwdRows;
  const int d = (int)(unit % slices * 64 + (threadIdx.x & 63)) * V;
  if (d >= a.H) return;
  typename VecOf<T, V>::type x[kFwdRows];
  int64_t t[kFwdRows];
#pragma unroll
  for (int r = 0; r < kFwdRows; ++r) t[r] = n0 + r < a.N ? a.tokens[n0 + r] : -1;
#pragma unroll
  for (int r = 0; r < kFwdRows; ++r) {
    x[r] = {};
    if (t[r] >= 0 && t[r] < a.V) x[r] = load_raw<T, V>((const T*)a.weight + t[r] * a.H, d, a.H);
  }
#pragma unroll
  for (int r = 0; r < kFwdRows; ++r) {
    if (n0 + r >= a.N) break;
    float y[V];
#pragma unroll
    for (int k = 0; k < V; ++k) y[k] = (float)x[r][k] * a.scale;
    store_part<T, V>((T*)a.y + (n0 + r) * a.H, d, a.H, y);
  }
}

// ---- sorting -----------------------------------------------------------------

// A token as a key; what is no row comes after every row.
__device__ __forceinline__ uint32_t key_of(int64_t t, int V) { return t >= 0 && t < V ? (uint32_t)t : (uint32_t)V; }

constexpr int kCountingN = 4096;
constexpr int kCountItems = 64;  // tokens a workgroup places, four threads each

__global__ __launch_bounds__(256) void sort_counting_kernel(const int64_t* __restrict__ tokens, int N, int V,
                                                            uint32_t* __restrict__ key, uint32_t* __restrict__ pos) {
  __shared__ __attribute__((aligned(16))) uint32_t all[kCountingN];
  const int padded = (N + 15) / 16 * 16;  // up to kCountingN
  for (int i = threadIdx.x; i < padded; i += 256) all[i] = i < N ? key_of(tokens[i], V) : 0xffffffffu;
  __syncthreads();
  const int part = threadIdx.x & 3, i = blockIdx.x * kCountItems + (int)(threadIdx.x >> 2);
  const uint32_t mine = all[i < N ? i : 0];
  int before = 0;
  for (int j = part * 4; j < padded; j += 16) {
    const uint4 k = *reinterpret_cast<const uint4*>(all + j);
    before += k.x < mine || (k.x == mine && j < i);
    before += k.y < mine || (k.y == mine && j + 1 < i);
    before += k.z < mine || (k.z == mine && j + 2 < i);
    before += k.w < mine || (k.w == mine && j + 3 < i);
  }
  before += __shfl_xor(before, 1, 64);
  before += __shfl_xor(before, 2, 64);
  if (part == 0 && i < N) {
    key[before] = mine;
    pos[before] = (uint32_t)i;
  }
}

constexpr int kMaxBits = 10;
constexpr int kRadixWaves = 8, kRadixThreads = kRadixWaves * 64;

// Counts of a pass's digits in each workgroup's tokens; clears the next pass's.
__global__ __launch_bounds__(kRadixThreads) void radix_count_kernel(const int64_t* __restrict__ tokens, int64_t N, int V,
                                                                    int bits, int64_t per, uint32_t* __restrict__ hist,
                                                                    uint32_t* __restrict__ next) {
  __shared__ uint32_t count[1 << kMaxBits];
  const int digits = 1 << bits;
  for (int d = threadIdx.x; d < digits; d += kRadixThreads) count[d] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * per, end = begin + per < N ? begin + per : N;
  for (int64_t i = begin + threadIdx.x; i < end; i += kRadixThreads)
    atomicAdd(&count[key_of(tokens[i], V) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kRadixThreads) {
    hist[(int64_t)blockIdx.x * digits + d] = count[d];
    next[(int64_t)blockIdx.x * digits + d] = 0;
  }
}

struct RadixPass {
  const int64_t* tokens;      // the first pass's input
  const uint32_t *key, *pos;  // the others'
  uint32_t *key_out, *pos_out;
  const uint32_t* hist;
  uint32_t *next, *after;  // the next pass's counts; those of the one after it, to be cleared (either may be NULL)
  int64_t N, per;
  int V, bits, shift, blocks;
};

// Moves a workgroup's tokens to their places by the pass's digit, each wave's
// in their order, and counts the next pass's digits by the places' workgroups
// (whole numbers, so that the order of the additions does not matter).
__global__ __launch_bounds__(kRadixThreads) void radix_move_kernel(RadixPass a) {
  __shared__ uint32_t at[kRadixWaves][1 << kMaxBits];
  __shared__ uint32_t wave_total[kRadixWaves];
  const int digits = 1 << a.bits, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t begin = blockIdx.x * a.per, end = begin + a.per < a.N ? begin + a.per : a.N;
  const int64_t each = (a.per + kRadixWaves - 1) / kRadixWaves;
  const int64_t w0 = begin + wave * each < end ? begin + wave * each : end, w1 = w0 + each < end ? w0 + each : end;
  const auto key_at = [&](int64_t i) { return a.tokens ? key_of(a.tokens[i], a.V) : a.key[i]; };
  for (int d = threadIdx.x; d < kRadixWaves * digits; d += kRadixThreads) at[d / digits][d % digits] = 0;
  __syncthreads();
  for (int64_t i = w0 + lane; i < w1; i += 64) atomicAdd(&at[wave][key_at(i) >> a.shift & (digits - 1)], 1u);
  // where each digit begins in this workgroup: all smaller digits, and the same in the workgroups before
  constexpr int per_thread = (1 << kMaxBits) / kRadixThreads;
  uint32_t total[per_thread], before[per_thread], sum = 0;
#pragma unroll
  for (int k = 0; k < per_thread; ++k) {
    const int d = (int)threadIdx.x * per_thread + k;
    total[k] = before[k] = 0;
    if (d >= digits) continue;
#pragma unroll 8
    for (int b = 0; b < a.blocks; ++b) {
      const uint32_t c = a.hist[(int64_t)b * digits + d];
      total[k] += c;
      before[k] += b < (int)blockIdx.x ? c : 0;
    }
    sum += total[k];
  }
  uint32_t run = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(run, o, 64);
    run += lane >= o ? v : 0;
  }
  if (lane == 63) wave_total[wave] = run;
  __syncthreads();  // the waves' counts are whole, too
  run -= sum;
  for (int w = 0; w < wave; ++w) run += wave_total[w];
#pragma unroll
  for (int k = 0; k < per_thread; ++k) {
    const int d = (int)threadIdx.x * per_thread + k;
    if (d >= digits) break;
    uint32_t place = run + before[k];
    run += total[k];
#pragma unroll
    for (int w = 0; w < kRadixWaves; ++w) {
      const uint32_t c = at[w][d];
      at[w][d] = place;
      place += c;
    }
  }
  if (a.after)
    for (int d = threadIdx.x; d < digits; d += kRadixThreads) a.after[(int64_t)blockIdx.x * digits + d] = 0;
  __syncthreads();
  for (int64_t i0 = w0; i0 < w1; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool in = i < w1;
    const uint32_t key = in ? key_at(i) : 0;
    const uint32_t pos = in ? (a.tokens ? (uint32_t)i : a.pos[i]) : 0;
    const uint32_t digit = key >> a.shift & (digits - 1);
    uint64_t same = __ballot(in);
    for (int k = 0; k < a.bits; ++k) {
      const uint64_t set = __ballot(digit >> k & 1);
      same &= digit >> k & 1 ? set : ~set;
    }
    if (in) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const uint32_t place = at[wave][digit] + rank;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // all have read before the first writes
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) at[wave][digit] = place + __popcll(same);
      a.key_out[place] = key;
      a.pos_out[place] = pos;
      if (a.next) atomicAdd(&a.next[(int64_t)(place / (uint32_t)a.per) * digits + (key >> (a.shift + a.bits) & (digits - 1))], 1u);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- adding ------------------------------------------------------------------

// Of the first d steps of the merge of N sorted keys with the row ends 0, 1,
// .. V - 1 (a row's end comes after its keys) how many are keys. A wave's
// search: each step leaves a 64th.
__device__ __forceinline__ int64_t keys_before(const uint32_t* __restrict__ key, int64_t N, int V, int64_t d, int lane) {
  int64_t lo = d > V ? d - V : 0, hi = d < N ? d : N;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64, i = lo + lane * step;
    const bool is = i < hi && (int64_t)key[i] <= d - 1 - i;
    const int n = __popcll(__ballot(is));
    if (n == 0) break;
    const int64_t upto = lo + n * step;
    lo += (n - 1) * step + 1;
    hi = upto < hi ? upto : hi;
  }
  return lo;
}

constexpr int kAddWaves = 4;
constexpr int kBatch = 8;  // rows of grad_y a wave has in flight

template <typename TG>
constexpr int add_vec = 16 / (int)sizeof(TG);  // columns a lane takes

template <typename TG, typename TW>
__global__ __launch_bounds__(kAddWaves * 64) void embed_add_kernel(EmbedBwd a, const uint32_t* __restrict__ key,
                                                                   const uint32_t* __restrict__ pos, uint32_t slices,
                                                                   int items, uint32_t ranges) {
  constexpr int V = add_vec<TG>;
  const int lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x * kAddWaves + uniform(threadIdx.x >> 6);
  const int64_t range = unit / slices;
  if (range >= ranges) return;
  const int slice = (int)(unit % slices), d = (slice * 64 + lane) * V;
  const bool in = d < a.H;
  int64_t i0, i1;
  int v, v1;  // the row at the range's start, and at its end
  if (a.accumulate) {
    i0 = range * items;
    i1 = i0 + items < a.N ? i0 + items : a.N;
    v = (int)key[i0];
    v1 = i1 < a.N ? (int)key[i1] : a.V;
  } else {
    const int64_t all = a.N + a.V, d0 = range * items, d1 = d0 + items < all ? d0 + items : all;
    i0 = keys_before(key, a.N, a.V, d0, lane);
    i1 = keys_before(key, a.N, a.V, d1, lane);
    v = (int)(d0 - i0);
    v1 = (int)(d1 - i1);
  }
  const int v0 = v;
  const bool shared = i0 > 0 && (int)key[i0 - 1] == v0;  // the first row's tokens begin in another range
  float sum[V];
  bool any = false;
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.f;
  TW* const w = (TW*)a.grad_weight;
  const auto end_row = [&]() {  // of row v
    if (shared && v == v0) {
      if (in) store_part<float, V>(a.head + range * a.H, d, a.H, sum);
    } else if (in && (any || !a.accumulate)) {
      float x[V];
      if (a.accumulate) {
        load_part<TW, V>(w + (int64_t)v * a.H, d, a.H, x);
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] += a.scale * sum[k];
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = a.scale * sum[k];
      }
      store_part<TW, V>(w + (int64_t)v * a.H, d, a.H, x);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] = 0.f;
    any = false;
  };
  for (int64_t b0 = i0; b0 < i1; b0 += 64) {
    const int64_t mine = b0 + lane < i1 ? b0 + lane : i1 - 1;
    const int keys = (int)key[mine], rows = (int)pos[mine];
    const int left = (int)(i1 - b0 < 64 ? i1 - b0 : 64);
    bool done = false;
    for (int j0 = 0; j0 < left && !done; j0 += kBatch) {
      typename VecOf<TG, V>::type x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int l = j0 + j < left ? j0 + j : left - 1;
        const int64_t row = (uint32_t)__builtin_amdgcn_readlane(rows, l);
        if (in) x[j] = load_raw<TG, V>((const TG*)a.grad_y + row * a.H, d, a.H);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (j0 + j >= left) break;
        const int k = __builtin_amdgcn_readlane(keys, j0 + j);
        if (k >= a.V) {  // no row, and nothing but those from here on
          done = true;
          break;
        }
        if (a.accumulate && v < k) {
          end_row();
          v = k;
        }
        for (; v < k; ++v) end_row();
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += (float)x[j][e];
        any = true;
      }
    }
    if (done) break;
  }
  if (a.accumulate && v < v1) {
    end_row();
    v = v1;
  }
  for (; v < v1; ++v) end_row();
  if (any && in) store_part<float, V>(a.tail + range * a.H, d, a.H, sum);
  if (slice == 0 && lane == 0) {
    a.head_row[range] = shared && v1 > v0 && v0 < a.V ? v0 : -1;
    a.tail_row[range] = any ? v : -1;
  }
}

constexpr int kJoinWaves = 8;
constexpr int kJoinAlone = 32;  // partial sums that one wave adds by itself

// The rows that several ranges share: those that end in a range and began in
// an earlier one. A wave adds the partial sums of one (64 lanes' columns), or
// all of the workgroup's waves do, one row after the other, where they are many.
template <typename TG, typename TW>
__global__ __launch_bounds__(kJoinWaves * 64) void embed_join_kernel(EmbedBwd a, uint32_t slices, uint32_t ranges) {
  constexpr int V = add_vec<TG>;
  __shared__ float part[kJoinWaves][64][V + 1];
  __shared__ int many[kJoinWaves];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t unit0 = blockIdx.x * kJoinWaves;
  // the ranges before `range` that hold a partial sum of row `row`, up to `most` of them
  const auto chain = [&](int64_t range, int row, int64_t most) {
    int64_t n = 0;
    for (;;) {
      const int64_t k = range - 1 - n - lane;
      const uint64_t other = __ballot(!(k >= 0 && a.tail_row[k < 0 ? 0 : k] == row));
      n += other ? __builtin_ctzll(other) : 64;
      if (other || n >= most) return n;
    }
  };
  const auto add = [&](int64_t from, int64_t to, int d, float(&sum)[V]) {
#pragma unroll 4
    for (int64_t k = from; k < to; ++k) {
      float x[V];
      load_part<float, V>(a.tail + k * a.H, d, a.H, x);
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] += x[e];
    }
  };
  const auto finish = [&](int64_t range, int row, int d, float(&sum)[V]) {
    TW* const w = (TW*)a.grad_weight + (int64_t)row * a.H;
    float x[V];
    load_part<float, V>(a.head + range * a.H, d, a.H, x);
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = a.scale * (sum[e] + x[e]);
    if (a.accumulate) {
      load_part<TW, V>(w, d, a.H, x);
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] += x[e];
    }
    store_part<TW, V>(w, d, a.H, sum);
  };
  bool long_one = false;
  {
    const uint32_t unit = unit0 + wave;
    const int64_t range = unit / slices;
    const int row = range < ranges ? a.head_row[range] : -1;
    if (row >= 0) {
      const int64_t n = chain(range, row, kJoinAlone + 1);
      const int d = ((int)(unit % slices) * 64 + lane) * V;
      long_one = n > kJoinAlone;
      if (!long_one && d < a.H) {
        float sum[V] = {};
        add(range - n, range, d, sum);
        finish(range, row, d, sum);
      }
    }
  }
  if (lane == 0) many[wave] = long_one;
  __syncthreads();
  for (int u = 0; u < kJoinWaves; ++u) {
    if (!many[u]) continue;  // the same for all threads
    const uint32_t unit = unit0 + u;
    const int64_t range = unit / slices;
    const int row = a.head_row[range], d = ((int)(unit % slices) * 64 + lane) * V;
    const int64_t n = chain(range, row, range), first = range - n, each = (n + kJoinWaves - 1) / kJoinWaves;
    const int64_t from = first + wave * each < range ? first + wave * each : range;
    float sum[V] = {};
    if (d < a.H) add(from, from + each < range ? from + each : range, d, sum);
#pragma unroll
    for (int e = 0; e < V; ++e) part[wave][lane][e] = sum[e];
    __syncthreads();
    if (wave == 0 && d < a.H) {
      for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += part[w][lane][e];
      finish(range, row, d, sum);
    }
    __syncthreads();
  }
}

// The gradient where there are no tokens.
__global__ __launch_bounds__(256) void embed_zero_kernel(uint32_t* p, int64_t words, uint16_t* rest) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += step) p[i] = 0;
  if (rest && blockIdx.x == 0 && threadIdx.x == 0) *rest = 0;
}

int slices_of(int H, int dtype) {
  const int lanes = 64 * (dtype == 0 ? 4 : 8);
  return (H + lanes - 1) / lanes;
}

template <typename TG, typename TW>
hipError_t add_rows(const EmbedBwd& a, const EmbedBwdPlan& p, const uint32_t* key, const uint32_t* pos, hipStream_t st) {
  const int64_t units = p.ranges * p.slices;
  embed_add_kernel<TG, TW><<<(unsigned)((units + kAddWaves - 1) / kAddWaves), kAddWaves * 64, 0, st>>>(
      a, key, pos, p.slices, p.items, (uint32_t)p.ranges);
  if (hipError_t e = hipGetLastError()) return e;
  embed_join_kernel<TG, TW><<<(unsigned)((units + kJoinWaves - 1) / kJoinWaves), kJoinWaves * 64, 0, st>>>(
      a, p.slices, (uint32_t)p.ranges);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedFwd& a, hipStream_t st) {
  const int slices = slices_of(a.H, a.dtype);
  const int64_t units = (a.N + kFwdRows - 1) / kFwdRows * slices;
  // a launch holds fewer than 2^32 threads
  const int64_t most = ((int64_t)1 << 23) / slices * slices;
  const size_t e = a.dtype == 0 ? 4 : 2;
  for (int64_t u = 0; u < units; u += most) {
    EmbedFwd b = a;
    const int64_t n0 = u / slices * kFwdRows, some = std::min(most, units - u);
    b.tokens = a.tokens + n0;
    b.y = (char*)a.y + (size_t)n0 * a.H * e;
    b.N = a.N - n0;
    const unsigned grid = (unsigned)((some + 3) / 4);
    if (a.dtype == 0)
      embed_fwd_kernel<float><<<grid, 256, 0, st>>>(b, slices, (uint32_t)some);
    else
      embed_fwd_kernel<__bf16><<<grid, 256, 0, st>>>(b, slices, (uint32_t)some);
    if (hipError_t err = hipGetLastError()) return err;
  }
  return hipSuccess;
}

EmbedBwdPlan embed_bwd_plan(int64_t N, int H, int V, int grad_y_dtype, bool accumulate) {
  EmbedBwdPlan p{};
  p.radix = N > kCountingN;
  int bits = 1;
  while ((int64_t)V >> bits) ++bits;  // keys are 0 .. V
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.blocks = (int)std::min<int64_t>(256, (N + 1023) / 1024);
  p.per = p.blocks ? (N + p.blocks - 1) / p.blocks : 0;
  p.slices = slices_of(H, grad_y_dtype);
  // some 16384 waves (eight rounds of what runs at once), but no range of fewer than 16
  const int64_t work = accumulate ? N : N + V;
  const int64_t most = std::max<int64_t>(1, 16384 / p.slices);
  p.items = (int)std::max<int64_t>(16, (work + most - 1) / most);
  p.ranges = (work + p.items - 1) / p.items;
  return p;
}

hipError_t launch_embed_bwd(const EmbedBwd& a, hipStream_t st) {
  if (a.N == 0) {
    if (a.accumulate) return hipSuccess;
    const int64_t bytes = (int64_t)a.V * a.H * (a.grad_weight_dtype == 0 ? 4 : 2);
    char* p = (char*)a.grad_weight;
    const int64_t head = (uintptr_t)p % 4;  // 0 or 2
    const int64_t words = (bytes - head) / 4;
    if (head) {
      embed_zero_kernel<<<1, 256, 0, st>>>(nullptr, 0, (uint16_t*)p);
      if (hipError_t e = hipGetLastError()) return e;
    }
    uint16_t* rest = bytes - head - words * 4 ? (uint16_t*)(p + head + words * 4) : nullptr;
    embed_zero_kernel<<<2048, 256, 0, st>>>((uint32_t*)(p + head), words, rest);
    return hipGetLastError();
  }
  const EmbedBwdPlan p = embed_bwd_plan(a.N, a.H, a.V, a.grad_y_dtype, a.accumulate);
  int at = 0;
  if (!p.radix) {
    sort_counting_kernel<<<(unsigned)((a.N + kCountItems - 1) / kCountItems), 256, 0, st>>>(a.tokens, (int)a.N, a.V,
                                                                                           a.key[0], a.pos[0]);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    radix_count_kernel<<<p.blocks, kRadixThreads, 0, st>>>(a.tokens, a.N, a.V, p.bits, p.per, a.hist[0], a.hist[1]);
    if (hipError_t e = hipGetLastError()) return e;
    for (int i = 0; i < p.passes; ++i) {
      const bool last = i + 1 == p.passes;
      RadixPass r{};
      r.tokens = i == 0 ? a.tokens : nullptr;
      r.key = a.key[at];
      r.pos = a.pos[at];
      if (i > 0) at ^= 1;
      r.key_out = a.key[at];
      r.pos_out = a.pos[at];
      r.hist = a.hist[i % 3];
      r.next = last ? nullptr : a.hist[(i + 1) % 3];
      r.after = i + 2 < p.passes ? a.hist[(i + 2) % 3] : nullptr;
      r.N = a.N;
      r.per = p.per;
      r.V = a.V;
      r.bits = p.bits;
      r.shift = i * p.bits;
      r.blocks = p.blocks;
      radix_move_kernel<<<p.blocks, kRadixThreads, 0, st>>>(r);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  if (a.grad_y_dtype == 0) return add_rows<float, float>(a, p, a.key[at], a.pos[at], st);
  if (a.grad_weight_dtype == 0) return add_rows<__bf16, float>(a, p, a.key[at], a.pos[at], st);
  return add_rows<__bf16, __bf16>(a, p, a.key[at], a.pos[at], st);
}

}  // namespace plp
