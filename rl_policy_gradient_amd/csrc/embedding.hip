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
// workgroups a pass. Without `accumulate` other workgroups of the same launches
// set grad_weight to zero, which takes longer than the sorting and does not
// wait for it.
//
// Adding: a wave takes a range of the sorted tokens, for 64 lanes' columns. A
// row whose tokens go on past a range's end by a few is finished there, else it
// is left in parts, which a last kernel adds up in their order.
//
// What bounds them. Forward: HBM, 25 us for 65536 rows of 896 bf16 (6.0 TB/s
// with the tables' rows that the tokens name read once). Backward of as many
// into 151936 x 896 bf16, 85 us: the zeros 46 (5.9 TB/s, the sort beside them),
// 32 to read the rows in the tokens' order and write the 15 000 that have any
// (4.2 TB/s: 16 rows of a range are two loads of eight), 9 for the rows that
// ranges share (the commonest token's 3300 rows are some 200 parts). One pass
// that wrote every row once, zeros where a merge of tokens and rows had none,
// took 108: the sort, which only latency bounds, came before all of it. 16384
// rows of 4096 fp32 into 32000: 150 (5.3 TB/s). Into a gradient that is there:
// 512 rows 14 to 15, its three launches' latency (3.6 the sort, 7.2 the adding's
// loads one after another, 3.6 a join of little), 65536 70 (their bytes 36: the
// gradient's row is loaded with each of its tokens, of which the last one's is
// used). Narrow rows leave lanes without columns: 65536 of 64 bf16 49, as of 128.
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

typedef unsigned __int128 Bits;

// Elements d .. d + V - 1 of a row of H, those past its end as 0.
template <typename T, int V, bool STREAM = false>
__device__ __forceinline__ typename VecOf<T, V>::type load_raw(const T* row, int d, int H) {
  typedef typename VecOf<T, V>::type TV;
  if (d + V <= H) {
    if constexpr (STREAM)
      return __builtin_nontemporal_load(reinterpret_cast<const TV*>(row + d));
    else
      return *reinterpret_cast<const TV*>(row + d);
  }
  if constexpr (sizeof(TV) == sizeof(Bits))
    if (H >= V) {  // the end of the row's last 16 bytes
      const Bits b = __builtin_bit_cast(Bits, *reinterpret_cast<const TV*>(row + H - V));
      const int past = d + V - H;  // elements; the whole of it where d is past the row
      return __builtin_bit_cast(TV, past < V ? (Bits)(b >> 8 * (int)sizeof(T) * past) : (Bits)0);
    }
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
template <typename T, int V, bool STREAM = false>
__device__ __forceinline__ void store_part(T* row, int d, int H, const float (&x)[V]) {
  typedef typename VecOf<T, V>::type TV;
  if (d + V <= H) {
    TV t;
#pragma unroll
    for (int k = 0; k < V; ++k) t[k] = (T)x[k];
    if constexpr (STREAM)
      __builtin_nontemporal_store(t, reinterpret_cast<TV*>(row + d));
    else
      *reinterpret_cast<TV*>(row + d) = t;
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (d + k < H) row[d + k] = (T)x[k];
  }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Outputs of this many bytes are stored past the caches. What reads them next
// finds little of them there: the lookup of 65536 rows of 896 bf16 (117 MB)
// takes 25 us so and 33 otherwise, with a norm of its rows after it 73 and 78;
// of 32768 rows 18.5 and 19.5, but with the norm 41 and 38.
constexpr int64_t kStreamBytes = (int64_t)1 << 26;
// Threads that set grad_weight to zero, two waves a CU: with 2^14 of them the
// backward of 65536 rows of 896 takes 112 us, with 2^15 86, 2^16 89, 2^17 95 and
// 2^19, as many as run at once, 98.
constexpr int kFillThreads = 1 << 15;

// ---- forward -----------------------------------------------------------------

constexpr int kFwdRows = 4;  // rows a wave has in flight

template <typename T, bool STREAM>
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
    store_part<T, V, STREAM>((T*)a.y + (n0 + r) * a.H, d, a.H, y);
  }
}

// ---- sorting -----------------------------------------------------------------

// What of grad_weight the workgroups of a launch that do not sort set to zero:
// `bytes` from p on, a multiple of 2. Streamed past the caches where it is more
// than they hold (embed_bwd_plan).
struct Fill {
  char* p;
  int64_t bytes;
  uint32_t groups;
  int stream;
};
__device__ __forceinline__ void fill(const Fill& f, uint32_t group) {
  typedef uint16_t Words __attribute__((ext_vector_type(8), aligned(2)));
  const int64_t step = (int64_t)f.groups * blockDim.x * 16;
  int64_t i = ((int64_t)group * blockDim.x + threadIdx.x) * 16;
  const Words zero = {};
  if (f.stream)
    for (; i + 16 <= f.bytes; i += step) __builtin_nontemporal_store(zero, reinterpret_cast<Words*>(f.p + i));
  else
    for (; i + 16 <= f.bytes; i += step) *reinterpret_cast<Words*>(f.p + i) = zero;
  for (; i < f.bytes; i += 2) *reinterpret_cast<uint16_t*>(f.p + i) = 0;  // fewer than 16, of one thread
}

// A token as a key; what is no row comes after every row.
__device__ __forceinline__ uint32_t key_of(int64_t t, int V) { return t >= 0 && t < V ? (uint32_t)t : (uint32_t)V; }

constexpr int kCountingN = 4096;  // a multiple of what the lanes of a token read at a time
constexpr int kCountLanes = 16;                  // threads that share a token
constexpr int kCountItems = 256 / kCountLanes;  // tokens a workgroup places

__global__ __launch_bounds__(256) void sort_counting_kernel(const int64_t* __restrict__ tokens, int N, int V,
                                                            uint32_t* __restrict__ key, uint32_t* __restrict__ pos,
                                                            uint32_t* __restrict__ shared_rows, uint32_t groups,
                                                            Fill f) {
  if (blockIdx.x >= groups) return fill(f, blockIdx.x - groups);
  if (blockIdx.x == 0 && threadIdx.x == 0) *shared_rows = 0;
  __shared__ __attribute__((aligned(16))) uint32_t all[kCountingN];
  constexpr int step = 4 * kCountLanes;
  const int padded = (N + step - 1) / step * step;  // up to kCountingN
  for (int i = threadIdx.x; i < padded; i += 256) all[i] = i < N ? key_of(tokens[i], V) : 0xffffffffu;
  __syncthreads();
  const int part = threadIdx.x % kCountLanes, i = blockIdx.x * kCountItems + (int)threadIdx.x / kCountLanes;
  const uint32_t mine = all[i < N ? i : 0];
  int before = 0;
#pragma unroll 4
  for (int j = part * 4; j < padded; j += step) {
    const uint4 k = *reinterpret_cast<const uint4*>(all + j);
    before += k.x < mine || (k.x == mine && j < i);
    before += k.y < mine || (k.y == mine && j + 1 < i);
    before += k.z < mine || (k.z == mine && j + 2 < i);
    before += k.w < mine || (k.w == mine && j + 3 < i);
  }
#pragma unroll
  for (int o = 1; o < kCountLanes; o <<= 1) before += __shfl_xor(before, o, 64);
  if (part == 0 && i < N) {
    key[before] = mine;
    pos[before] = (uint32_t)i;
  }
}

constexpr int kMinBits = 8, kMaxBits = 10;
constexpr int kHeld = 2;
constexpr int kRadixWaves = 8, kRadixThreads = kRadixWaves * 64;

struct RadixPass {
  const int64_t* tokens;      // the first pass's input
  const uint32_t *key, *pos;  // the others'
  uint32_t *key_out, *pos_out;
  uint32_t* hist;         // [blocks][1 << bits]
  uint32_t* shared_rows;  // cleared
  int64_t N, per;
  int V, bits, shift, blocks;
  __device__ __forceinline__ uint32_t key_at(int64_t i) const { return tokens ? key_of(tokens[i], V) : key[i]; }
};

// Counts of a pass's digits in each workgroup's tokens. (Counted by the pass
// before at the tokens' new places, with atomics, these cost it 9 us, twice
// this kernel: half of the tokens of a vocabulary share their upper digit.)
__global__ __launch_bounds__(kRadixThreads) void radix_count_kernel(RadixPass a, Fill f) {
  if (blockIdx.x >= (uint32_t)a.blocks) return fill(f, blockIdx.x - a.blocks);
  __shared__ uint32_t count[1 << kMaxBits];
  const int digits = 1 << a.bits;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.shared_rows = 0;
  for (int d = threadIdx.x; d < digits; d += kRadixThreads) count[d] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.per, end = begin + a.per < a.N ? begin + a.per : a.N;
  for (int64_t i = begin + threadIdx.x; i < end; i += kRadixThreads)
    atomicAdd(&count[a.key_at(i) >> a.shift & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kRadixThreads) a.hist[(int64_t)blockIdx.x * digits + d] = count[d];
}

// Moves a workgroup's tokens to their places by the pass's digit, each wave's
// in their order.
__global__ __launch_bounds__(kRadixThreads) void radix_move_kernel(RadixPass a, Fill f) {
  if (blockIdx.x >= (uint32_t)a.blocks) return fill(f, blockIdx.x - a.blocks);
  __shared__ uint32_t at[kRadixWaves][1 << kMaxBits];
  __shared__ uint32_t wave_total[kRadixWaves];
  __shared__ __attribute__((aligned(16))) uint32_t part_all[kRadixThreads * 4], part_prior[kRadixThreads * 4];
  const int digits = 1 << a.bits, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t begin = blockIdx.x * a.per, end = begin + a.per < a.N ? begin + a.per : a.N;
  const int64_t each = (a.per + kRadixWaves - 1) / kRadixWaves;
  const int64_t w0 = begin + wave * each < end ? begin + wave * each : end, w1 = w0 + each < end ? w0 + each : end;
  // the first tokens of each wave, which are all of them in a batch of up to 256 K, stay in registers
  uint32_t held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int64_t i = w0 + k * 64 + lane;
    held[k] = i < w1 ? a.key_at(i) : 0;
  }
  // where each digit begins in this workgroup: all smaller digits, and the same in the workgroups before.
  // Four digits a load, the workgroups' counts shared out to the threads.
  const int quads = digits / 4, subsets = kRadixThreads / quads, quad = (int)threadIdx.x % quads;
  uint4 all = {0, 0, 0, 0}, prior = {0, 0, 0, 0};
#pragma unroll 8
  for (int b = (int)threadIdx.x / quads; b < a.blocks; b += subsets) {
    const uint4 c = *reinterpret_cast<const uint4*>(a.hist + (int64_t)b * digits + quad * 4);
    const uint32_t here = b < (int)blockIdx.x ? ~0u : 0u;
    all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
    prior.x += c.x & here, prior.y += c.y & here, prior.z += c.z & here, prior.w += c.w & here;
  }
  for (int d = threadIdx.x; d < kRadixWaves * digits; d += kRadixThreads) at[d / digits][d % digits] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (w0 + k * 64 + lane < w1) atomicAdd(&at[wave][held[k] >> a.shift & (digits - 1)], 1u);
  for (int64_t i = w0 + kHeld * 64 + lane; i < w1; i += 64) atomicAdd(&at[wave][a.key_at(i) >> a.shift & (digits - 1)], 1u);
  reinterpret_cast<uint4*>(part_all)[threadIdx.x] = all;
  reinterpret_cast<uint4*>(part_prior)[threadIdx.x] = prior;
  __syncthreads();  // the waves' counts are whole, too
  const int per_thread = digits > kRadixThreads ? digits / kRadixThreads : 1;  // 1 or 2
  uint32_t total[2] = {0, 0}, before[2] = {0, 0}, sum = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = (int)threadIdx.x * per_thread + k;
    if (k >= per_thread || d >= digits) continue;
    for (int i = 0; i < subsets; ++i) total[k] += part_all[i * digits + d], before[k] += part_prior[i * digits + d];
    sum += total[k];
  }
  uint32_t run = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(run, o, 64);
    run += lane >= o ? v : 0;
  }
  if (lane == 63) wave_total[wave] = run;
  __syncthreads();
  run -= sum;
  for (int w = 0; w < wave; ++w) run += wave_total[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = (int)threadIdx.x * per_thread + k;
    if (k >= per_thread || d >= digits) continue;
    uint32_t place = run + before[k];
    run += total[k];
#pragma unroll
    for (int w = 0; w < kRadixWaves; ++w) {
      const uint32_t c = at[w][d];
      at[w][d] = place;
      place += c;
    }
  }
  __syncthreads();
  int step = 0;
  for (int64_t i0 = w0; i0 < w1; i0 += 64, ++step) {
    const int64_t i = i0 + lane;
    const bool in = i < w1;
    uint32_t key = 0;
    if (step < kHeld) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) key = step == k ? held[k] : key;
    } else if (in) {
      key = a.key_at(i);
    }
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
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- adding ------------------------------------------------------------------

constexpr int kAddWaves = 4;
constexpr int kBatch = 8;  // rows of grad_y a wave has in flight
// Tokens that a row has past a range's end, at least, for it to be shared: with
// fewer the range before goes on to the row's end and the next one begins there.
constexpr int kShared = 16;

template <typename TG>
constexpr int add_vec = 16 / (int)sizeof(TG);  // columns a lane takes

// Where a range ends and the next begins: before token i of the sorted order.
// open: the row of that token has tokens before it; shared: and kShared or more
// from it on; past: the first token that is not in the row, if it is not shared.
struct Edge {
  int64_t i, past;
  bool open, shared;
};
// From `before` and `at`, the keys around it, and the lanes whose keys are from
// token i on (lane 0: token i) and equal to `at`.
__device__ __forceinline__ Edge edge_of(int64_t N, int V, int64_t i, int before, int at, uint64_t same) {
  Edge e{i, i, i > 0 && i < N && at < V && before == at, false};
  if (!e.open) return e;
  const int n = __builtin_ctzll(~same);  // sorted: they lie side by side
  e.shared = n >= kShared;
  e.past = i + n;
  return e;
}
__device__ __forceinline__ Edge edge_at(const uint32_t* __restrict__ key, int64_t N, int V, int64_t i, int lane) {
  if (i == 0 || i >= N) return Edge{i, i, false, false};
  const int v = (int)key[i];
  return edge_of(N, V, i, (int)key[i - 1], v, __ballot(lane < kShared && i + lane < N && (int)key[i + lane < N ? i + lane : i] == v));
}

template <typename TG, typename TW, bool ACC>
__global__ __launch_bounds__(kAddWaves * 64) void embed_add_kernel(EmbedBwd a, const uint32_t* __restrict__ key,
                                                                   const uint32_t* __restrict__ pos, uint32_t slices,
                                                                   int items, uint32_t ranges) {
  constexpr int V = add_vec<TG>;
  typedef typename VecOf<TG, V>::type GV;
  typedef typename VecOf<TW, V>::type WV;
  const int lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x * kAddWaves + uniform(threadIdx.x >> 6);
  const int64_t range = unit / slices;
  if (range >= ranges) return;
  const int slice = (int)(unit % slices), d = (slice * 64 + lane) * V;
  const bool in = d < a.H;
  const int64_t first = range * items, next = first + items < a.N ? first + items : a.N;
  // The tokens from one before the range on, a lane each: where they hold the
  // range and what its edges go by, nothing more is loaded before the rows.
  const bool window = items + kShared < 64;
  int keys = 0, rows = 0, at = 0;  // the tokens at hand, and the lane of the next one
  Edge from, to;
  if (window) {
    const int64_t i = first - 1 + lane;
    const bool is = i >= 0 && i < a.N;
    keys = is ? (int)key[i] : -1;
    rows = is ? (int)pos[i] : 0;
    const auto edge = [&](int64_t i, int l) {  // lane l has token i
      const int k = __builtin_amdgcn_readlane(keys, l);
      return edge_of(a.N, a.V, i, __builtin_amdgcn_readlane(keys, l - 1), k, __ballot(keys == k) >> l);
    };
    from = edge(first, 1);
    to = edge(next, (int)(next - first) + 1);
  } else {
    from = edge_at(key, a.N, a.V, first, lane);
    to = edge_at(key, a.N, a.V, next, lane);
  }
  // a row that began before and is not shared is not this range's; one that goes on and is not shared is
  const int64_t i0 = from.open && !from.shared ? from.past : from.i, end = to.open && !to.shared ? to.past : to.i;
  int v = -1, v0 = -1;  // the row being added up; the one that began before
  float sum[V];
  bool any = false, headed = false;
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.f;
  TW* const w = (TW*)a.grad_weight;
  const auto end_row = [&](const WV& old) {  // of row v
    if (v == v0) {
      if (in) store_part<float, V>(a.head + range * part_width(a.H), d, part_width(a.H), sum);
      headed = true;
    } else if (in) {
      float x[V];
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = a.scale * sum[k];
      if constexpr (ACC)
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] += (float)old[k];
      store_part<TW, V>(w + (int64_t)v * a.H, d, a.H, x);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] = 0.f;
    any = false;
  };
  WV before = {};  // what grad_weight holds of the row last added to
  for (int64_t b0 = i0; b0 < end; b0 += 64) {
    if (window) {
      at = (int)(i0 - first) + 1;
    } else {
      const int64_t mine = b0 + lane < end ? b0 + lane : end - 1;
      keys = (int)key[mine], rows = (int)pos[mine];
    }
    const int left = (int)(end - b0 < 64 ? end - b0 : 64);
    bool done = false;
    for (int j0 = 0; j0 < left && !done; j0 += kBatch) {
      GV x[kBatch];
      WV old[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (j0 + j >= left) break;
        const int64_t row = (uint32_t)__builtin_amdgcn_readlane(rows, at + j0 + j);
        const int k = __builtin_amdgcn_readlane(keys, at + j0 + j);
        if (in) x[j] = load_raw<TG, V, true>((const TG*)a.grad_y + row * a.H, d, a.H);
        if constexpr (ACC)
          if (in && k < a.V) old[j] = load_raw<TW, V>(w + (int64_t)k * a.H, d, a.H);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (j0 + j >= left) break;
        const int k = __builtin_amdgcn_readlane(keys, at + j0 + j);
        if (k >= a.V) {  // no row, and nothing but those from here on
          done = true;
          break;
        }
        if (any && v < k) end_row(before);
        v = k;
        if (from.shared && b0 + j0 + j == i0) v0 = v;
        if constexpr (ACC) before = old[j];
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += (float)x[j][e];
        any = true;
      }
    }
    if (done) break;
  }
  if (any && !to.shared) end_row(before);
  if (any && in) store_part<float, V>(a.tail + range * part_width(a.H), d, part_width(a.H), sum);
  if (slice == 0 && lane == 0) {
    a.tail_row[range] = any ? v : -1;
    // listed in any order: each is added up by itself
    if (headed) a.shared_list[atomicAdd(a.shared_rows, 1u)] = make_uint2((uint32_t)range, (uint32_t)v0);
  }
}

constexpr int kJoinWaves = 8;
constexpr int kJoinGroups = 1024;

// The rows that several ranges share, from their partial sums: a workgroup a
// row and slice, its waves a part of the sums each.
template <typename TG, typename TW, bool ACC>
__global__ __launch_bounds__(kJoinWaves * 64) void embed_join_kernel(EmbedBwd a, uint32_t slices) {
  constexpr int V = add_vec<TG>;
  __shared__ float part[kJoinWaves][64][V + 1];
  __shared__ int found[kJoinWaves];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t units = *a.shared_rows * slices;  // at most some 16384
  for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t range = a.shared_list[unit / slices].x;
    const int row = (int)a.shared_list[unit / slices].y, d = ((int)(unit % slices) * 64 + lane) * V;
    // the ranges before this one that hold a partial sum of the row: the waves look at 64 each
    int64_t n = 0;
    for (bool on = true; on;) {
      const int64_t k = range - 1 - n - (wave * 64 + lane);
      const uint64_t other = __ballot(!(k >= 0 && a.tail_row[k < 0 ? 0 : k] == row));
      if (lane == 0) found[wave] = other ? __builtin_ctzll(other) : 64;
      __syncthreads();
      for (int p = 0; p < kJoinWaves && on; ++p) {
        n += found[p];
        on = found[p] == 64;
      }
      __syncthreads();
    }
    const int64_t first = range - n, each = (n + kJoinWaves - 1) / kJoinWaves;
    const int64_t from = first + wave * each < range ? first + wave * each : range;
    const int64_t to = from + each < range ? from + each : range;
    float sum[V] = {};
    if (d < a.H)
#pragma unroll 8
      for (int64_t k = from; k < to; ++k) {
        float x[V];
        load_part<float, V>(a.tail + k * part_width(a.H), d, part_width(a.H), x);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += x[e];
      }
#pragma unroll
    for (int e = 0; e < V; ++e) part[wave][lane][e] = sum[e];
    __syncthreads();
    if (wave == 0 && d < a.H) {
      TW* const w = (TW*)a.grad_weight + (int64_t)row * a.H;
      float x[V], old[V] = {};
      load_part<float, V>(a.head + range * part_width(a.H), d, part_width(a.H), x);
      if constexpr (ACC) load_part<TW, V>(w, d, a.H, old);
      for (int p = 1; p < kJoinWaves; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += part[p][lane][e];
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] = a.scale * (sum[e] + x[e]) + old[e];
      store_part<TW, V>(w, d, a.H, sum);
    }
    __syncthreads();  // the sums have been read
  }
}

// The gradient where there are no tokens.
__global__ __launch_bounds__(256) void embed_zero_kernel(Fill f) { fill(f, blockIdx.x); }

int slices_of(int H, int dtype) {
  const int lanes = 64 * (dtype == 0 ? 4 : 8);
  return (H + lanes - 1) / lanes;
}

template <typename TG, typename TW, bool ACC>
hipError_t add_rows(const EmbedBwd& a, const EmbedBwdPlan& p, const uint32_t* key, const uint32_t* pos, hipStream_t st) {
  const int64_t units = p.ranges * p.slices;
  embed_add_kernel<TG, TW, ACC><<<(unsigned)((units + kAddWaves - 1) / kAddWaves), kAddWaves * 64, 0, st>>>(
      a, key, pos, p.slices, p.items, (uint32_t)p.ranges);
  if (hipError_t e = hipGetLastError()) return e;
  if (!p.shared) return hipSuccess;
  embed_join_kernel<TG, TW, ACC><<<kJoinGroups, kJoinWaves * 64, 0, st>>>(a, p.slices);
  return hipGetLastError();
}
template <typename TG, typename TW>
hipError_t add_rows(const EmbedBwd& a, const EmbedBwdPlan& p, const uint32_t* key, const uint32_t* pos, hipStream_t st) {
  return a.accumulate ? add_rows<TG, TW, true>(a, p, key, pos, st) : add_rows<TG, TW, false>(a, p, key, pos, st);
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedFwd& a, hipStream_t st) {
  const int slices = slices_of(a.H, a.dtype);
  const int64_t units = (a.N + kFwdRows - 1) / kFwdRows * slices;
  // a launch holds fewer than 2^32 threads
  const int64_t most = ((int64_t)1 << 23) / slices * slices;
  const size_t e = a.dtype == 0 ? 4 : 2;
  const bool stream = (int64_t)(a.N * a.H * e) >= kStreamBytes;
  for (int64_t u = 0; u < units; u += most) {
    EmbedFwd b = a;
    const int64_t n0 = u / slices * kFwdRows, some = std::min(most, units - u);
    b.tokens = a.tokens + n0;
    b.y = (char*)a.y + (size_t)n0 * a.H * e;
    b.N = a.N - n0;
    const unsigned grid = (unsigned)((some + 3) / 4);
    if (a.dtype == 0)
      stream ? embed_fwd_kernel<float, true><<<grid, 256, 0, st>>>(b, slices, (uint32_t)some)
             : embed_fwd_kernel<float, false><<<grid, 256, 0, st>>>(b, slices, (uint32_t)some);
    else
      stream ? embed_fwd_kernel<__bf16, true><<<grid, 256, 0, st>>>(b, slices, (uint32_t)some)
             : embed_fwd_kernel<__bf16, false><<<grid, 256, 0, st>>>(b, slices, (uint32_t)some);
    if (hipError_t err = hipGetLastError()) return err;
  }
  return hipSuccess;
}

EmbedBwdPlan embed_bwd_plan(int64_t N, int H, int V, int grad_y_dtype) {
  EmbedBwdPlan p{};
  p.radix = N > kCountingN;
  int bits = 1;
  while ((int64_t)V >> bits) ++bits;  // keys are 0 .. V
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = std::max(kMinBits, (bits + p.passes - 1) / p.passes);
  p.blocks = (int)std::min<int64_t>(256, (N + 1023) / 1024);
  p.per = p.blocks ? (N + p.blocks - 1) / p.blocks : 0;
  p.slices = slices_of(H, grad_y_dtype);
  // some 8192 waves, about what runs at once, but no range of fewer than the
  // tokens that are loaded together (16384 of 896 bf16, into the head's: 41 us,
  // 46 with ranges of 4), or half of that for the few that are sorted by
  // counting (512: 14.2 with 4, 15.0 with 8, 14.6 with 1)
  const int64_t most = std::max<int64_t>(1, 8192 / p.slices);
  p.items = (int)std::max<int64_t>(p.radix ? kBatch : kBatch / 2, (N + most - 1) / most);
  p.ranges = (N + p.items - 1) / p.items;
  p.shared = N > kShared;  // a row has kShared tokens past a range's end, and one before
  return p;
}

hipError_t launch_embed_bwd(const EmbedBwd& a, hipStream_t st) {
  // the zeros, shared out to the launches of the sort
  const int64_t bytes = a.accumulate ? 0 : (int64_t)a.V * a.H * (a.grad_weight_dtype == 0 ? 4 : 2);
  const EmbedBwdPlan p = embed_bwd_plan(a.N, a.H, a.V, a.grad_y_dtype);
  const int launches = a.N == 0 || !p.radix ? 1 : 2 * p.passes;
  const auto part = [&](int i, int threads) {
    const int64_t each = (bytes / launches + 15) / 16 * 16, from = std::min(bytes, i * each);
    Fill f;
    f.p = (char*)a.grad_weight + from;
    f.bytes = i + 1 == launches ? bytes - from : std::min(bytes - from, each);
    f.groups = (uint32_t)std::min<int64_t>(kFillThreads / threads, (f.bytes + threads * 16 - 1) / (threads * 16));
    f.stream = bytes >= kStreamBytes;
    return f;
  };
  if (a.N == 0) {
    if (bytes == 0) return hipSuccess;
    const Fill f = part(0, 256);
    embed_zero_kernel<<<f.groups, 256, 0, st>>>(f);
    return hipGetLastError();
  }
  int at = 0;
  if (!p.radix) {
    const uint32_t groups = (uint32_t)((a.N + kCountItems - 1) / kCountItems);
    const Fill f = part(0, 256);
    sort_counting_kernel<<<groups + f.groups, 256, 0, st>>>(a.tokens, (int)a.N, a.V, a.key[0], a.pos[0], a.shared_rows,
                                                           groups, f);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    for (int i = 0; i < p.passes; ++i) {
      RadixPass r{};
      r.tokens = i == 0 ? a.tokens : nullptr;
      r.key = a.key[at];
      r.pos = a.pos[at];
      if (i > 0) at ^= 1;
      r.key_out = a.key[at];
      r.pos_out = a.pos[at];
      r.hist = a.hist;
      r.shared_rows = a.shared_rows;
      r.N = a.N;
      r.per = p.per;
      r.V = a.V;
      r.bits = p.bits;
      r.shift = i * p.bits;
      r.blocks = p.blocks;
      Fill f = part(2 * i, kRadixThreads);
      radix_count_kernel<<<p.blocks + f.groups, kRadixThreads, 0, st>>>(r, f);
      if (hipError_t e = hipGetLastError()) return e;
      f = part(2 * i + 1, kRadixThreads);
      radix_move_kernel<<<p.blocks + f.groups, kRadixThreads, 0, st>>>(r, f);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  if (a.grad_y_dtype == 0) return add_rows<float, float>(a, p, a.key[at], a.pos[at], st);
  if (a.grad_weight_dtype == 0) return add_rows<__bf16, float>(a, p, a.key[at], a.pos[at], st);
  return add_rows<__bf16, __bf16>(a, p, a.key[at], a.pos[at], st);
}

}  // namespace plp
