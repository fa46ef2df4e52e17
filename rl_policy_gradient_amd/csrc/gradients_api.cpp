// Host side of the embedding, its gradient, the gradients' global norm and
// their clipping: argument checks and workspace sizes. No allocation, no host
// synchronisation.
#include <math.h>

#include <algorithm>

#include "checks.h"
#include "training_ops.h"

using namespace plp;

namespace {

constexpr int kMaxEmbedH = 65536;

int check_embed_sizes(int64_t N, int32_t H, int32_t V, int32_t dtype) {
  if (!known_dtype(dtype)) return fail(PLP_E_INVALID, "unknown dtype %d", dtype);
  if (N < 0 || N >= kMaxRows) return fail(PLP_E_INVALID, "N=%lld outside [0, 2^31)", (long long)N);
  if (H < 1) return fail(PLP_E_INVALID, "H must be >= 1 (got %d)", H);
  if (V < 1) return fail(PLP_E_INVALID, "V must be >= 1 (got %d)", V);
  if (H > kMaxEmbedH) return fail(PLP_E_UNSUPPORTED, "H=%d is above %d", H, kMaxEmbedH);
  return PLP_OK;
}

size_t carve_embed_bwd(void* ws, EmbedBwd& a) {
  Carver c(ws);
  if (a.N == 0) return 0;
  const EmbedBwdPlan p = embed_bwd_plan(a.N, a.H, a.V, a.grad_y_dtype);
  const size_t n = (size_t)a.N;
  a.key[0] = c.take<uint32_t>(n);
  a.pos[0] = c.take<uint32_t>(n);
  const bool more = p.radix && p.passes > 1;
  a.key[1] = c.take<uint32_t>(more ? n : 0);
  a.pos[1] = c.take<uint32_t>(more ? n : 0);
  a.hist = c.take<uint32_t>(p.radix ? (size_t)p.blocks << p.bits : 0);
  a.tail_row = c.take<int32_t>((size_t)p.ranges);
  a.shared_rows = c.take<uint32_t>(1);
  a.shared_list = c.take<uint2>((size_t)p.ranges);
  a.head = c.take<float>((size_t)p.ranges * part_width(a.H));
  a.tail = c.take<float>((size_t)p.ranges * part_width(a.H));
  return c.off;
}

// Elements of all tensors together: a tile's stay below 2^31.
constexpr int64_t kMaxGradNumel = (int64_t)1 << 40;
constexpr int kMaxGrads = 1 << 20;
// Elements of a tile, log2: at least 2048 (a load of 16 bytes a thread for
// bf16), and at most 4096 tiles and one a tensor for the finishing workgroup to
// add (20000 tensors 7 us, 200000 42: little beside the launches that sum them, of
// up to 240 tensors each, which take 0.85 ms for 20000).
constexpr int kMinTileShift = 11;
constexpr int64_t kMostTiles = 4096;

// Elements and tiles of a list whose norm one workgroup forms in one launch. A
// call from Python takes 9 to 11 us so, and 12 to 14 in two launches, whose time
// on the host is what counts there; of 100 tensors 12 and 15, but of 200 it is
// the one workgroup that counts, 21 and 19.
constexpr int64_t kSmallTotal = (int64_t)1 << 17;

int check_grads(const plp_grad_tensor* t, int32_t count, int64_t* total) {
  if (count < 0 || count > kMaxGrads || (count > 0 && !t))
    return fail(PLP_E_INVALID, "tensors is NULL or count=%d outside [0, 2^20]", count);
  int64_t sum = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].numel < 0 || t[i].numel > kMaxGradNumel)
      return fail(PLP_E_INVALID, "tensor %d: numel=%lld outside [0, 2^40]", i, (long long)t[i].numel);
    if (!known_dtype(t[i].dtype)) return fail(PLP_E_INVALID, "tensor %d: unknown dtype %d", i, t[i].dtype);
    if (t[i].numel > 0 && !t[i].grad) return fail(PLP_E_INVALID, "tensor %d: grad is required", i);
    if (misaligned(t[i].grad, esize(t[i].dtype)))
      return fail(PLP_E_INVALID, "tensor %d: grad is not aligned to its elements", i);
    sum += t[i].numel;  // at most 2^60
  }
  if (sum > kMaxGradNumel) return fail(PLP_E_INVALID, "%lld elements in all are above 2^40", (long long)sum);
  *total = sum;
  return PLP_OK;
}

int tile_shift(int64_t total) {
  int s = kMinTileShift;
  while (total >> s >= kMostTiles) ++s;
  return s;
}
int64_t tiles_of(const plp_grad_tensor& t, int shift) {
  return t.numel == 0 ? 1 : ((t.numel - 1) >> shift) + 1;  // an empty tensor has an empty tile
}

// Calls f for each launch's worth of the list.
template <typename F>
int for_launches(const plp_grad_tensor* tensors, int32_t count, int shift, F f) {
  GradLaunch l;
  l.tile_shift = (uint32_t)shift;
  l.count = l.groups = l.first_tensor = l.first_tile = 0;
  for (int i = 0; i < count; ++i) {
    const plp_grad_tensor& t = tensors[i];
    const int64_t n = tiles_of(t, shift), tail = t.numel - ((n - 1) << shift);
    if (l.count == kGradMaxTensors) {
      int rc = f(l);
      if (rc) return rc;
      l.first_tensor += l.count;
      l.first_tile += l.groups;
      l.count = l.groups = 0;
    }
    l.t[l.count++] = GradEntry{t.grad, l.groups, (uint32_t)tail << 1 | (t.dtype == PLP_DTYPE_BF16 ? 1u : 0u)};
    l.groups += (uint32_t)n;
  }
  return l.count ? f(l) : PLP_OK;
}

struct GradWork {
  double* part;
  uint32_t* start;
};
size_t carve_grads(void* ws, const plp_grad_tensor* t, int32_t count, int shift, GradWork& w, int64_t* tiles) {
  *tiles = 0;
  for (int i = 0; i < count; ++i) *tiles += tiles_of(t[i], shift);
  Carver c(ws);
  w.part = c.take<double>((size_t)*tiles);
  w.start = c.take<uint32_t>((size_t)count);
  return c.off;
}

}  // namespace

extern "C" {

PLP_API int plp_embedding_fwd(const int64_t* tokens, const void* weight, int64_t N, int32_t H, int32_t V, int32_t dtype,
                              float scale, void* y, hipStream_t st) {
  int rc = check_embed_sizes(N, H, V, dtype);
  if (rc) return rc;
  if (!isfinite(scale)) return fail(PLP_E_INVALID, "scale must be finite");
  if (N == 0) return ok();
  if (!tokens || !weight || !y) return fail(PLP_E_INVALID, "tokens, weight and y are required");
  const size_t e = esize(dtype);
  if (misaligned(tokens, 8) || misaligned(weight, e) || misaligned(y, e))
    return fail(PLP_E_INVALID, "a tensor is not aligned to its elements");
  const Range in[] = {{tokens, (size_t)N * 8}, {weight, (size_t)V * H * e}}, out[] = {{y, (size_t)N * H * e}};
  rc = check_apart(in, out);
  if (rc) return rc;
  HIP_TRY(launch_embed_fwd(EmbedFwd{tokens, weight, y, N, H, V, dtype, scale}, st));
  return ok();
}

PLP_API int plp_embedding_bwd_workspace_size(int64_t N, int32_t H, int32_t V, int32_t grad_y_dtype, size_t* bytes) {
  if (!bytes) return fail(PLP_E_INVALID, "bytes is NULL");
  int rc = check_embed_sizes(N, H, V, grad_y_dtype);
  if (rc) return rc;
  EmbedBwd a{};
  a.N = N;
  a.H = H;
  a.V = V;
  a.grad_y_dtype = grad_y_dtype;
  *bytes = carve_embed_bwd(nullptr, a);
  return ok();
}

PLP_API int plp_embedding_bwd(const int64_t* tokens, const void* grad_y, int64_t N, int32_t H, int32_t V,
                              int32_t grad_y_dtype, int32_t grad_weight_dtype, float scale, int32_t accumulate,
                              void* grad_weight, void* ws, size_t ws_bytes, hipStream_t st) {
  int rc = check_embed_sizes(N, H, V, grad_y_dtype);
  if (rc) return rc;
  if (!known_dtype(grad_weight_dtype)) return fail(PLP_E_INVALID, "unknown dtype %d", grad_weight_dtype);
  if (grad_y_dtype == PLP_DTYPE_F32 && grad_weight_dtype != PLP_DTYPE_F32)
    return fail(PLP_E_UNSUPPORTED, "grad_weight of an fp32 grad_y is fp32");
  if (!isfinite(scale)) return fail(PLP_E_INVALID, "scale must be finite");
  if (!grad_weight) return fail(PLP_E_INVALID, "grad_weight is required");
  if (N > 0 && (!tokens || !grad_y)) return fail(PLP_E_INVALID, "tokens and grad_y are required");
  const size_t e = esize(grad_y_dtype), we = esize(grad_weight_dtype);
  if (misaligned(tokens, 8) || misaligned(grad_y, e) || misaligned(grad_weight, we))
    return fail(PLP_E_INVALID, "a tensor is not aligned to its elements");
  EmbedBwd a{};
  a.tokens = tokens;
  a.grad_y = grad_y;
  a.grad_weight = grad_weight;
  a.N = N;
  a.H = H;
  a.V = V;
  a.grad_y_dtype = grad_y_dtype;
  a.grad_weight_dtype = grad_weight_dtype;
  a.accumulate = accumulate ? 1 : 0;
  a.scale = scale;
  const size_t need = carve_embed_bwd(ws, a);
  const Range in[] = {{tokens, (size_t)N * 8}, {grad_y, (size_t)N * H * e}},
              out[] = {{grad_weight, (size_t)V * H * we}, {ws, need}};
  rc = check_apart(in, out);
  if (rc) return rc;
  rc = check_ws(ws, ws_bytes, need);
  if (rc) return rc;
  HIP_TRY(launch_embed_bwd(a, st));
  return ok();
}

PLP_API int plp_grad_norm_workspace_size(const plp_grad_tensor* tensors, int32_t count, size_t* bytes) {
  if (!bytes) return fail(PLP_E_INVALID, "bytes is NULL");
  int64_t total = 0, tiles = 0;
  int rc = check_grads(tensors, count, &total);
  if (rc) return rc;
  GradWork w;
  *bytes = carve_grads(nullptr, tensors, count, tile_shift(total), w, &tiles);
  return ok();
}

PLP_API int plp_grad_norm(const plp_grad_tensor* tensors, int32_t count, double max_norm, double eps,
                          const float* grad_scale, float* norm_out, float* scale_out, float* norms_out, void* ws,
                          size_t ws_bytes, hipStream_t st) {
  int64_t total = 0, tiles = 0;
  int rc = check_grads(tensors, count, &total);
  if (rc) return rc;
  if (!(max_norm >= 0.0)) return fail(PLP_E_INVALID, "max_norm must be >= 0");
  if (!(eps >= 0.0) || !isfinite(eps)) return fail(PLP_E_INVALID, "eps must be finite and >= 0");
  if (!norm_out || !scale_out) return fail(PLP_E_INVALID, "norm_out and scale_out are required");
  if (misaligned(grad_scale, 4) || misaligned(norm_out, 4) || misaligned(scale_out, 4) || misaligned(norms_out, 4))
    return fail(PLP_E_INVALID, "an array is not aligned to its elements");
  const int shift = tile_shift(total);
  GradWork w;
  const size_t need = carve_grads(ws, tensors, count, shift, w, &tiles);
  const Range out[] = {{norm_out, 4}, {scale_out, 4}, {norms_out, (size_t)count * 4}, {ws, need}};
  const Range given[] = {{grad_scale, 4}};
  rc = check_apart(given, out);
  for (int i = 0; i < count && !rc; ++i) {
    const Range g = {tensors[i].grad, (size_t)tensors[i].numel * esize(tensors[i].dtype)};
    for (const Range& o : out)
      if (overlap(g.p, g.n, o.p, o.n)) return fail(PLP_E_INVALID, "tensor %d overlaps an output or the workspace", i);
  }
  if (rc) return rc;
  rc = check_ws(ws, ws_bytes, need);
  if (rc) return rc;
  GradFinish f;
  f.part = w.part;
  f.start = w.start;
  f.grad_scale = grad_scale;
  f.norm = norm_out;
  f.scale = scale_out;
  f.norms = norms_out;
  f.max_norm = max_norm;
  f.eps = eps;
  f.tiles = (uint32_t)tiles;
  f.count = (uint32_t)count;
  if (count > 0 && tiles <= kGradSmallTiles && total <= kSmallTotal) {
    rc = for_launches(tensors, count, shift, [&](const GradLaunch& l) {
      HIP_TRY(launch_grad_small(l, f, st));
      return (int)PLP_OK;
    });
    return rc ? rc : ok();
  }
  rc = for_launches(tensors, count, shift, [&](const GradLaunch& l) {
    HIP_TRY(launch_grad_squares(l, w.part, w.start, st));
    return (int)PLP_OK;
  });
  if (rc) return rc;
  HIP_TRY(launch_grad_finish(f, st));
  return ok();
}

PLP_API int plp_clip_grads(const plp_grad_tensor* tensors, int32_t count, const float* scale, hipStream_t st) {
  int64_t total = 0;
  int rc = check_grads(tensors, count, &total);
  if (rc) return rc;
  if (!scale) return fail(PLP_E_INVALID, "scale is required");
  if (misaligned(scale, 4)) return fail(PLP_E_INVALID, "scale is not aligned to its type");
  for (int i = 0; i < count; ++i)
    if (overlap(tensors[i].grad, (size_t)tensors[i].numel * esize(tensors[i].dtype), scale, 4))
      return fail(PLP_E_INVALID, "tensor %d overlaps scale", i);
  rc = for_launches(tensors, count, tile_shift(total), [&](const GradLaunch& l) {
    HIP_TRY(launch_grad_clip(l, scale, st));
    return (int)PLP_OK;
  });
  return rc ? rc : ok();
}

}  // extern "C"
