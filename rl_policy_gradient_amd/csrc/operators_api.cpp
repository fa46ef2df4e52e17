// Host side of the operators around the fused loss: argument checks and
// workspace sizes of the norm, the AdamW step and token sampling. No
// allocation, no host synchronisation.
#include <math.h>

#include "checks.h"
#include "ops.h"

using namespace plp;

namespace {

// Workgroups of one AdamW launch (times 256 threads stays below 2^32), and the
// largest tensor, which fits one.
constexpr int64_t kMaxAdamGrid = (int64_t)1 << 23;
constexpr int64_t kMaxAdamNumel = kMaxAdamGrid * kAdamTile;

bool in_unit(double b) { return b >= 0.0 && b < 1.0; }

int check_adamw_tensor(const plp_adamw_tensor& t, int i) {
  if (t.numel < 0 || t.numel > kMaxAdamNumel)
    return fail(PLP_E_INVALID, "tensor %d: numel=%lld outside [0, 2^33]", i, (long long)t.numel);
  if (!known_dtype(t.param_dtype) || !known_dtype(t.grad_dtype))
    return fail(PLP_E_INVALID, "tensor %d: unknown dtype (param %d, grad %d)", i, t.param_dtype, t.grad_dtype);
  if (t.state_bits != 8 && t.state_bits != 32)
    return fail(PLP_E_INVALID, "tensor %d: state_bits must be 8 or 32 (got %d)", i, t.state_bits);
  if (!(t.weight_decay >= 0.f) || !isfinite(t.weight_decay))
    return fail(PLP_E_INVALID, "tensor %d: weight_decay must be finite and >= 0", i);
  if (t.master && t.param_dtype != PLP_DTYPE_BF16)
    return fail(PLP_E_INVALID, "tensor %d: a master copy is for bf16 parameters", i);
  if (t.numel == 0) return PLP_OK;
  const bool b8 = t.state_bits == 8;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq)
    return fail(PLP_E_INVALID, "tensor %d: param, grad, exp_avg and exp_avg_sq are required", i);
  if (b8 != (t.exp_avg_scale != nullptr) || b8 != (t.exp_avg_sq_scale != nullptr))
    return fail(PLP_E_INVALID, "tensor %d: 8-bit states have two arrays of scales, 32-bit states none", i);
  const size_t n = (size_t)t.numel, pe = esize(t.param_dtype), ge = esize(t.grad_dtype), se = b8 ? 1 : 4;
  const size_t sb = (n + kAdamBlock - 1) / kAdamBlock * sizeof(float);
  if (misaligned(t.param, pe) || misaligned(t.grad, ge) || misaligned(t.master, 4) || misaligned(t.exp_avg, se) ||
      misaligned(t.exp_avg_sq, se) || misaligned(t.exp_avg_scale, 4) || misaligned(t.exp_avg_sq_scale, 4))
    return fail(PLP_E_INVALID, "tensor %d: an array is not aligned to its elements", i);
  const Range r[] = {{t.param, n * pe},        {t.master, n * 4},           {t.exp_avg, n * se}, {t.exp_avg_sq, n * se},
           {t.exp_avg_scale, sb}, {t.exp_avg_sq_scale, sb}, {t.grad, n * ge}};
  for (int x = 0; x < 7; ++x)
    for (int y = 0; y < x; ++y)
      if (overlap(r[x].p, r[x].n, r[y].p, r[y].n))
        return fail(PLP_E_INVALID, "tensor %d: two of its arrays overlap", i);
  return PLP_OK;
}

constexpr int kMaxNormH = 65536;

size_t carve_sample(void* ws, int64_t N, int32_t V, SampleArgs& a) {
  Carver c(ws);
  a.block_sum = c.take<double>((size_t)N * sample_blocks(V));
  a.block_max = c.take<float>((size_t)N * sample_blocks(V));
  return c.off;
}

int check_norm_sizes(int64_t N, int32_t H, int32_t dtype) {
  if (!known_dtype(dtype)) return fail(PLP_E_INVALID, "unknown dtype %d", dtype);
  if (N < 0 || N >= kMaxRows) return fail(PLP_E_INVALID, "N=%lld outside [0, 2^31)", (long long)N);
  if (H < 1) return fail(PLP_E_INVALID, "H must be >= 1 (got %d)", H);
  if (H > kMaxNormH) return fail(PLP_E_UNSUPPORTED, "H=%d is above %d", H, kMaxNormH);
  return PLP_OK;
}

}  // namespace

extern "C" {

PLP_API int plp_layer_norm_fwd(const void* x, const void* weight, const void* bias, int64_t N, int32_t H,
                               int32_t dtype, int32_t rms, double eps, void* y, float* mean_out, float* rstd_out,
                               hipStream_t st) {
  int rc = check_norm_sizes(N, H, dtype);
  if (rc) return rc;
  if (!(eps >= 0.0) || !isfinite(eps)) return fail(PLP_E_INVALID, "eps must be finite and >= 0");
  if (!weight) return fail(PLP_E_INVALID, "weight is required");
  if (rms && mean_out) return fail(PLP_E_INVALID, "the norm without a mean (rms) has no mean_out");
  if (N == 0) return ok();
  if (!x || !y) return fail(PLP_E_INVALID, "x and y are required");
  const size_t e = esize(dtype), xb = (size_t)N * H * e, sb = (size_t)N * sizeof(float);
  if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, e) || misaligned(bias, e) || misaligned(mean_out, 4) ||
      misaligned(rstd_out, 4))
    return fail(PLP_E_INVALID, "a tensor is not aligned to its elements");
  const Range in[] = {{x, xb}, {weight, H * e}, {bias, H * e}}, out[] = {{y, xb}, {mean_out, sb}, {rstd_out, sb}};
  rc = check_apart(in, out);
  if (rc) return rc;
  HIP_TRY(launch_norm_fwd(NormFwd{x, weight, bias, y, mean_out, rstd_out, N, H, dtype, rms ? 1 : 0, (float)eps}, st));
  return ok();
}

PLP_API int plp_layer_norm_bwd_workspace_size(int64_t N, int32_t H, int32_t dtype, size_t* bytes) {
  if (!bytes) return fail(PLP_E_INVALID, "bytes is NULL");
  int rc = check_norm_sizes(N, H, dtype);
  if (rc) return rc;
  Carver c(nullptr);
  c.take<float>((size_t)2 * norm_bwd_groups(N, H) * H);
  *bytes = c.off;
  return ok();
}

PLP_API int plp_layer_norm_bwd(const void* grad_y, const void* x, const void* weight, const float* mean,
                               const float* rstd, int64_t N, int32_t H, int32_t dtype, int32_t rms, void* grad_x,
                               void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, hipStream_t st) {
  size_t need = 0;
  int rc = plp_layer_norm_bwd_workspace_size(N, H, dtype, &need);
  if (rc) return rc;
  if (!weight) return fail(PLP_E_INVALID, "weight is required");
  if (N > 0 && (!grad_y || !x || !rstd || (!rms && !mean)))
    return fail(PLP_E_INVALID, "grad_y, x, rstd and (but for rms) mean are required");
  const size_t e = esize(dtype), xb = (size_t)N * H * e, wb = (size_t)H * e;
  if (misaligned(grad_y, e) || misaligned(x, e) || misaligned(weight, e) || misaligned(grad_x, e) ||
      misaligned(grad_weight, e) || misaligned(grad_bias, e) || misaligned(mean, 4) || misaligned(rstd, 4))
    return fail(PLP_E_INVALID, "a tensor is not aligned to its elements");
  const size_t sb = (size_t)N * sizeof(float);
  const Range in[] = {{grad_y, xb}, {x, xb}, {weight, wb}, {rms ? nullptr : mean, sb}, {rstd, sb}},
              out[] = {{grad_x, xb}, {grad_weight, wb}, {grad_bias, wb}};
  rc = check_apart(in, out);
  if (rc) return rc;
  rc = check_ws(ws, ws_bytes, grad_weight || grad_bias ? need : 0);
  if (rc) return rc;
  HIP_TRY(launch_norm_bwd(NormBwd{grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                                  grad_weight || grad_bias ? (float*)ws : nullptr, N, H, dtype, rms ? 1 : 0},
                          st));
  return ok();
}

PLP_API int plp_adamw_step(const plp_adamw_args* a, const plp_adamw_tensor* tensors, int32_t count, hipStream_t st) {
  if (!a) return fail(PLP_E_INVALID, "args is NULL");
  if (a->struct_size < sizeof(plp_adamw_args) || a->tensor_size != sizeof(plp_adamw_tensor))
    return fail(PLP_E_INVALID, "args->struct_size %u or tensor_size %u is not this library's (%zu, %zu)",
                a->struct_size, a->tensor_size, sizeof(plp_adamw_args), sizeof(plp_adamw_tensor));
  if (count < 0 || (count > 0 && !tensors)) return fail(PLP_E_INVALID, "tensors is NULL or count negative");
  if (!isfinite(a->lr) || a->lr < 0.0) return fail(PLP_E_INVALID, "lr must be finite and >= 0");
  if (!in_unit(a->beta1) || !in_unit(a->beta2)) return fail(PLP_E_INVALID, "beta1 and beta2 must lie in [0, 1)");
  if (!(a->eps >= 0.0) || !isfinite(a->eps)) return fail(PLP_E_INVALID, "eps must be finite and >= 0");
  if (!a->step_dev && a->step < 1) return fail(PLP_E_INVALID, "step counts from 1 (got %lld)", (long long)a->step);
  if (misaligned(a->step_dev, 8) || misaligned(a->lr_dev, 4) || misaligned(a->grad_scale, 4))
    return fail(PLP_E_INVALID, "step_dev, lr_dev or grad_scale is not aligned to its type");
  for (int i = 0; i < count; ++i) {
    int rc = check_adamw_tensor(tensors[i], i);
    if (rc) return rc;
  }
  AdamLaunch l;
  l.b1 = (float)a->beta1;
  l.c1 = (float)(1.0 - a->beta1);
  l.b2 = (float)a->beta2;
  l.c2 = (float)(1.0 - a->beta2);
  l.eps = (float)a->eps;
  l.lr = a->lr;
  l.ln_b1 = log(a->beta1);  // -inf for 0: 1 - b^t is 1
  l.ln_b2 = log(a->beta2);
  l.step = a->step;
  l.step_dev = a->step_dev;
  l.lr_dev = a->lr_dev;
  l.grad_scale = a->grad_scale;
  l.step_size = l.inv_root = 0.f;
  if (!a->step_dev) {
    l.step_size = (float)(a->lr / -expm1((double)a->step * l.ln_b1));
    l.inv_root = (float)(1.0 / sqrt(-expm1((double)a->step * l.ln_b2)));
  }
  l.count = 0;
  l.first[0] = 0;
  for (int i = 0; i < count; ++i) {
    const plp_adamw_tensor& t = tensors[i];
    if (t.numel == 0) continue;
    const uint32_t groups = (uint32_t)((t.numel + kAdamTile - 1) / kAdamTile);
    if (l.count == kAdamMaxTensors || l.first[l.count] + groups > kMaxAdamGrid) {
      HIP_TRY(launch_adamw(l, st));
      l.count = 0;
    }
    AdamTensor& d = l.t[l.count];
    d.param = t.param;
    d.grad = t.grad;
    d.master = t.master;
    d.m = t.exp_avg;
    d.v = t.exp_avg_sq;
    d.ms = t.exp_avg_scale;
    d.vs = t.exp_avg_sq_scale;
    d.n = t.numel;
    d.decay = a->lr_dev ? t.weight_decay : (float)(a->lr * (double)t.weight_decay);
    d.param_bf16 = t.param_dtype == PLP_DTYPE_BF16;
    d.grad_bf16 = t.grad_dtype == PLP_DTYPE_BF16;
    d.bits8 = t.state_bits == 8;
    l.first[l.count + 1] = l.first[l.count] + groups;
    ++l.count;
  }
  if (l.count > 0) HIP_TRY(launch_adamw(l, st));
  return ok();
}

PLP_API int plp_sample_tokens_workspace_size(int64_t N, int32_t V, size_t* bytes) {
  if (!bytes) return fail(PLP_E_INVALID, "bytes is NULL");
  if (N < 0 || N >= kMaxRows) return fail(PLP_E_INVALID, "N=%lld outside [0, 2^31)", (long long)N);
  if (V < 1) return fail(PLP_E_INVALID, "V must be >= 1 (got %d)", V);
  if (V > kSampleMaxV) return fail(PLP_E_UNSUPPORTED, "V=%d is above %d", V, kSampleMaxV);
  SampleArgs s;
  *bytes = carve_sample(nullptr, N, V, s);
  return ok();
}

PLP_API int plp_sample_tokens(const plp_sample_args* a, void* ws, size_t ws_bytes, hipStream_t st) {
  if (!a) return fail(PLP_E_INVALID, "args is NULL");
  if (a->struct_size < sizeof(plp_sample_args))
    return fail(PLP_E_INVALID, "args->struct_size %u < %zu", a->struct_size, sizeof(plp_sample_args));
  if (!known_dtype(a->dtype)) return fail(PLP_E_INVALID, "unknown dtype %d", a->dtype);
  size_t need = 0;
  int rc = plp_sample_tokens_workspace_size(a->N, a->V, &need);
  if (rc) return rc;
  if (a->row_stride < 0) return fail(PLP_E_INVALID, "row_stride must be >= 0");
  if (!a->temperature_rows && (!(a->temperature >= 0.f) || !isfinite(a->temperature)))
    return fail(PLP_E_INVALID, "temperature must be finite and >= 0");
  if (!a->top_k_rows && a->top_k < 0) return fail(PLP_E_INVALID, "top_k must be >= 0");
  if (!a->top_p_rows && !(a->top_p >= 0.f && a->top_p <= 1.f))
    return fail(PLP_E_INVALID, "top_p must lie in [0, 1]");
  if (!a->min_p_rows && !(a->min_p >= 0.f && a->min_p <= 1.f))
    return fail(PLP_E_INVALID, "min_p must lie in [0, 1]");
  if (a->N == 0) return ok();
  if (!a->logits || !a->uniforms || !a->token_out)
    return fail(PLP_E_INVALID, "logits, uniforms and token_out are required");
  const void* f32[] = {a->uniforms,   a->temperature_rows, a->top_k_rows,   a->top_p_rows,
                       a->min_p_rows, a->logp_out,         a->kept_logp_out};
  for (const void* p : f32)
    if (misaligned(p, 4)) return fail(PLP_E_INVALID, "an array is not aligned to its elements");
  if (misaligned(a->logits, esize(a->dtype)) || misaligned(a->token_out, 8))
    return fail(PLP_E_INVALID, "an array is not aligned to its elements");
  int64_t span = 0;  // bytes from the first row's start to the last one's end
  if (__builtin_mul_overflow(a->N - 1, a->row_stride, &span) || __builtin_add_overflow(span, (int64_t)a->V, &span) ||
      __builtin_mul_overflow(span, (int64_t)esize(a->dtype), &span))
    return fail(PLP_E_INVALID, "row_stride=%lld is past the address space", (long long)a->row_stride);
  const size_t rb = (size_t)a->N * 4;
  const Range in[] = {{a->logits, (size_t)span},  {a->uniforms, rb},   {a->temperature_rows, rb},
                      {a->top_k_rows, rb},        {a->top_p_rows, rb}, {a->min_p_rows, rb}},
              out[] = {{a->token_out, rb * 2}, {a->logp_out, rb}, {a->kept_logp_out, rb}};
  rc = check_apart(in, out);
  if (rc) return rc;
  rc = check_ws(ws, ws_bytes, need);
  if (rc) return rc;
  SampleArgs s;
  carve_sample(ws, a->N, a->V, s);
  s.logits = a->logits;
  s.uniforms = a->uniforms;
  s.tau = a->temperature;
  s.top_p = a->top_p;
  s.min_p = a->min_p;
  s.top_k = a->top_k;
  s.tau_rows = a->temperature_rows;
  s.top_p_rows = a->top_p_rows;
  s.min_p_rows = a->min_p_rows;
  s.top_k_rows = a->top_k_rows;
  s.token = a->token_out;
  s.logp = a->logp_out;
  s.kept_logp = a->kept_logp_out;
  s.N = a->N;
  s.stride = a->row_stride;
  s.V = a->V;
  s.dtype = a->dtype;
  HIP_TRY(launch_sample(s, st));
  return ok();
}

}  // extern "C"
