// Host side of the verification of drafted tokens: argument checks and the
// workspace's size. No allocation, no host synchronisation.
#include <math.h>

#include "checks.h"
#include "verify_ops.h"

using namespace plp;

namespace {

int check_sizes(int64_t B, int32_t K, int32_t V) {
  if (B < 0 || B >= kMaxRows) return fail(PLP_E_INVALID, "B=%lld outside [0, 2^31)", (long long)B);
  if (K < 0) return fail(PLP_E_INVALID, "K must be >= 0 (got %d)", K);
  if (V < 1) return fail(PLP_E_INVALID, "V must be >= 1 (got %d)", V);
  if (K > kVerifyMaxK) return fail(PLP_E_UNSUPPORTED, "K=%d is above %d", K, kVerifyMaxK);
  if (V > kSampleMaxV) return fail(PLP_E_UNSUPPORTED, "V=%d is above %d", V, kSampleMaxV);
  return PLP_OK;
}

size_t carve_verify(void* ws, int64_t B, int32_t K, int32_t V, bool drafts, VerifyArgs& a) {
  Carver c(ws);
  const size_t rows = (size_t)B * verify_rows(K, drafts);
  a.block_sum = c.take<double>(rows * sample_blocks(V));
  a.block_max = c.take<float>(rows * sample_blocks(V));
  a.rows = c.take<VerifyRow>(rows);
  a.chance = c.take<double>((size_t)B * K * 2);
  a.refused = c.take<int32_t>((size_t)B);
  a.verdicts = c.take<Verdict>((size_t)B);
  a.rest = c.take<double>((size_t)B * verify_blocks(V));
  return c.off;
}

int check_limits(const plp_token_limits& t, const char* who) {
  if (!t.temperature_rows && (!(t.temperature >= 0.f) || !isfinite(t.temperature)))
    return fail(PLP_E_INVALID, "%s temperature must be finite and >= 0", who);
  if (!t.top_k_rows && t.top_k < 0) return fail(PLP_E_INVALID, "%s top_k must be >= 0", who);
  if (!t.top_p_rows && !(t.top_p >= 0.f && t.top_p <= 1.f))
    return fail(PLP_E_INVALID, "%s top_p must lie in [0, 1]", who);
  if (!t.min_p_rows && !(t.min_p >= 0.f && t.min_p <= 1.f))
    return fail(PLP_E_INVALID, "%s min_p must lie in [0, 1]", who);
  if (misaligned(t.temperature_rows, 4) || misaligned(t.top_k_rows, 4) || misaligned(t.top_p_rows, 4) ||
      misaligned(t.min_p_rows, 4))
    return fail(PLP_E_INVALID, "an array is not aligned to its elements");
  return PLP_OK;
}

// Bytes from the first row's start to the last one's end; false if they are
// past the address space.
bool span_of(int64_t B, int64_t rows, int64_t seq_stride, int64_t row_stride, int32_t V, int32_t dtype, size_t* bytes) {
  int64_t a = 0, b = 0;
  if (B == 0 || rows == 0) {
    *bytes = 0;
    return true;
  }
  if (__builtin_mul_overflow(B - 1, seq_stride, &a) || __builtin_mul_overflow(rows - 1, row_stride, &b) ||
      __builtin_add_overflow(a, b, &a) || __builtin_add_overflow(a, (int64_t)V, &a) ||
      __builtin_mul_overflow(a, (int64_t)esize(dtype), &a))
    return false;
  *bytes = (size_t)a;
  return true;
}

VerifyRows rows_of(const void* logits, int64_t seq_stride, int64_t row_stride, const plp_token_limits& t) {
  VerifyRows r;
  r.logits = logits;
  r.seq_stride = seq_stride;
  r.row_stride = row_stride;
  r.tau = t.temperature;
  r.top_k = t.top_k;
  r.top_p = t.top_p;
  r.min_p = t.min_p;
  r.tau_seq = t.temperature_rows;
  r.top_k_seq = t.top_k_rows;
  r.top_p_seq = t.top_p_rows;
  r.min_p_seq = t.min_p_rows;
  return r;
}

}  // namespace

extern "C" {

PLP_API int plp_verify_tokens_workspace_size(int64_t B, int32_t K, int32_t V, int32_t draft_logits, size_t* bytes) {
  if (!bytes) return fail(PLP_E_INVALID, "bytes is NULL");
  int rc = check_sizes(B, K, V);
  if (rc) return rc;
  VerifyArgs v;
  *bytes = carve_verify(nullptr, B, K, V, draft_logits != 0, v);
  return ok();
}

PLP_API int plp_verify_tokens(const plp_verify_args* a, void* ws, size_t ws_bytes, hipStream_t st) {
  if (!a) return fail(PLP_E_INVALID, "args is NULL");
  if (a->struct_size < sizeof(plp_verify_args))
    return fail(PLP_E_INVALID, "args->struct_size %u < %zu", a->struct_size, sizeof(plp_verify_args));
  if (!known_dtype(a->dtype)) return fail(PLP_E_INVALID, "unknown dtype %d", a->dtype);
  int rc = check_sizes(a->B, a->K, a->V);
  if (rc) return rc;
  const bool drafts = a->draft_logits && a->K > 0;
  if (a->seq_stride < 0 || a->row_stride < 0 || (drafts && (a->draft_seq_stride < 0 || a->draft_row_stride < 0)))
    return fail(PLP_E_INVALID, "strides must be >= 0");
  rc = check_limits(a->target, "the target's");
  if (!rc && drafts) rc = check_limits(a->draft, "the draft's");
  if (rc) return rc;
  if (a->B == 0) return ok();
  if (!a->logits || !a->uniforms || !a->tokens_out || !a->accepted_out || (a->K > 0 && !a->draft_tokens))
    return fail(PLP_E_INVALID, "logits, draft_tokens, uniforms, tokens_out and accepted_out are required");
  const size_t e = esize(a->dtype);
  if (misaligned(a->logits, e) || misaligned(a->draft_logits, e) || misaligned(a->draft_tokens, 8) ||
      misaligned(a->tokens_out, 8) || misaligned(a->num_drafts, 4) || misaligned(a->uniforms, 4) ||
      misaligned(a->accepted_out, 4) || misaligned(a->logp_out, 4) || misaligned(a->kept_logp_out, 4))
    return fail(PLP_E_INVALID, "an array is not aligned to its elements");
  size_t span = 0, draft_span = 0;
  if (!span_of(a->B, (int64_t)a->K + 1, a->seq_stride, a->row_stride, a->V, a->dtype, &span) ||
      (drafts && !span_of(a->B, a->K, a->draft_seq_stride, a->draft_row_stride, a->V, a->dtype, &draft_span)))
    return fail(PLP_E_INVALID, "the strides are past the address space");
  VerifyArgs v;
  const size_t need = carve_verify(ws, a->B, a->K, a->V, drafts, v);
  const size_t sb = (size_t)a->B * 4, ob = sb * (a->K + 1);
  const plp_token_limits &t = a->target, &d = a->draft;
  const Range in[] = {{a->logits, span},
                      {drafts ? a->draft_logits : nullptr, draft_span},
                      {a->draft_tokens, sb * 2 * a->K},
                      {a->num_drafts, sb},
                      {a->uniforms, ob},
                      {t.temperature_rows, sb},
                      {t.top_k_rows, sb},
                      {t.top_p_rows, sb},
                      {t.min_p_rows, sb},
                      {drafts ? d.temperature_rows : nullptr, sb},
                      {drafts ? d.top_k_rows : nullptr, sb},
                      {drafts ? d.top_p_rows : nullptr, sb},
                      {drafts ? d.min_p_rows : nullptr, sb}},
              out[] = {{a->tokens_out, ob * 2}, {a->accepted_out, sb}, {a->logp_out, ob}, {a->kept_logp_out, ob}, {ws, need}};
  rc = check_apart(in, out);
  if (rc) return rc;
  rc = check_ws(ws, ws_bytes, need);
  if (rc) return rc;
  v.of[0] = rows_of(a->logits, a->seq_stride, a->row_stride, a->target);
  v.of[1] = rows_of(drafts ? a->draft_logits : nullptr, a->draft_seq_stride, a->draft_row_stride, a->draft);
  v.draft_tokens = a->draft_tokens;
  v.num_drafts = a->num_drafts;
  v.uniforms = a->uniforms;
  v.tokens = a->tokens_out;
  v.accepted = a->accepted_out;
  v.logp = a->logp_out;
  v.kept_logp = a->kept_logp_out;
  v.B = a->B;
  v.K = a->K;
  v.V = a->V;
  v.dtype = a->dtype;
  HIP_TRY(launch_verify(v, st));
  return ok();
}

}  // extern "C"
