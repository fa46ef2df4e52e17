// The launcher of the verification of drafted tokens; it enqueues on `st` and
// returns the launches' hipError_t, every argument checked by the host
// (verify_api.cpp).
#pragma once

#include "ops.h"

namespace plp {

// Rows of logits and what they are sampled with, one value a sequence or one
// for all.
struct VerifyRows {
  const void* logits;
  int64_t seq_stride, row_stride;
  float tau, top_p, min_p;
  int top_k;
  double rate;  // of the temperature, where that is one for all: the launcher's
  const float *tau_seq, *top_p_seq, *min_p_seq;  // instead of the scalars, or NULL
  const int32_t* top_k_seq;
};
// What the second launch leaves of a row.
struct VerifyRow {
  double mass, whole;  // of the kept weights and of all, the largest logit's being 1
  float most;          // the largest logit
  float tau;
  float least;         // min_p, or -1
  float cut;           // kept are the logits above it, and those equal to it up to index `upto`
  int32_t upto;
  int32_t state;       // kNoRow, kWeights, or kOneToken: the token is `upto`
};
enum { kNoRow = 0, kWeights = 1, kOneToken = 2 };

// How far a sequence is accepted, and what its last token is drawn from.
struct Verdict {
  int32_t count;    // drafts accepted
  int32_t refused;  // whether the next one was refused
  int32_t state;    // kNoRow if the last token has no distribution
  int32_t certain;  // the refused draft where drafts are certain, or -1
  double log_whole, log_mass;  // of the target's row
  VerifyRow p, q;   // the target's row; the draft's, if a draft was refused and has one
};
struct VerifyArgs {
  VerifyRows of[2];  // the targets', and the drafts', whose logits are NULL if they are certain
  const int64_t* draft_tokens;
  const int32_t* num_drafts;
  const float* uniforms;
  int64_t* tokens;
  int32_t* accepted;
  float *logp, *kept_logp;
  // workspace: of every sequence's rows (targets, then drafts) the blocks and
  // what is left of them; the blocks of what the last token is drawn from
  double* block_sum;
  float* block_max;
  VerifyRow* rows;
  double* chance;       // [B][K][2] of each draft: the target's chance of it, and the draft's own
  int32_t* refused;     // [B] a draft that is refused, as far as is known
  Verdict* verdicts;
  double* rest;
  int64_t B;
  int K, V, dtype;
  int skip;  // whether rows look at `refused`, and go by their place in the sequence
  int slot;  // then the first place of a launch: a target's row and its draft's are two places
};
constexpr int kVerifyMaxK = 1024;
inline int verify_rows(int K, bool drafts) { return K + 1 + (drafts ? K : 0); }
// Blocks of 256 logits of a row, from its first.
inline int verify_blocks(int V) { return (V + kSampleBlock - 1) / kSampleBlock; }
hipError_t launch_verify(const VerifyArgs& a, hipStream_t st);

}  // namespace plp
