// Calls of the operators for packed batches, between the C entry points (sl_api.cu) and their kernels: q/k norm and
// rotation, token log probabilities, attention over intervals of keys.
#pragma once

#include "sl_internal.h"

namespace sl {

// Device error code beside those of the tile kernels: an attention plan of other sizes than the call's
constexpr int DEV_BAD_PLAN = 7;

// ---- q/k norm and rotation (sl_rotary.cu)
struct RotaryArgs {
  const void *xq, *xk;        // [n_tok, heads * hd] (backward without the norm: not read)
  int64_t ldxq, ldxk;
  const void *dyq, *dyk;      // backward: the outputs' gradients (null: forward)
  int64_t lddq, lddk;
  void *oq, *ok;
  int64_t ldoq, ldok;
  const int32_t* pos;         // null without rotation (rot = 0)
  const float* inv_freq;      // [rot / 2]
  const void *gq, *gk;        // [hd] gains (null: no norm)
  float eps;
  int64_t n_tok;
  int hq, hkv, hd, rot, pairs;
  float *dgq, *dgk;           // [hd] gradients of the gains (optional)
  float* partial;             // rotary_partial_floats() when a gain gradient is asked for
};
int64_t rotary_partial_floats(int64_t n_tok, int hd);
int rotary(const RotaryArgs& a, cudaStream_t s);

// ---- token log probabilities (sl_logprob.cu)
struct LogprobArgs {
  const void* z;              // [rows, vocab] bf16 or fp32
  int fp32;
  int64_t ld, rows, vocab;
  const int32_t* target;
  float *logp, *stats;        // stats: [rows][2]
  float* entropy;             // optional (read by the backward when g_entropy is given)
  int k;
  int32_t* top_ids;
  float* top_logp;
  const float *g_logp, *g_entropy;
  void* dz;
  int64_t ldd;
};
// Both return 0, 1 (size out of range), 5 (launch).
int token_logprobs_fwd(const LogprobArgs& a, cudaStream_t s);
int token_logprobs_bwd(const LogprobArgs& a, cudaStream_t s);

// ---- attention over intervals of keys (sl_attention_mask.cu)
int64_t attention_plan_bytes(int n_seq, int S);
int attention_plan(const int32_t* row_lo, const int32_t* row_hi, int n_seq, int S, void* plan, cudaStream_t s);
struct MaskedArgs {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  void* o;                    // forward
  int64_t ldo;
  const float* lse;           // written by the forward
  const void* plan;
  int n_seq, S, hq, hkv, hd;
  float scale, cap;           // scale 0: 1 / sqrt(hd); cap 0: none
  const float* slopes;        // [hq] or null
  int* err;
  const void* d_o;
  int64_t lddo;
  void *dq, *dk, *dv;
  int64_t lddq, lddk, lddv;
  void* scratch;              // attention_masked_scratch() bytes: D per query row and head
};
// The scale itself (0: 1 / sqrt(hd)), mul of the kernels' score() and cap_mul of their tanh_n()
void masked_score_constants(float scale, float cap, int hd, float* sc, float* mul, float* cap_mul);
// Both return 0, 2 (tensor map), 5 (launch).
int attention_masked_fwd(const MaskedArgs& a, cudaStream_t s);
int attention_masked_bwd(const MaskedArgs& a, cudaStream_t s);
size_t attention_masked_scratch(int n_seq, int S, int hq);

}  // namespace sl
