/* moe_v41 — the operators of a decode or prompt step around the MoE layer:
 * the norms before and after a block, products with 4-bit weights, and the log
 * probabilities of given tokens.
 *
 * Conventions are those of moe_v41.h: caller-owned device pointers, every call
 * asynchronous on `stream`, host-visible errors as MOE_ERR_*, nothing
 * allocated.  Row pitches (ld*) count elements, not bytes, and may be any
 * value of at least the row's length unless a call states more; 64-bit row
 * offsets are used throughout.  A call for zero tokens checks its
 * configuration, returns MOE_OK and launches nothing.
 */
#ifndef MOE_V41_OPS_H
#define MOE_V41_OPS_H

#include "moe_v41.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of the operators' tensors */
enum { MOE_T_F32 = 0, MOE_T_BF16 = 1, MOE_T_F16 = 2 };

/* ------------------------------------------------ 4-bit weights, group scales
 *   out[t, r] = sum_k x[t, k] * s[r, k / group] * (q[r, k] - z[r, k / group])
 * q and z in 0..15.  Sums are f32, with more than eight tokens from a group's
 * sum of (q - z) x on (which then has to stay in the range of f32); each out is
 * rounded once to its type. */
typedef struct {
  int32_t n;           /* rows of the weight (outputs per token): 1..2^24 */
  int32_t k;           /* inputs per token: a multiple of 32, 32..32768 */
  int32_t group;       /* weights per scale: 32, 64 or 128; the last group may be shorter */
  int32_t x_type;      /* MOE_T_BF16 or MOE_T_F16 */
  int32_t scale_type;  /* MOE_T_BF16 or MOE_T_F16 */
  int32_t out_type;    /* MOE_T_F32, MOE_T_BF16 or MOE_T_F16 */
  int32_t max_tokens;  /* largest m the workspace is sized for: 1..65536 */
} moe_v41_q4_cfg;

/* Bytes of workspace (0 for an invalid configuration).  Prepare it once with
 * moe_v41_workspace_init; it serves one call at a time, and every call leaves
 * it ready for the next.  moe_v41_read_status reads its status word. */
MOE_API size_t moe_v41_q4_workspace_bytes(const moe_v41_q4_cfg* cfg);

/* x [m, k] (pitch ldx, a multiple of 8; 16-B aligned), w u8 [n, k/2] (16-B
 * aligned; the even k of a pair in the low nibble), scales [n, ceil(k/group)],
 * zeros u8 of the same shape or NULL for 8 throughout (codes 0..15), out
 * [m, n] (pitch ldo, aligned to its element).  0 <= m <= cfg->max_tokens.
 * Results do not depend on the order in which blocks run.  When a wait runs
 * out (MOE_STATUS_TIMEOUT), the outputs are invalid: those it concerns are NaN
 * with up to eight tokens, and unwritten with more; the workspace is ready for
 * the next call all the same. */
MOE_API int moe_v41_q4_linear(const moe_v41_q4_cfg* cfg, const void* x, int m, int64_t ldx, const void* w,
                              const void* scales, const uint8_t* zeros, void* out, int64_t ldo, void* ws,
                              size_t ws_bytes, void* stream);

/* --------------------------------------------- norms before and after a block
 *   h' = residual_scale * h + block_scale * gate * N_post(y)
 *   x  = N_pre(h')
 * for each of m rows: y is a block's output (moe_v41_forward's out), h the
 * residual stream, x the next block's input.  With
 *   MOE_NORM_RMS    N(v) = v / sqrt(mean(v^2) + eps) * w + b
 *   MOE_NORM_LAYER  N(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * w + b
 *   MOE_NORM_NONE   N(v) = v
 * (w NULL: 1, b NULL: 0).  Statistics and sums are f32; N_pre works on h'
 * before its rounding to h_type, so x carries one rounding. */
enum { MOE_NORM_NONE = 0, MOE_NORM_RMS = 1, MOE_NORM_LAYER = 2 };
enum {
  MOE_GATE_NONE = 0,  /* 1 */
  MOE_GATE_ROW = 1,   /* gate[t / gate_group, :]; gate_group >= m shares one [dim] gate */
  MOE_GATE_TOKEN = 2  /* gate[t / gate_group], one scalar */
};

typedef struct {
  int32_t dim;         /* 1..16384 */
  int32_t post_kind;   /* MOE_NORM_* of the block's output */
  int32_t pre_kind;    /* MOE_NORM_* of the next block's input */
  int32_t y_type, h_type, x_type;  /* MOE_T_* */
  int32_t w_type;      /* of the norms' weights and biases */
  int32_t gate_kind;   /* MOE_GATE_* */
  int32_t gate_type;   /* MOE_T_* */
  int32_t gate_group;  /* consecutive tokens that share a gate row or scalar, >= 1 */
  float eps;           /* >= 0, added to the mean square */
  float residual_scale;
  float block_scale;
} moe_v41_norm_cfg;

/* y [m, dim] or NULL (then h' = residual_scale * h), h [m, dim], h_out [m, dim]
 * (may be h itself, or NULL when only x is wanted), x_out [m, dim] or NULL (no
 * next block; then h_out is needed).  gate as its kind says, ldg the pitch of
 * its rows.  post_w .. pre_b [dim], each may be NULL.  Pointers are aligned to
 * their element; outputs overlap no input except h_out == h (with
 * ldh_out == ldh).  Rows that a block could not read within two seconds (a copy
 * that never lands) are NaN in h_out and x_out. */
MOE_API int moe_v41_block_norm(const moe_v41_norm_cfg* cfg, int m, const void* y, int64_t ldy, const void* post_w,
                               const void* post_b, const void* gate, int64_t ldg, const void* h, int64_t ldh,
                               void* h_out, int64_t ldh_out, const void* pre_w, const void* pre_b, void* x_out,
                               int64_t ldx, void* stream);

/* ------------------------------------- log probabilities of given tokens
 * z = logit / temperature over the allowed entries of a row,
 *   lse = log sum exp z          logprob = z[target] - lse
 *   entropy = lse - sum p z      rank = 1 + number of allowed z_j > z[target]
 * and the top_k largest entries by descending z, equal ones by ascending id.
 *  - An entry is allowed when bit (id & 31) of allowed[row, id / 32] is set, or
 *    when allowed is NULL.  What a masked place holds has no influence.
 *  - A row with nothing allowed, or with -inf alone: lse and logprobs -inf,
 *    entropy 0.  Fewer than top_k allowed entries: the rest are id -1, -inf.
 *  - A masked target counts as -inf.  Target -1: not scored, logprob 0 and
 *    rank 0; any other target outside the vocabulary: logprob NaN, rank -1.
 *  - NaN or +inf in an allowed place: the row's lse, entropy and logprobs are
 *    NaN.  Ids and rank stay defined: a NaN ranks below every number (so the
 *    rank of a NaN target is 1 + the number of allowed entries that are
 *    numbers).
 *  - Rows that a block could not read within two seconds (a copy that never
 *    lands): lse, entropy and logprobs NaN, ids and the rank of a target -1. */
typedef struct {
  int32_t vocab;       /* 1..2^28 */
  int32_t logit_type;  /* MOE_T_* */
  int32_t top_k;       /* 0..32 */
  float temperature;   /* 1e-36..1e36 */
} moe_v41_logprob_cfg;

/* logits [m, vocab] (pitch ld, aligned to the element), allowed u32
 * [m, ceil(vocab/32)] (pitch ld_allowed) or NULL, target i32 [m], m <= 2^30.  Each of
 * logprob f32 [m], rank i32 [m], lse f32 [m], entropy f32 [m] may be NULL
 * (target too, when neither logprob nor rank is asked for); top_logprob f32
 * [m, top_k] and top_id i32 [m, top_k] are needed when top_k > 0. */
MOE_API int moe_v41_token_logprobs(const moe_v41_logprob_cfg* cfg, const void* logits, int m, int64_t ld,
                                   const uint32_t* allowed, int64_t ld_allowed, const int32_t* target,
                                   float* logprob, int32_t* rank, float* lse, float* entropy, float* top_logprob,
                                   int32_t* top_id, void* stream);

#ifdef __cplusplus
}
#endif
#endif
