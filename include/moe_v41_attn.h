/* moe_v41 — the operators of an attention block around the MoE layer: rotary
 * positions, appending keys and values to a paged cache, and the attention of
 * new tokens over it (a decode step's single tokens, drafted tokens, chunks of
 * a prompt, whole prompts, and cross attention).
 *
 * Conventions are those of moe_v41_ops.h.  Pitches count elements and are
 * 64-bit.  The heads of a token lie behind one another (head h of a row at
 * h * head_dim) unless a call has a pitch for them.
 */
#ifndef MOE_V41_ATTN_H
#define MOE_V41_ATTN_H

#include "moe_v41_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a sequence's page number lay outside 0 .. n_pages - 1, or a length beyond its
 * table: see the call (read with moe_v41_read_status where it lies in a workspace) */
enum { MOE_STATUS_BAD_PAGE = 8u };

/* ------------------------------------------------------------ rotary positions
 * Of each head, rot_dim values from rot_first on are rotated in pairs (a, b):
 *   a' = magnitude (a cos t - b sin t)    b' = magnitude (b cos t + a sin t)
 * with t = pos * freqs[i] for pair i, the others copied.  inverse turns by -t:
 * the transposed map, which takes the output's gradient to the input's. */
enum {
  MOE_ROPE_HALF = 0,        /* pair i: values i and i + rot_dim / 2 */
  MOE_ROPE_INTERLEAVED = 1  /* pair i: values 2 i and 2 i + 1 */
};

typedef struct {
  int32_t head_dim;   /* 1..1024 */
  int32_t rot_dim;    /* even, 0..head_dim - rot_first; 0 rotates nothing */
  int32_t rot_first;
  int32_t layout;     /* MOE_ROPE_* */
  int32_t x_type;     /* MOE_T_* of the values given */
  int32_t inverse;    /* non-zero: turn back */
  float magnitude;    /* finite; 1, or the factor of a scaled rotation */
} moe_v41_rope_cfg;

/* Angles per position (radians) of the rot_dim / 2 pairs, on the HOST, and the
 * magnitude that belongs to them (NULL if not wanted).  With f_i = base^(-2 i / rot_dim)
 * and a context `factor` times as long as the one trained on (`trained` positions):
 *   NONE    f_i
 *   LINEAR  f_i / factor
 *   BASE    the same with base * factor^(rot_dim / (rot_dim - 2)): the slowest pair
 *           is stretched by factor, the fastest not at all
 *   PARTS   g f_i + (1 - g) f_i / factor, where g goes from 0 at one turn within
 *           the trained positions to 1 at 32 turns; magnitude 0.1 ln(factor) + 1
 *           (the by-parts scaling of YaRN, Peng et al. 2023, as the paper writes it).
 *           g is linear in the turns, and 1 and 32 are fixed.  Model code that
 *           interpolates over the pair's number i between two rounded bounds, or has
 *           other bounds or another magnitude, gives other angles for the same
 *           factor: its checkpoints need a table of its own making. */
enum { MOE_ROPE_SCALE_NONE = 0, MOE_ROPE_SCALE_LINEAR = 1, MOE_ROPE_SCALE_BASE = 2, MOE_ROPE_SCALE_PARTS = 3 };
MOE_API int moe_v41_rope_freqs(int rot_dim, double base, int kind, double factor, int trained, double* freqs,
                               float* magnitude);

/* x and out [m, heads, head_dim] of x_type: rows ldx (ldo) apart, heads ldx_head
 * (ldo_head) apart, any values of at least head_dim that keep them from
 * overlapping; out may be x at the same pitches.  pos int32 [m] and freqs f64
 * [rot_dim / 2] on the device (both may be NULL when rot_dim is 0).  Angles are
 * computed and reduced in 64 bits.  m < 2^24, heads <= 65536. */
MOE_API int moe_v41_rope(const moe_v41_rope_cfg* cfg, int m, int heads, const void* x, int64_t ldx, int64_t ldx_head,
                         const int32_t* pos, const double* freqs, void* out, int64_t ldo, int64_t ldo_head,
                         void* stream);

/* ---------------------------------------------------------------- paged cache
 * Keys and values of one layer in pages of page_size tokens.  Value d of head h
 * of the token in slot s of page p lies at
 *   p * page_pitch + s * token_pitch + h * head_pitch + d
 * in k_cache, and at the same place in v_cache. */
typedef struct {
  int32_t kv_heads;   /* 1..1024 */
  int32_t head_dim;   /* a multiple of 8, 16..128 */
  int32_t page_size;  /* a power of two, 8..4096 */
  int32_t n_pages;    /* 1..2^31 - 1 */
  int32_t type;       /* MOE_T_BF16 or MOE_T_F16 */
  int32_t reserved;
  int64_t page_pitch, token_pitch, head_pitch;  /* multiples of 8, at least head_dim, below 2^38 */
} moe_v41_kv_cfg;

/* The sequences of a call; the arrays are on the device, so that a captured step
 * serves every length.  New token i of sequence b is row cu_new[b] + i of the
 * call's tensors, and its position is kv_len[b] - n + i, n = cu_new[b + 1] -
 * cu_new[b] of them.  Rows behind the last sequence's belong to nobody: what
 * they hold has no influence, and their outputs stay as they were.  A length below 0 counts as 0;
 * rows from m on are left out. */
typedef struct {
  int32_t batch;           /* sequences: 0..65536 */
  int32_t max_pages;       /* entries of a table row: 1..2^27, max_pages * page_size <= 2^30 */
  const int32_t* cu_new;   /* [batch + 1], ascending */
  const int32_t* kv_len;   /* [batch] tokens of the sequence, the new ones among them (cross attention: of
                              the encoder's states) */
  const int32_t* table;    /* [batch, max_pages] pages of the sequence in order, rows ld_table apart */
  int64_t ld_table;
} moe_v41_seqs;

/* Appends m rows' keys and values to the cache at their positions, keys rotated;
 * with q also rotates the queries into q_out.  rope->x_type is the type of k, v
 * and q; the cache and q_out have kv's type (one rounding).  k and v
 * [m, kv_heads, head_dim] (pitches ldk, ldv), q and q_out [m, q_heads, head_dim]
 * (both NULL: none; q_out may be q at the same pitch and type).  freqs as above.
 * pos int32 [m]: positions to rotate by instead of those in the sequence, or
 * NULL.  A token before position 0, beyond its table or on a page outside
 * 0 .. n_pages - 1 is not stored; the latter two set MOE_STATUS_BAD_PAGE in
 * *status (device, may be NULL; bits are added, never cleared).  The pages that a
 * call writes are its sequences' own.  m < 2^24. */
MOE_API int moe_v41_kv_append(const moe_v41_kv_cfg* kv, const moe_v41_rope_cfg* rope, const moe_v41_seqs* seqs, int m,
                              const void* k, int64_t ldk, const void* v, int64_t ldv, void* k_cache, void* v_cache,
                              int q_heads, const void* q, int64_t ldq, void* q_out, int64_t ldq_out,
                              const double* freqs, const int32_t* pos, uint32_t* status, void* stream);

/* ------------------------------------------------- attention over a paged cache
 *   out[t, h] = sum_j softmax_j(scale q[t, h] . K[j, h / group]) V[j, h / group]
 *   lse[t, h] = log sum_j exp(scale q[t, h] . K[j, h / group])
 * over the cached tokens j of t's sequence that t sees, group = heads / kv_heads.
 * With p the position of t:
 *   causal             0 <= j <= p, and j > p - window when window > 0
 *   causal == 0        every j < kv_len (cross attention)
 *  - The new tokens' own keys and values have been appended before.
 *  - A token that sees nothing (or only scores of -inf): out 0, lse -inf.
 *  - What lies in slots that none of a sequence's new tokens sees has no
 *    influence, whatever it holds; pages that hold no slot that one of them sees
 *    are not looked up.  A key that a token does not see has none on it either;
 *    but an infinity or a NaN among the values that one new token sees may make
 *    NaN of the outputs of the sequence's others (a product with weight zero).
 *  - Scores, maxima and sums are f32.  exp(score - maximum) is rounded once to the
 *    cache's type, as the tensor cores take it with the values; outputs are
 *    rounded once more to that type.
 *  - A page outside 0 .. n_pages - 1 reads as zeros, and what lies beyond the table
 *    (kv_len > max_pages * page_size) is not seen; either sets MOE_STATUS_BAD_PAGE
 *    in the workspace.
 *  - A wait that runs out (a copy that never lands) sets MOE_STATUS_TIMEOUT;
 *    what it concerns is NaN, and the workspace is ready for the next call.
 *  - Results do not depend on the order in which blocks run. */
typedef struct {
  moe_v41_kv_cfg kv;
  int32_t heads;   /* query heads: a multiple of kv_heads, up to 4096 */
  int32_t causal;
  int32_t window;  /* 0: all; else causal, 1..2^30 */
  float scale;     /* 1e-36..1e36 */
} moe_v41_attn_cfg;

/* Bytes of workspace (0 for an invalid configuration): whatever the number of
 * tokens and sequences.  Prepare it once with moe_v41_workspace_init; it serves
 * one call at a time, and every call leaves it ready for the next. */
MOE_API size_t moe_v41_attn_workspace_bytes(const moe_v41_attn_cfg* cfg);

/* q and out [m, heads, head_dim] of kv.type (pitches ldq, a multiple of 8 with q
 * 16-B aligned, and ldo, the same), lse f32 [m, heads] (pitch ld_lse) or NULL.
 * out overlaps nothing that the call reads.
 * max_new: about how many new tokens the longest sequence has; it chooses the
 * kernel, and results are right for any.  m * heads <= 2^30. */
MOE_API int moe_v41_paged_attention(const moe_v41_attn_cfg* cfg, const moe_v41_seqs* seqs, int m, int max_new,
                                    const void* q, int64_t ldq, const void* k_cache, const void* v_cache, void* out,
                                    int64_t ldo, float* lse, int64_t ld_lse, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
