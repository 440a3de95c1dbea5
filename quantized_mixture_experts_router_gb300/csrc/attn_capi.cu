// C entry points of the attention block's operators (declared in
// include/moe_v41_attn.h): argument checks on the host, then the launch.
#include <cmath>

#include "attn.h"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_type(int t) { return t == MOE_T_F32 || t == MOE_T_BF16 || t == MOE_T_F16; }

int check_rope(const moe_v41_rope_cfg* c) {
  if (!c) return MOE_ERR_ARG;
  if (c->head_dim < 1 || c->head_dim > 1024) return MOE_ERR_ARG;
  if (c->rot_first < 0 || c->rot_first > c->head_dim) return MOE_ERR_ARG;
  if (c->rot_dim < 0 || c->rot_dim % 2 || c->rot_dim > c->head_dim - c->rot_first) return MOE_ERR_ARG;
  if (c->layout != MOE_ROPE_HALF && c->layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_ARG;
  if (!is_type(c->x_type) || !std::isfinite(c->magnitude)) return MOE_ERR_ARG;
  return MOE_OK;
}

bool pitch_ok(int64_t v, int dim) { return v >= dim && v < (int64_t(1) << 38); }

int check_kv(const moe_v41_kv_cfg* c) {
  if (!c) return MOE_ERR_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 1024 || c->n_pages < 1) return MOE_ERR_ARG;
  if (c->head_dim < 16 || c->head_dim > 128 || c->head_dim % 8) return MOE_ERR_ARG;
  if (c->page_size < 8 || c->page_size > 4096 || (c->page_size & (c->page_size - 1))) return MOE_ERR_ARG;
  if (c->type != MOE_T_BF16 && c->type != MOE_T_F16) return MOE_ERR_ARG;
  // a pitch that is never stepped by may be anything
  if (!pitch_ok(c->token_pitch, c->head_dim) || (c->n_pages > 1 && !pitch_ok(c->page_pitch, c->head_dim)) ||
      (c->kv_heads > 1 && !pitch_ok(c->head_pitch, c->head_dim)))
    return MOE_ERR_ARG;
  if (c->token_pitch % 8 || (c->n_pages > 1 && c->page_pitch % 8) || (c->kv_heads > 1 && c->head_pitch % 8))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}

int check_seqs(const moe_v41_seqs* s, int page_size) {
  if (!s || s->batch < 0 || s->batch > 65536) return MOE_ERR_ARG;
  if (s->batch == 0) return MOE_OK;
  if (s->max_pages < 1 || (int64_t)s->max_pages * page_size > (int64_t(1) << 30)) return MOE_ERR_ARG;
  if (!s->cu_new || !s->kv_len || !s->table || s->ld_table < s->max_pages) return MOE_ERR_ARG;
  if (!aligned(s->cu_new, 4) || !aligned(s->kv_len, 4) || !aligned(s->table, 4)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

int check_attn(const moe_v41_attn_cfg* c) {
  if (!c) return MOE_ERR_ARG;
  int rc = check_kv(&c->kv);
  if (rc) return rc;
  if (c->heads < 1 || c->heads > 4096 || c->heads % c->kv.kv_heads) return MOE_ERR_ARG;
  if (c->window < 0 || c->window > (1 << 30) || (c->window > 0 && !c->causal)) return MOE_ERR_ARG;
  // scale log2 e is a normal number
  if (!(c->scale >= 1.0e-36f) || !(c->scale <= 1.0e36f)) return MOE_ERR_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_v41_rope_freqs(int rot_dim, double base, int kind, double factor, int trained, double* freqs,
                       float* magnitude) {
  if (rot_dim < 0 || rot_dim > 1024 || rot_dim % 2 || (rot_dim && !freqs)) return MOE_ERR_ARG;
  if (!(base > 0.0) || !std::isfinite(base)) return MOE_ERR_ARG;
  if (kind < MOE_ROPE_SCALE_NONE || kind > MOE_ROPE_SCALE_PARTS) return MOE_ERR_ARG;
  if (kind != MOE_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return MOE_ERR_ARG;
  if (kind == MOE_ROPE_SCALE_BASE && rot_dim == 2) return MOE_ERR_ARG;  // the one pair cannot be stretched and kept
  if (kind == MOE_ROPE_SCALE_PARTS && trained < 1) return MOE_ERR_ARG;
  if (kind == MOE_ROPE_SCALE_BASE && rot_dim) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  const double two_pi = 2.0 * std::acos(-1.0);
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (kind == MOE_ROPE_SCALE_LINEAR) f /= factor;
    if (kind == MOE_ROPE_SCALE_PARTS) {
      const double turns = trained * f / two_pi, g = std::fmin(std::fmax((turns - 1.0) / 31.0, 0.0), 1.0);
      f = g * f + (1.0 - g) * f / factor;
    }
    freqs[i] = f;
  }
  if (magnitude) *magnitude = kind == MOE_ROPE_SCALE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return MOE_OK;
}

int moe_v41_rope(const moe_v41_rope_cfg* cfg, int m, int heads, const void* x, int64_t ldx, int64_t ldx_head,
                 const int32_t* pos, const double* freqs, void* out, int64_t ldo, int64_t ldo_head, void* stream) {
  int rc = check_rope(cfg);
  if (rc) return rc;
  if (m < 0 || m >= (1 << 24) || heads < 0 || heads > 65536) return MOE_ERR_ARG;
  if (m == 0 || heads == 0) return MOE_OK;
  if (!x || !out || (cfg->rot_dim && (!pos || !freqs))) return MOE_ERR_ARG;
  const int64_t d = cfg->head_dim;
  if ((m > 1 && (ldx < d || ldo < d)) || (heads > 1 && (ldx_head < d || ldo_head < d))) return MOE_ERR_ARG;
  if (x == out && ((m > 1 && ldx != ldo) || (heads > 1 && ldx_head != ldo_head))) return MOE_ERR_ARG;
  const size_t a = (size_t)type_bytes(cfg->x_type);
  if (!aligned(x, a) || !aligned(out, a) || !aligned(pos, 4) || !aligned(freqs, 8)) return MOE_ERR_ALIGN;
  RopeParams p{};
  p.c = *cfg; p.m = m; p.heads_q = heads; p.q = x; p.q_out = out; p.out_type = cfg->x_type;
  p.ldq = ldx; p.ldq_head = ldx_head; p.ldo = ldo; p.ldo_head = ldo_head; p.pos = pos; p.freqs = freqs;
  return launch_rope(p, (cudaStream_t)stream);
}

int moe_v41_kv_append(const moe_v41_kv_cfg* kv, const moe_v41_rope_cfg* rope, const moe_v41_seqs* seqs, int m,
                      const void* k, int64_t ldk, const void* v, int64_t ldv, void* k_cache, void* v_cache, int q_heads,
                      const void* q, int64_t ldq, void* q_out, int64_t ldq_out, const double* freqs, const int32_t* pos,
                      uint32_t* status, void* stream) {
  int rc = check_kv(kv);
  if (rc) return rc;
  if ((rc = check_rope(rope))) return rc;
  if (rope->head_dim != kv->head_dim) return MOE_ERR_ARG;
  if ((rc = check_seqs(seqs, kv->page_size))) return rc;
  if (m < 0 || m >= (1 << 24) || q_heads < 0 || q_heads > 4096) return MOE_ERR_ARG;
  if (m == 0 || seqs->batch == 0) return MOE_OK;
  if (!k || !v || !k_cache || !v_cache || (!q) != (!q_out) || (q && q_heads < 1)) return MOE_ERR_ARG;
  if (rope->rot_dim && !freqs) return MOE_ERR_ARG;
  const int64_t d = kv->head_dim, row = d * kv->kv_heads, qrow = d * q_heads;
  if (m > 1 && (ldk < row || ldv < row || (q && (ldq < qrow || ldq_out < qrow)))) return MOE_ERR_ARG;
  if (q && q == q_out && (rope->x_type != kv->type || (m > 1 && ldq != ldq_out))) return MOE_ERR_ARG;
  const size_t a = (size_t)type_bytes(rope->x_type);
  if (!aligned(k, a) || !aligned(v, a) || !aligned(q, a) || !aligned(q_out, 2) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(freqs, 8) || !aligned(pos, 4) || !aligned(status, 4))
    return MOE_ERR_ALIGN;
  RopeParams p{};
  p.c = *rope; p.m = m; p.heads_q = q ? q_heads : 0; p.heads_kv = kv->kv_heads;
  p.q = q; p.k = k; p.v = v; p.q_out = q_out; p.k_cache = k_cache; p.v_cache = v_cache; p.out_type = kv->type;
  p.ldq = ldq; p.ldq_head = d; p.ldo = ldq_out; p.ldo_head = d; p.ldk = ldk; p.ldv = ldv;
  p.pos = pos; p.freqs = freqs; p.kv = *kv; p.s = *seqs; p.status = status;
  return launch_rope(p, (cudaStream_t)stream);
}

size_t moe_v41_attn_workspace_bytes(const moe_v41_attn_cfg* cfg) {
  return check_attn(cfg) == MOE_OK ? attn_workspace_bytes(*cfg) : 0;
}

int moe_v41_paged_attention(const moe_v41_attn_cfg* cfg, const moe_v41_seqs* seqs, int m, int max_new, const void* q,
                            int64_t ldq, const void* k_cache, const void* v_cache, void* out, int64_t ldo, float* lse,
                            int64_t ld_lse, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_attn(cfg);
  if (rc) return rc;
  if ((rc = check_seqs(seqs, cfg->kv.page_size))) return rc;
  if (m < 0 || (int64_t)m * cfg->heads > (int64_t(1) << 30) || max_new < 0) return MOE_ERR_ARG;
  if (m == 0 || seqs->batch == 0) return MOE_OK;
  const int64_t row = (int64_t)cfg->heads * cfg->kv.head_dim;
  if (!q || !k_cache || !v_cache || !out) return MOE_ERR_ARG;
  if (m > 1 && (ldq < row || ldo < row || (lse && ld_lse < cfg->heads))) return MOE_ERR_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lse, 4) ||
      (m > 1 && (ldq % 8 || ldo % 8)))
    return MOE_ERR_ALIGN;
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
  if (ws_bytes < attn_workspace_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  AttnParams p{};
  p.c = *cfg; p.s = *seqs; p.m = m; p.q = q; p.k_cache = k_cache; p.v_cache = v_cache; p.out = out; p.lse = lse;
  p.ldq = ldq; p.ldo = ldo; p.ld_lse = ld_lse;
  return launch_paged_attention(p, max_new, ws, (cudaStream_t)stream);
}

}  // extern "C"
