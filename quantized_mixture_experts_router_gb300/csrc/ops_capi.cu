// C entry points of the operators around the MoE layer (declared in
// include/moe_v41_ops.h): argument checks on the host, then the launch.
#include "ops.h"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_type(int t) { return t == MOE_T_F32 || t == MOE_T_BF16 || t == MOE_T_F16; }
bool is_half_type(int t) { return t == MOE_T_BF16 || t == MOE_T_F16; }

int check_q4(const moe_v41_q4_cfg* c) {
  if (!c) return MOE_ERR_ARG;
  if (c->n < 1 || c->n > (1 << 24)) return MOE_ERR_ARG;
  if (c->k < 32 || c->k > 32768 || c->k % 32) return MOE_ERR_ARG;
  if (c->group != 32 && c->group != 64 && c->group != 128) return MOE_ERR_ARG;
  if (!is_half_type(c->x_type) || !is_half_type(c->scale_type) || !is_type(c->out_type)) return MOE_ERR_ARG;
  if (c->max_tokens < 1 || c->max_tokens > 65536) return MOE_ERR_ARG;
  return MOE_OK;
}

int check_norm(const moe_v41_norm_cfg* c) {
  if (!c) return MOE_ERR_ARG;
  if (c->dim < 1 || c->dim > 16384) return MOE_ERR_ARG;
  if (c->post_kind < MOE_NORM_NONE || c->post_kind > MOE_NORM_LAYER) return MOE_ERR_ARG;
  if (c->pre_kind < MOE_NORM_NONE || c->pre_kind > MOE_NORM_LAYER) return MOE_ERR_ARG;
  if (!is_type(c->y_type) || !is_type(c->h_type) || !is_type(c->x_type) || !is_type(c->w_type)) return MOE_ERR_ARG;
  if (c->gate_kind < MOE_GATE_NONE || c->gate_kind > MOE_GATE_TOKEN) return MOE_ERR_ARG;
  if (c->gate_kind != MOE_GATE_NONE && (!is_type(c->gate_type) || c->gate_group < 1)) return MOE_ERR_ARG;
  if (!(c->eps >= 0.0f)) return MOE_ERR_ARG;
  return MOE_OK;
}

int check_logprob(const moe_v41_logprob_cfg* c) {
  if (!c) return MOE_ERR_ARG;
  if (c->vocab < 1 || c->vocab > (1 << 28) || !is_type(c->logit_type)) return MOE_ERR_ARG;
  if (c->top_k < 0 || c->top_k > 32) return MOE_ERR_ARG;
  // 1 / T and log2(e) / T are finite normal numbers, and a difference of logits that overflows f32 has no weight
  if (!(c->temperature >= 1.0e-36f) || !(c->temperature <= 1.0e36f)) return MOE_ERR_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_v41_q4_workspace_bytes(const moe_v41_q4_cfg* cfg) {
  return check_q4(cfg) == MOE_OK ? q4_workspace_bytes(*cfg) : 0;
}

int moe_v41_q4_linear(const moe_v41_q4_cfg* cfg, const void* x, int m, int64_t ldx, const void* w, const void* scales,
                      const uint8_t* zeros, void* out, int64_t ldo, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_q4(cfg);
  if (rc) return rc;
  if (m < 0 || m > cfg->max_tokens) return MOE_ERR_ARG;
  if (m == 0) return MOE_OK;
  if (!x || !w || !scales || !out || ldx < cfg->k || ldo < cfg->n) return MOE_ERR_ARG;
  if (!aligned(x, 16) || ldx % 8 || !aligned(w, 16) || !aligned(scales, 2) ||
      !aligned(out, (size_t)type_bytes(cfg->out_type)))
    return MOE_ERR_ALIGN;
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
  if (ws_bytes < q4_workspace_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  Q4Params p{};
  p.m = m; p.n = cfg->n; p.k = cfg->k; p.group = cfg->group; p.ng = (cfg->k + cfg->group - 1) / cfg->group;
  p.x_type = cfg->x_type; p.scale_type = cfg->scale_type; p.out_type = cfg->out_type;
  p.x = static_cast<const uint16_t*>(x); p.ldx = ldx;
  p.w = static_cast<const uint8_t*>(w);
  p.scales = static_cast<const uint16_t*>(scales); p.zeros = zeros;
  p.out = out; p.ldo = ldo;
  return launch_q4_linear(p, ws, (cudaStream_t)stream);
}

int moe_v41_block_norm(const moe_v41_norm_cfg* cfg, int m, const void* y, int64_t ldy, const void* post_w,
                       const void* post_b, const void* gate, int64_t ldg, const void* h, int64_t ldh, void* h_out,
                       int64_t ldh_out, const void* pre_w, const void* pre_b, void* x_out, int64_t ldx, void* stream) {
  int rc = check_norm(cfg);
  if (rc) return rc;
  if (m < 0) return MOE_ERR_ARG;
  if (m == 0) return MOE_OK;
  const int64_t d = cfg->dim;
  if (!h || ldh < d || (!h_out && !x_out) || (h_out && ldh_out < d) || (x_out && ldx < d)) return MOE_ERR_ARG;
  if (h_out == h && ldh_out != ldh) return MOE_ERR_ARG;
  if (y) {
    if (ldy < d) return MOE_ERR_ARG;
    if (cfg->gate_kind != MOE_GATE_NONE && !gate) return MOE_ERR_ARG;
    if (cfg->gate_kind == MOE_GATE_ROW && ldg < d) return MOE_ERR_ARG;
    if (cfg->gate_kind != MOE_GATE_NONE && !aligned(gate, (size_t)type_bytes(cfg->gate_type))) return MOE_ERR_ALIGN;
    if (!aligned(y, (size_t)type_bytes(cfg->y_type))) return MOE_ERR_ALIGN;
  }
  const size_t wa = (size_t)type_bytes(cfg->w_type), ha = (size_t)type_bytes(cfg->h_type);
  if (!aligned(h, ha) || !aligned(h_out, ha) || !aligned(x_out, (size_t)type_bytes(cfg->x_type)) ||
      !aligned(post_w, wa) || !aligned(post_b, wa) || !aligned(pre_w, wa) || !aligned(pre_b, wa))
    return MOE_ERR_ALIGN;
  NormParams p{};
  p.c = *cfg; p.m = m;
  p.y = y; p.post_w = post_w; p.post_b = post_b; p.gate = gate; p.h = h; p.pre_w = pre_w; p.pre_b = pre_b;
  p.h_out = h_out; p.x_out = x_out;
  p.ldy = ldy; p.ldg = ldg; p.ldh = ldh; p.ldh_out = ldh_out; p.ldx = ldx;
  return launch_block_norm(p, (cudaStream_t)stream);
}

int moe_v41_token_logprobs(const moe_v41_logprob_cfg* cfg, const void* logits, int m, int64_t ld,
                           const uint32_t* allowed, int64_t ld_allowed, const int32_t* target, float* logprob,
                           int32_t* rank, float* lse, float* entropy, float* top_logprob, int32_t* top_id,
                           void* stream) {
  int rc = check_logprob(cfg);
  if (rc) return rc;
  if (m < 0 || m > (1 << 30)) return MOE_ERR_ARG;
  if (m == 0) return MOE_OK;
  if (!logits || ld < cfg->vocab) return MOE_ERR_ARG;
  if (allowed && ld_allowed < (cfg->vocab + 31) / 32) return MOE_ERR_ARG;
  if ((logprob || rank) && !target) return MOE_ERR_ARG;
  if (cfg->top_k > 0 && (!top_logprob || !top_id)) return MOE_ERR_ARG;
  if (!logprob && !rank && !lse && !entropy && cfg->top_k == 0) return MOE_ERR_ARG;
  if (!aligned(logits, (size_t)type_bytes(cfg->logit_type)) || !aligned(allowed, 4) || !aligned(target, 4) ||
      !aligned(logprob, 4) || !aligned(rank, 4) || !aligned(lse, 4) || !aligned(entropy, 4) ||
      !aligned(top_logprob, 4) || !aligned(top_id, 4))
    return MOE_ERR_ALIGN;
  LogprobParams p{};
  p.c = *cfg; p.m = m; p.logits = logits; p.ld = ld; p.allowed = allowed; p.ld_allowed = ld_allowed;
  p.target = target; p.logprob = logprob; p.rank = rank; p.lse = lse; p.entropy = entropy;
  p.top_logprob = top_logprob; p.top_id = top_id;
  return launch_token_logprobs(p, (cudaStream_t)stream);
}

}  // extern "C"
