// Parameter blocks and launchers of the attention block's operators
// (include/moe_v41_attn.h), shared by their kernels and the C entry points.
#pragma once

#include "../../include/moe_v41_attn.h"
#include "ops.h"

namespace moe {

// Rotation of m rows of heads_q heads; with kv.page_size > 0 also the append of
// heads_kv keys (rotated) and values (copied).
struct RopeParams {
  moe_v41_rope_cfg c;
  int m, heads_q, heads_kv;
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  int out_type;                                   // of q_out and the caches
  long long ldq, ldq_head, ldo, ldo_head, ldk, ldv;
  const int* pos;
  const double* freqs;
  moe_v41_kv_cfg kv;
  moe_v41_seqs s;
  unsigned* status;
};

struct AttnParams {
  moe_v41_attn_cfg c;
  moe_v41_seqs s;
  int m;
  const void *q, *k_cache, *v_cache;
  void* out;
  float* lse;
  long long ldq, ldo, ld_lse;
};

int launch_rope(const RopeParams& p, cudaStream_t s);
size_t attn_workspace_bytes(const moe_v41_attn_cfg& c);
int launch_paged_attention(const AttnParams& p, int max_new, void* ws, cudaStream_t s);

}  // namespace moe
