// A kernel of the operators, built with a bulk copy that can get lost: the one
// whose source is `lost`.  KERNEL is the kernel's file.  Its waits are bounded,
// so a lost copy ends in the kernel's own error handling.
#include "ops.h"

namespace moe {
__device__ unsigned long long lost;
__device__ __forceinline__ void bulk_g2s_or_lose(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  if (reinterpret_cast<unsigned long long>(src) != lost) bulk_g2s(dst, src, bytes, bar);
}
}  // namespace moe

#define bulk_g2s bulk_g2s_or_lose
#include KERNEL

extern "C" {

__attribute__((visibility("default"))) int lose(unsigned long long src) {
  return cudaMemcpyToSymbol(moe::lost, &src, sizeof src) == cudaSuccess ? 0 : 1;
}

#ifdef NORM
__attribute__((visibility("default"))) int block_norm(const moe_v41_norm_cfg* cfg, int m, const void* y, const void* h,
                                                      void* h_out, void* x_out) {
  moe::NormParams p{};
  p.c = *cfg; p.m = m; p.y = y; p.h = h; p.h_out = h_out; p.x_out = x_out;
  p.ldy = p.ldh = p.ldh_out = p.ldx = cfg->dim;
  return moe::launch_block_norm(p, nullptr);
}
#endif

#ifdef LOGPROB
__attribute__((visibility("default"))) int token_logprobs(const moe_v41_logprob_cfg* cfg, const void* logits, int m,
                                                          const int* target, float* logprob, int* rank, float* lse,
                                                          float* entropy, float* top_logprob, int* top_id) {
  moe::LogprobParams p{};
  p.c = *cfg; p.m = m; p.logits = logits; p.ld = cfg->vocab; p.target = target; p.logprob = logprob; p.rank = rank;
  p.lse = lse; p.entropy = entropy; p.top_logprob = top_logprob; p.top_id = top_id;
  return moe::launch_token_logprobs(p, nullptr);
}
#endif

}  // extern "C"
