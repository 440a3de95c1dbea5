// A kernel of the operators, built with copies that can get lost: the bulk copy
// whose source is `lost`, or (LINEAR) part of each box that a block's first warp
// expects, the block being `lost` - 1.  KERNEL is the kernel's file.  Its waits
// are bounded, so a lost copy ends in the kernel's own error handling.
#include "ops.h"

namespace moe {
__device__ unsigned long long lost;
__device__ __forceinline__ void bulk_g2s_or_lose(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  if (reinterpret_cast<unsigned long long>(src) != lost) bulk_g2s(dst, src, bytes, bar);
}
__device__ __forceinline__ void expect_more(uint64_t* bar, uint32_t bytes) {
  mbar_arrive_expect_tx(bar, threadIdx.x == 0 && blockIdx.x + 1 == lost ? bytes + 16 : bytes);
}
}  // namespace moe

#ifdef LINEAR
#define mbar_arrive_expect_tx expect_more
namespace moe {
int launch_q4_gemm(const Q4Params&, unsigned*, int, bool*, cudaStream_t) { return MOE_ERR_CUDA; }  // not under test
}  // namespace moe
#else
#define bulk_g2s bulk_g2s_or_lose
#endif
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

#ifdef LINEAR
__attribute__((visibility("default"))) int q4_linear(const moe_v41_q4_cfg* cfg, const void* x, int m, const void* w,
                                                     const void* scales, void* out, void* ws) {
  moe::Q4Params p{};
  p.m = m; p.n = cfg->n; p.k = cfg->k; p.group = cfg->group; p.ng = (cfg->k + cfg->group - 1) / cfg->group;
  p.x_type = cfg->x_type; p.scale_type = cfg->scale_type; p.out_type = cfg->out_type;
  p.x = static_cast<const uint16_t*>(x); p.ldx = cfg->k; p.w = static_cast<const uint8_t*>(w);
  p.scales = static_cast<const uint16_t*>(scales); p.out = out; p.ldo = cfg->n;
  return moe::launch_q4_linear(p, ws, nullptr);
}
#endif

}  // extern "C"
