// An attention kernel (KERNEL, its file) built with copies that can get lost: the
// boxes of the page `lost` of the cache.  Its waits are bounded, so a lost copy ends
// in the kernel's own error handling.
#include "attn_work.cuh"

namespace moe {
__device__ int lost = -1;
__device__ __forceinline__ void tma_load_4d_or_lose(uint32_t dst, const void* map, int x, int slot, int head, int page,
                                                    uint64_t* bar) {
  if (page != lost) tma_load_4d(dst, map, x, slot, head, page, bar);
}
}  // namespace moe
#define tma_load_4d tma_load_4d_or_lose
#include KERNEL
#undef tma_load_4d

namespace moe {
#ifdef TILES
int launch_attn_rows(const AttnArgs&, int, cudaStream_t) { return MOE_ERR_CUDA; }  // not under test
#else
int launch_attn_tiles(const AttnArgs&, int, bool*, cudaStream_t) { return MOE_ERR_CUDA; }
#endif
}  // namespace moe
#include "attn_launch.cu"

extern "C" {

__attribute__((visibility("default"))) int lose(int page) {
  return cudaMemcpyToSymbol(moe::lost, &page, sizeof page) == cudaSuccess ? 0 : 1;
}

__attribute__((visibility("default"))) int attend(const moe_v41_attn_cfg* cfg, const moe_v41_seqs* seqs, int m,
                                                  const void* q, const void* k, const void* v, void* out, float* lse,
                                                  void* ws) {
  moe::AttnParams p{};
  p.c = *cfg; p.s = *seqs; p.m = m; p.q = q; p.k_cache = k; p.v_cache = v; p.out = out; p.lse = lse;
  p.ldq = p.ldo = (long long)cfg->heads * cfg->kv.head_dim;
  p.ld_lse = cfg->heads;
#ifdef TILES
  return moe::launch_paged_attention(p, 1 << 30, ws, nullptr);
#else
  return moe::launch_paged_attention(p, 0, ws, nullptr);
#endif
}

}  // extern "C"
