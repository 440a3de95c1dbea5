// The attention kernel for many rows, built with a walking warp that stops telling its
// block's items: at item `lost_item` > 0 of block `lost_block`, which it does not announce,
// or (-1) where it first waits for a slot.  Waits for an item end after half a second.
#include "attn_work.cuh"

namespace moe {
__device__ int lost_block = -1, lost_item = 0;
__device__ __forceinline__ uint32_t tell_or_not(uint32_t* told, uint32_t n, uint32_t next) {
  if ((int)blockIdx.x == lost_block && (int)n == lost_item && next == n + 1) return ~n;
  return atomicCAS(told, n, next);
}
__device__ __forceinline__ bool wait_a_little(uint64_t* bar, uint32_t parity, uint64_t ns, unsigned* status) {
  if ((int)blockIdx.x == lost_block && lost_item < 0 && threadIdx.x / 32 == 10) {
    atomicOr(status, (unsigned)MOE_STATUS_TIMEOUT);
    return false;
  }
  return mbar_wait_for(bar, parity, ns / 16, status);
}
}  // namespace moe
#define atomicCAS tell_or_not
#define mbar_wait_for wait_a_little
#include "lost_tiles.cu"

extern "C" __attribute__((visibility("default"))) int lose_item(int block, int item) {
  return cudaMemcpyToSymbol(moe::lost_block, &block, sizeof block) == cudaSuccess &&
                 cudaMemcpyToSymbol(moe::lost_item, &item, sizeof item) == cudaSuccess ? 0 : 1;
}
