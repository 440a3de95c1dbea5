// A CUDA runtime that launches nothing, for the launchers' host code on a machine
// without a GPU: it is linked with the library's objects in the place of the
// real one.  Every thread may be on a device of its own; launches are counted,
// and those that a GPU would refuse.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <thread>
#include <vector>

#include "../include/moe_v41_ops.h"

namespace {
thread_local int device = 0;
std::atomic<int> registers{64}, launches{0}, bad{0}, grid{0};
std::atomic<const void*> kernel{nullptr};

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  std::memset(a, 0, sizeof *a);
  a->numRegs = registers;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  std::this_thread::yield();
  *n = 16;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *f = reinterpret_cast<void*>(&encode);
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* func, void**) {
  unsigned cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
  ++launches;
  if (c->gridDim.x == 0 || c->gridDim.x % cluster || c->blockDim.x == 0 || c->blockDim.x > 1024) ++bad;
  grid = (int)c->gridDim.x;
  kernel = func;
  return cudaSuccess;
}

// what the objects register when they are loaded
void** __cudaRegisterFatBinary(void*) {
  static void* handle = nullptr;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void*) {
  *k = nullptr;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorUnknown; }

void set_registers(int n) { registers = n; }

// since the last call: launches, and those that a GPU would refuse; and the last one's blocks
void counts(int* out) {
  out[0] = launches.exchange(0);
  out[1] = bad.exchange(0);
  out[2] = grid;
}
const void* last_kernel() { return kernel; }

// `threads` threads, on two devices by turns, call every operator `calls` times.
// Returns the number of calls that failed.
int call_from_threads(int threads, int calls) {
  std::atomic<int> failed{0}, ready{0};
  std::vector<std::thread> all;
  void* a = reinterpret_cast<void*>(uintptr_t(1) << 20);
  for (int t = 0; t < threads; ++t)
    all.emplace_back([&, t] {
      device = t % 2;
      const moe_v41_logprob_cfg lp{131072, t % 3, 20, 1.0f};
      const moe_v41_norm_cfg nm{4096, 1, 1, 0, 0, 1, 0, 0, 0, 1, 1e-6f, 1.0f, 1.0f};
      const moe_v41_q4_cfg q4{131072, 5120, t % 2 ? 64 : 128, 1, 2, 0, 512};
      for (++ready; ready < threads;) std::this_thread::yield();
      for (int i = 0; i < calls; ++i) {
        const int m = 1 << (i + t) % 7;  // clusters of 16 to 4 blocks
        failed += moe_v41_token_logprobs(&lp, a, m, 131072, nullptr, 0, static_cast<int*>(a), static_cast<float*>(a),
                                         static_cast<int*>(a), nullptr, nullptr, static_cast<float*>(a),
                                         static_cast<int*>(a), nullptr) != MOE_OK;
        failed += moe_v41_block_norm(&nm, 4096, a, 4096, nullptr, nullptr, nullptr, 0, a, 4096, a, 4096, nullptr, nullptr,
                                     a, 4096, nullptr) != MOE_OK;
        failed += moe_v41_q4_linear(&q4, a, 512, 5120, a, a, nullptr, a, 131072, a, size_t(1) << 40, nullptr) != MOE_OK;
        failed += moe_v41_q4_linear(&q4, a, 2, 5120, a, a, nullptr, a, 131072, a, size_t(1) << 40, nullptr) != MOE_OK;
      }
    });
  for (std::thread& th : all) th.join();
  return failed;
}

}  // extern "C"
