// Parameter blocks and launchers of the operators around the MoE layer
// (include/moe_v41_ops.h), shared by their kernels and the C entry points.
#pragma once

#include <cudaTypedefs.h>

#include "../../include/moe_v41_ops.h"
#include "common.cuh"
#include "per_device.h"

namespace moe {

struct Q4Params {
  int m, n, k, group, ng;    // ng = ceil(k / group)
  int x_type, scale_type, out_type;
  const uint16_t* x;
  long long ldx;
  const uint8_t* w;          // [n][k / 2]
  const uint16_t* scales;    // [n][ng]
  const uint8_t* zeros;      // [n][ng] or NULL
  void* out;
  long long ldo;
};

struct NormParams {
  moe_v41_norm_cfg c;
  int m;
  const void *y, *post_w, *post_b, *gate, *h, *pre_w, *pre_b;
  void *h_out, *x_out;
  long long ldy, ldg, ldh, ldh_out, ldx;
};

struct LogprobParams {
  moe_v41_logprob_cfg c;
  int m;
  const void* logits;
  long long ld;
  const uint32_t* allowed;
  long long ld_allowed;
  const int* target;
  float* logprob;
  int* rank;
  float* lse;
  float* entropy;
  float* top_logprob;
  int* top_id;
};

// A tensor map of a row-major matrix [rows][cols] with `pitch` bytes from row to
// row, read in boxes of box_cols x box_rows with the swizzle of box rows of
// `swizzle` bytes (64 or 128); what lies outside reads zero.
bool make_map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t cols, uint64_t rows,
                 uint64_t pitch, uint32_t box_cols, uint32_t box_rows, int swizzle);

// Many tokens (k_q4_gemm.cu); *taken: whether it was launched (see there).
int launch_q4_gemm(const Q4Params& p, unsigned* status, int sms, bool* taken, cudaStream_t s);
int launch_q4_linear(const Q4Params& p, void* ws, cudaStream_t s);
size_t q4_workspace_bytes(const moe_v41_q4_cfg& c);
int launch_block_norm(const NormParams& p, cudaStream_t s);
int launch_token_logprobs(const LogprobParams& p, cudaStream_t s);

__host__ __device__ inline int type_bytes(int t) { return t == MOE_T_F32 ? 4 : 2; }

// Wait on an mbarrier phase, at most timeout_ns after its first few tries:
// false (and the timeout bit in *status) when that ran out.  The timer is read
// only once a wait is long.
__device__ __forceinline__ bool mbar_wait_for(uint64_t* bar, uint32_t parity, uint64_t timeout_ns, unsigned* status) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
  return mbar_wait_bounded(bar, parity, globaltimer_ns() + timeout_ns, status);
}

// Programmatic dependent launch: the next kernel of the stream may be set up
// from here on; and the wait for everything the stream ran before.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch of a kernel that calls grid_wait() before it touches global memory:
// its blocks may be set up while the stream's previous kernel ends.
template <class P>
int launch_overlapped(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const P& p,
                      int cluster = 1) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// One element of a tensor of type T (MOE_T_*) as f32, and back with one
// rounding to nearest.
template <int T>
struct Elem;
template <>
struct Elem<MOE_T_F32> {
  using type = float;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<MOE_T_BF16> {
  using type = __nv_bfloat16;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<MOE_T_F16> {
  using type = __half;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

// The same with the type known at run time only.
__device__ __forceinline__ float load_elem(const void* p, long long i, int t) {
  if (t == MOE_T_F32) return static_cast<const float*>(p)[i];
  if (t == MOE_T_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, long long i, int t, float v) {
  if (t == MOE_T_F32) static_cast<float*>(p)[i] = v;
  else if (t == MOE_T_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

}  // namespace moe
