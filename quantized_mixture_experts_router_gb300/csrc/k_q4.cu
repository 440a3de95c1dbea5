// Products with 4-bit weights and group scales:
//   out[t, r] = sum_k x[t, k] s[r, k/G] (q[r, k] - z[r, k/G])
// One warp per weight row and eight tokens: a lane takes every 32nd word of
// eight codes, f32 sums, one butterfly at the end.
#include "ops.h"

namespace moe {

namespace {

constexpr int TOK = 8;

__device__ __forceinline__ float bits_to_f32(uint16_t v, int t) {
  return t == MOE_T_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

__global__ void __launch_bounds__(128) k_q4_rows(const Q4Params p) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t0 = blockIdx.y * TOK;
  if (row >= p.n) return;
  const uint32_t* wr = reinterpret_cast<const uint32_t*>(p.w + (size_t)row * (p.k / 2));
  float acc[TOK] = {};
  for (int wd = lane; wd < p.k / 8; wd += 32) {
    const uint32_t v = wr[wd];
    const size_t g = (size_t)row * p.ng + 8 * wd / p.group;
    const float s = bits_to_f32(p.scales[g], p.scale_type);
    const float z = p.zeros ? (float)p.zeros[g] : 8.0f;
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (t0 + t >= p.m) break;
      const uint16_t* xr = p.x + (size_t)(t0 + t) * p.ldx + 8 * wd;
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d = fmaf(bits_to_f32(xr[i], p.x_type), (float)((v >> (4 * i)) & 15u) - z, d);
      acc[t] = fmaf(s, d, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
#pragma unroll
    for (int o = 16; o; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if (lane == 0 && t0 + t < p.m) store_elem(p.out, (t0 + t) * p.ldo + row, p.out_type, acc[t]);
  }
}

}  // namespace

size_t q4_workspace_bytes(const moe_v41_q4_cfg&) { return align256(sizeof(Ctrl)); }

int launch_q4_linear(const Q4Params& p, void*, cudaStream_t s) {
  const dim3 grid((unsigned)((p.n + 3) / 4), (unsigned)((p.m + TOK - 1) / TOK));
  k_q4_rows<<<grid, 128, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
