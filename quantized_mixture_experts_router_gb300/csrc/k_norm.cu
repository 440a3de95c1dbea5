// The norms before and after a block with its gate and residual scale:
//   h' = a h + c gate N_post(y),  x = N_pre(h')
// One block per token row, the row in registers between its single read and
// its single write: the statistics of y need one block reduction, those of h'
// a second (a layer norm takes its mean first and then the squares around it,
// so that a large common offset costs no digits).
#include "ops.h"

namespace moe {

namespace {

constexpr int MAXW = 32;  // warps of a block

__device__ __forceinline__ float block_sum(float v, float* red, int nw) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the previous sum has been read
  if (lane == 0) red[w] = v;
  __syncthreads();
  float s = lane < nw ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Eight elements of a thread, in their stored type: two 16-byte words for f32,
// one for the 16-bit types.
struct Raw8 {
  uint4 a, b;
};

__device__ __forceinline__ Raw8 load_raw8(const void* base, long long i, int t) {
  Raw8 r;
  const char* q = static_cast<const char*>(base) + i * (t == MOE_T_F32 ? 4 : 2);
  r.a = *reinterpret_cast<const uint4*>(q);
  r.b = make_uint4(0, 0, 0, 0);
  if (t == MOE_T_F32) r.b = *reinterpret_cast<const uint4*>(q + 16);
  return r;
}

__device__ __forceinline__ void raw_to_f32(const Raw8& r, int t, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (t == MOE_T_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else if (t == MOE_T_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = half_bits_to_float(w[i]);
      v[2 * i + 1] = half_bits_to_float(w[i] >> 16);
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int t) {
  if (t == MOE_T_BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 b = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void store_f32x8(void* base, long long i, int t, const float (&v)[8]) {
  char* q = static_cast<char*>(base) + i * (t == MOE_T_F32 ? 4 : 2);
  if (t == MOE_T_F32) {
    *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(q + 16) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(q) =
        make_uint4(pack2(v[0], v[1], t), pack2(v[2], v[3], t), pack2(v[4], v[5], t), pack2(v[6], v[7], t));
  }
}

// A thread's elements of a row: NV groups of eight.  VEC: group i is elements
// 8 (i T + tid) .. + 7 (16-byte accesses; dim a multiple of 8).  Otherwise
// element e of group i is (8 i + e) T + tid (any dim and alignment).
template <int NV, bool VEC>
struct Row {
  static __device__ __forceinline__ int at(int i, int e) {
    return VEC ? 8 * (i * (int)blockDim.x + (int)threadIdx.x) + e : (8 * i + e) * (int)blockDim.x + (int)threadIdx.x;
  }
  // v = the row's elements, `other` past its end
  static __device__ __forceinline__ void load(const void* p, long long off, int t, int d, float other,
                                              float (&v)[NV][8]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (VEC) {
        if (at(i, 0) < d) {
          raw_to_f32(load_raw8(p, off + at(i, 0), t), t, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = other;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = at(i, e) < d ? load_elem(p, off + at(i, e), t) : other;
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, long long off, int t, int d, const float (&v)[NV][8]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (VEC) {
        if (at(i, 0) < d) store_f32x8(p, off + at(i, 0), t, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at(i, e) < d) store_elem(p, off + at(i, e), t, v[i][e]);
      }
    }
  }
};

// v <- N(v); elements past the row's end stay out of the statistics.
template <int NV, bool VEC>
__device__ __forceinline__ void normalise(float (&v)[NV][8], int kind, const void* w, const void* b, int wt, int d,
                                          float eps, float* red, int nw) {
  using R = Row<NV, VEC>;
  if (kind == MOE_NORM_NONE) return;
  const float inv = 1.0f / (float)d;
  float mean = 0.f;
  if (kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += R::at(i, e) < d ? v[i][e] : 0.f;
    mean = block_sum(s, red, nw) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = R::at(i, e) < d ? v[i][e] - mean : 0.f;
      v[i][e] = c;
      q = fmaf(c, c, q);
    }
  const float r = 1.0f / sqrtf(block_sum(q, red, nw) * inv + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= r;
  if (w) {
    float u[NV][8];
    R::load(w, 0, wt, d, 0.f, u);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= u[i][e];
  }
  if (b) {
    float u[NV][8];
    R::load(b, 0, wt, d, 0.f, u);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += u[i][e];
  }
}

template <int NV, bool VEC>
__global__ void __launch_bounds__(1024) k_block_norm(const NormParams p) {
  using R = Row<NV, VEC>;
  __shared__ float red[MAXW];
  const int nw = (int)blockDim.x >> 5;
  const long long t = blockIdx.x;
  const int d = p.c.dim;
  float v[NV][8], h[NV][8];
  R::load(p.h, t * p.ldh, p.c.h_type, d, 0.f, h);
  if (p.y) {
    R::load(p.y, t * p.ldy, p.c.y_type, d, 0.f, v);
    normalise<NV, VEC>(v, p.c.post_kind, p.post_w, p.post_b, p.c.w_type, d, p.c.eps, red, nw);
    if (p.c.gate_kind == MOE_GATE_ROW) {
      float g[NV][8];
      R::load(p.gate, (t / p.c.gate_group) * p.ldg, p.c.gate_type, d, 0.f, g);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= g[i][e];
    } else if (p.c.gate_kind == MOE_GATE_TOKEN) {
      const float g = load_elem(p.gate, t / p.c.gate_group, p.c.gate_type);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= g;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = fmaf(p.c.residual_scale, h[i][e], p.c.block_scale * v[i][e]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = p.c.residual_scale * h[i][e];
  }
  if (p.h_out) R::store(p.h_out, t * p.ldh_out, p.c.h_type, d, v);
  if (p.x_out) {
    normalise<NV, VEC>(v, p.c.pre_kind, p.pre_w, p.pre_b, p.c.w_type, d, p.c.eps, red, nw);
    R::store(p.x_out, t * p.ldx, p.c.x_type, d, v);
  }
}

// Whether rows of this tensor can be read 16 bytes at a time.
bool vec_ok(const void* p, long long ld, int t) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * type_bytes(t)) % 16 == 0);
}

}  // namespace

int launch_block_norm(const NormParams& p, cudaStream_t s) {
  const moe_v41_norm_cfg& c = p.c;
  const bool vec = c.dim % 8 == 0 && vec_ok(p.y, p.ldy, c.y_type) && vec_ok(p.h, p.ldh, c.h_type) &&
                   vec_ok(p.h_out, p.ldh_out, c.h_type) && vec_ok(p.x_out, p.ldx, c.x_type) &&
                   vec_ok(c.gate_kind == MOE_GATE_ROW ? p.gate : nullptr, p.ldg, c.gate_type) &&
                   vec_ok(p.post_w, 0, c.w_type) && vec_ok(p.post_b, 0, c.w_type) && vec_ok(p.pre_w, 0, c.w_type) &&
                   vec_ok(p.pre_b, 0, c.w_type);
  const int per = (c.dim + 7) / 8;                 // groups of eight
  const int nv = per <= 1024 ? 1 : 2;              // dim <= 16384
  const int threads = ((per + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1) {
    if (vec) k_block_norm<1, true><<<p.m, threads, 0, s>>>(p);
    else k_block_norm<1, false><<<p.m, threads, 0, s>>>(p);
  } else {
    if (vec) k_block_norm<2, true><<<p.m, threads, 0, s>>>(p);
    else k_block_norm<2, false><<<p.m, threads, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
