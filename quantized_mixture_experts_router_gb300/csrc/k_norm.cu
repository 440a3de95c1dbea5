// The norms before and after a block with its gate and residual scale:
//   h' = a h + c gate N_post(y),  x = N_pre(h')
// A row stays in registers between its single read and its single write: the
// statistics of y need one block reduction, those of h' a second (a layer norm
// takes its mean first and then the squares around it, so that a large common
// offset costs no digits).  Bound by the bytes of y, h, h' and x for many rows,
// by the chain load - reduce - reduce - store for few.
//   k_norm_row   one block per row; weights and gate are loaded together with
//                the row, so that the chain holds one memory latency.
//   k_norm_rows  many rows: blocks walk through the rows, the next rows' y and
//                h arrive in shared memory by bulk copies meanwhile, and the
//                norms' weights stay in registers.
// Measured: 4096 rows of 5120, f32 y and h, bf16 x: 52.2 us, 5.6 TB/s (copies
// reach 6.8; the two barriers a row keep warps waiting).  One row: 3.2 us.
// Widths that are no multiple of 8 go element by element, a block a row: 8000 rows
// of 2305 (16-bit types) 96 us, 1.5 TB/s.
#include "ops.h"

namespace moe {

namespace {

constexpr int MAX_WARPS = 32;
constexpr int STAGES = 2;             // rows in shared memory (k_norm_rows)
constexpr int MAX_STREAMED = 8192;    // elements of a row there: 512 threads of 16
constexpr int MAX_STAGES_BYTES = STAGES * 2 * 4 * MAX_STREAMED;
constexpr uint64_t TIMEOUT_NS = 2000000000ull;  // of one wait for a copy

// Sum over the block; one barrier.  Two buffers alternate: a thread writes the
// one of the sum before last only after the barrier of the last, which every
// thread reaches after it has read the one before.
struct BlockSum {
  float* red;  // [2][MAX_WARPS], zero beyond the block's warps
  int nw;
  int turn;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    float* r = red + (turn & 1) * MAX_WARPS;
    ++turn;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < nw; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(r + i);
      s += (q.x + q.y) + (q.z + q.w);
    }
    return s;
  }
};

// Four elements of type T (16 bytes of f32, 8 of the 16-bit types).
template <int T>
__device__ __forceinline__ void load4(const void* base, long long i, float (&v)[4]) {
  if (T == MOE_T_F32) {
    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    if (T == MOE_T_BF16) {
      v[0] = bf16lo(r.x); v[1] = bf16hi(r.x); v[2] = bf16lo(r.y); v[3] = bf16hi(r.y);
    } else {
      v[0] = half_bits_to_float(r.x); v[1] = half_bits_to_float(r.x >> 16);
      v[2] = half_bits_to_float(r.y); v[3] = half_bits_to_float(r.y >> 16);
    }
  }
}
template <int T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (T == MOE_T_BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 b = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <int T>
__device__ __forceinline__ void store4(void* base, long long i, const float (&v)[4]) {
  if (T == MOE_T_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
}

// A thread's elements of a row: NG groups of four.  VEC: group i is elements
// 4 (i T + tid) .. + 3, so that a warp's accesses are contiguous (dim a multiple
// of 8, rows 16-byte aligned).  Otherwise element e of group i is
// (4 i + e) T + tid (any dim and alignment).
template <int NG, bool VEC>
struct Row {
  static __device__ __forceinline__ int at(int i, int e) {
    return VEC ? 4 * (i * (int)blockDim.x + (int)threadIdx.x) + e : (4 * i + e) * (int)blockDim.x + (int)threadIdx.x;
  }
  template <int T>
  static __device__ __forceinline__ void load_t(const void* p, long long off, int d, float (&v)[NG][4]) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (VEC) {
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
        if (at(i, 0) < d) load4<T>(p, off + at(i, 0), v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[i][e] = at(i, e) < d ? Elem<T>::get(static_cast<const typename Elem<T>::type*>(p)[off + at(i, e)]) : 0.f;
      }
    }
  }
  // the row's elements, 0 past its end; one branch on the type a row
  static __device__ __forceinline__ void load(const void* p, long long off, int t, int d, float (&v)[NG][4]) {
    if (t == MOE_T_F32) load_t<MOE_T_F32>(p, off, d, v);
    else if (t == MOE_T_BF16) load_t<MOE_T_BF16>(p, off, d, v);
    else load_t<MOE_T_F16>(p, off, d, v);
  }
  template <int T>
  static __device__ __forceinline__ void store_t(void* p, long long off, int d, const float (&v)[NG][4]) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (VEC) {
        if (at(i, 0) < d) store4<T>(p, off + at(i, 0), v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at(i, e) < d) store_elem(p, off + at(i, e), T, v[i][e]);
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, long long off, int t, int d, const float (&v)[NG][4]) {
    if (t == MOE_T_F32) store_t<MOE_T_F32>(p, off, d, v);
    else if (t == MOE_T_BF16) store_t<MOE_T_BF16>(p, off, d, v);
    else store_t<MOE_T_F16>(p, off, d, v);
  }
};

// v <- v - mean (layer norm); returns the factor 1 / sqrt(mean square + eps).
// Elements past the row's end are 0 before and after.
template <int NG, bool VEC>
__device__ __forceinline__ float centre(float (&v)[NG][4], int kind, int d, float eps, BlockSum& sum) {
  using R = Row<NG, VEC>;
  if (kind == MOE_NORM_NONE) return 1.0f;
  const float inv = 1.0f / (float)d;
  if (kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) s += (v[i][0] + v[i][1]) + (v[i][2] + v[i][3]);
    const float mean = sum(s) * inv;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (VEC) {
        const float m = R::at(i, 0) < d ? mean : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] -= m;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] -= R::at(i, e) < d ? mean : 0.f;
      }
    }
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) q = fmaf(v[i][e], v[i][e], q);
  return 1.0f / sqrtf(sum(q) * inv + eps);
}

// The norms' weights (1 where there are none).
template <int NG, bool VEC>
__device__ __forceinline__ void load_weights(const NormParams& p, float (&w1)[NG][4], float (&w2)[NG][4]) {
  using R = Row<NG, VEC>;
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) w1[i][e] = w2[i][e] = 1.0f;
  if (p.y && p.post_w && p.c.post_kind != MOE_NORM_NONE) R::load(p.post_w, 0, p.c.w_type, p.c.dim, w1);
  if (p.x_out && p.pre_w && p.c.pre_kind != MOE_NORM_NONE) R::load(p.pre_w, 0, p.c.w_type, p.c.dim, w2);
}

// v <- v * u for whole rows.
template <int NG>
__device__ __forceinline__ void scale_row(float (&v)[NG][4], const float (&u)[NG][4]) {
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] *= u[i][e];
}

// Everything after the row's loads: h' from v = y and h, its store, x.  tg: the
// token's gate (1 without one); row_gate(v) applies a gate row, if there is one.
template <int NG, bool VEC, class Gate>
__device__ __forceinline__ void finish_row(const NormParams& p, long long t, float (&v)[NG][4], const float (&h)[NG][4],
                                           const float (&w1)[NG][4], const float (&w2)[NG][4], float tg, Gate row_gate,
                                           BlockSum& sum) {
  using R = Row<NG, VEC>;
  const int d = p.c.dim;
  const float ra = p.c.residual_scale;
  if (p.y) {
    const float r = centre<NG, VEC>(v, p.c.post_kind, d, p.c.eps, sum);
    scale_row<NG>(v, w1);
    float f = r * (p.c.block_scale * tg);
    if (p.post_b && p.c.post_kind != MOE_NORM_NONE) {
      float b[NG][4];
      R::load(p.post_b, 0, p.c.w_type, d, b);
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = fmaf(v[i][e], r, b[i][e]);
      f = p.c.block_scale * tg;
    }
    row_gate(v);
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = fmaf(v[i][e], f, ra * h[i][e]);
  } else {
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = ra * h[i][e];
  }
  if (p.h_out) R::store(p.h_out, t * p.ldh_out, p.c.h_type, d, v);
  if (p.x_out) {
    const float r = centre<NG, VEC>(v, p.c.pre_kind, d, p.c.eps, sum);
    if (p.c.pre_kind != MOE_NORM_NONE) {
      scale_row<NG>(v, w2);
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] *= r;
      if (p.pre_b) {
        float b[NG][4];
        R::load(p.pre_b, 0, p.c.w_type, d, b);
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] += b[i][e];
      }
    }
    R::store(p.x_out, t * p.ldx, p.c.x_type, d, v);
  }
}

__device__ __forceinline__ void clear_sums(float* red) {
  for (int i = threadIdx.x; i < 2 * MAX_WARPS; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
}

template <int NG, bool VEC>
__global__ void __launch_bounds__(1024, 1) k_norm_row(const NormParams p) {
  using R = Row<NG, VEC>;
  __shared__ alignas(16) float red[2 * MAX_WARPS];
  grid_launch_dependents();
  clear_sums(red);
  BlockSum sum{red, (int)blockDim.x >> 5, 0};
  const long long t = blockIdx.x;
  const int d = p.c.dim;
  grid_wait();
  float v[NG][4], h[NG][4], w1[NG][4], w2[NG][4], g[NG][4];
  R::load(p.h, t * p.ldh, p.c.h_type, d, h);
  if (p.y) R::load(p.y, t * p.ldy, p.c.y_type, d, v);
  const bool rows = p.y && p.c.gate_kind == MOE_GATE_ROW;
  if (rows) R::load(p.gate, (t / p.c.gate_group) * p.ldg, p.c.gate_type, d, g);
  const float tg = p.y && p.c.gate_kind == MOE_GATE_TOKEN ? load_elem(p.gate, t / p.c.gate_group, p.c.gate_type) : 1.0f;
  load_weights<NG, VEC>(p, w1, w2);
  finish_row<NG, VEC>(p, t, v, h, w1, w2, tg,
                      [&](float (&u)[NG][4]) {
                        if (rows) scale_row<NG>(u, g);
                      },
                      sum);
}

// This row and the block's later ones become NaN.
template <int NG>
__device__ __noinline__ void store_nan(const NormParams& p, long long r, int step) {
  using R = Row<NG, true>;
  float v[NG][4];
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = __uint_as_float(0x7FC00000u);
  for (; r < p.m; r += step) {
    if (p.h_out) R::store(p.h_out, r * p.ldh_out, p.c.h_type, p.c.dim, v);
    if (p.x_out) R::store(p.x_out, r * p.ldx, p.c.x_type, p.c.dim, v);
  }
}

struct NormRowsArgs {
  NormParams p;
  uint32_t y_bytes, h_bytes;  // of a row; a stage holds y, then h
};

template <int NG, int MAX_THREADS, int BLOCKS>
__global__ void __launch_bounds__(MAX_THREADS, BLOCKS) k_norm_rows(const NormRowsArgs a) {
  using R = Row<NG, true>;
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ alignas(16) float red[2 * MAX_WARPS];
  __shared__ alignas(8) uint64_t full[STAGES];
  __shared__ unsigned timed_out;  // where a wait that runs out leaves its bit; each thread also learns it from the wait
  const NormParams& p = a.p;
  const int d = p.c.dim;
  const uint32_t stage_bytes = a.y_bytes + a.h_bytes;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
    timed_out = 0u;
  }
  clear_sums(red);
  BlockSum sum{red, (int)blockDim.x >> 5, 0};
  grid_wait();
  const int step = (int)gridDim.x;
  auto fetch = [&](long long r, int st) {  // one thread
    uint8_t* s = stages + (uint32_t)st * stage_bytes;
    mbar_arrive_expect_tx(full + st, stage_bytes);
    if (a.y_bytes) bulk_g2s(s, static_cast<const char*>(p.y) + r * p.ldy * type_bytes(p.c.y_type), a.y_bytes, full + st);
    bulk_g2s(s + a.y_bytes, static_cast<const char*>(p.h) + r * p.ldh * type_bytes(p.c.h_type), a.h_bytes, full + st);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < STAGES && blockIdx.x + (long long)i * step < p.m; ++i) fetch(blockIdx.x + (long long)i * step, i);
  float w1[NG][4], w2[NG][4];
  load_weights<NG, true>(p, w1, w2);
  int st = 0;
  uint32_t phase = 0;
  for (long long r = blockIdx.x; r < p.m; r += step) {
    const bool here = mbar_try_wait(full + st, phase) || mbar_wait_for(full + st, phase, TIMEOUT_NS, &timed_out);
    const uint8_t* s = stages + (uint32_t)st * stage_bytes;
    float v[NG][4], h[NG][4];
    if (p.y) R::load(s, 0, p.c.y_type, d, v);
    R::load(s + a.y_bytes, 0, p.c.h_type, d, h);
    const float tg = p.y && p.c.gate_kind == MOE_GATE_TOKEN ? load_elem(p.gate, r / p.c.gate_group, p.c.gate_type) : 1.0f;
    // the stage has been read; where it had not arrived for some thread, the block
    // gives up, once its copies in flight have landed (or two seconds later)
    if (__syncthreads_or(!here)) {
      store_nan<NG>(p, r, step);
      const uint64_t deadline = globaltimer_ns() + TIMEOUT_NS;
      if (threadIdx.x == 0)
        for (int j = 0; j < STAGES && r + (long long)j * step < p.m; ++j)
          mbar_wait_bounded(full + (st + j) % STAGES, phase ^ (st + j >= STAGES ? 1u : 0u), deadline, &timed_out);
      return;
    }
    if (threadIdx.x == 0 && r + (long long)STAGES * step < p.m) fetch(r + (long long)STAGES * step, st);
    finish_row<NG, true>(p, r, v, h, w1, w2, tg,
                         [&](float (&u)[NG][4]) {
                           if (p.c.gate_kind != MOE_GATE_ROW) return;
                           float g[NG][4];
                           R::load(p.gate, (r / p.c.gate_group) * p.ldg, p.c.gate_type, d, g);
                           scale_row<NG>(u, g);
                         },
                         sum);
    if (++st == STAGES) {
      st = 0;
      phase ^= 1u;
    }
  }
}

// Whether rows of this tensor can be read 16 bytes at a time.
bool vec_ok(const void* p, long long ld, int t) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * type_bytes(t)) % 16 == 0);
}

template <int MAX_THREADS, int BLOCKS>
int launch_rows_t(const NormRowsArgs& a, int threads, uint32_t smem, int sms, int dev, cudaStream_t s) {
  const auto kernel = k_norm_rows<4, MAX_THREADS, BLOCKS>;
  static PerDevice allocated;  // registers a thread
  const int regs = allocated.get(dev, [&] {
    cudaFuncAttributes fa{};
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_STAGES_BYTES) == cudaSuccess &&
                   cudaFuncGetAttributes(&fa, kernel) == cudaSuccess
               ? (fa.numRegs + 7) / 8 * 8
               : 0;
  });
  if (regs < 1) return MOE_ERR_CUDA;
  // blocks an SM holds
  int occ = (int)(228u * 1024u / (smem + 2048u));
  if (occ > 65536 / (threads * regs)) occ = 65536 / (threads * regs);
  if (occ > 2048 / threads) occ = 2048 / threads;
  if (occ > 16) occ = 16;
  if (occ < 1) occ = 1;
  const int grid = a.p.m < sms * occ ? a.p.m : sms * occ;
  return launch_overlapped(kernel, dim3((unsigned)grid), dim3((unsigned)threads), smem, s, a);
}

// k_norm_row: groups of four elements a thread takes, and a block's threads
int row_groups(int dim) { return dim <= 8192 ? 2 : 4; }
int row_threads(int dim) {
  const int per = 4 * row_groups(dim);
  return ((dim + per - 1) / per + 31) / 32 * 32;
}

int launch_rows(const NormParams& p, int sms, int dev, bool* taken, cudaStream_t s) {
  // From more rows on than blocks of k_norm_row (64 registers a thread: 1024
  // threads an SM) are resident at once.  f32 rows of 5120: 152 rows 4.0 us here,
  // 3.3 us a block each; 180 rows 5.3 and 5.6, 600 rows 8.4 and 11.1, 4096 rows 52
  // and 82.  f32 rows of 8192, whose stages leave an SM one block: 153 rows 6.4 and
  // 7.5, 4096 rows 74 and 111.  bf16 rows of 2304: 420 rows 4.4 and 3.4, 500 rows
  // 4.4 and 5.4.
  *taken = false;
  NormRowsArgs a{};
  a.p = p;
  a.y_bytes = p.y ? (uint32_t)(p.c.dim * type_bytes(p.c.y_type)) : 0u;
  a.h_bytes = (uint32_t)(p.c.dim * type_bytes(p.c.h_type));
  const uint32_t smem = STAGES * (a.y_bytes + a.h_bytes);
  const int threads = (p.c.dim + 16 * 32 - 1) / (16 * 32) * 32;  // 16 elements each
  if (p.c.dim > MAX_STREAMED || p.m <= 1024 / row_threads(p.c.dim) * sms) return MOE_OK;
  *taken = true;
  return threads <= 320 ? launch_rows_t<320, 2>(a, threads, smem, sms, dev, s)
                        : launch_rows_t<512, 1>(a, threads, smem, sms, dev, s);
}

}  // namespace

int launch_block_norm(const NormParams& p, cudaStream_t s) {
  const moe_v41_norm_cfg& c = p.c;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return MOE_ERR_CUDA;
  const bool vec = c.dim % 8 == 0 && vec_ok(p.y, p.ldy, c.y_type) && vec_ok(p.h, p.ldh, c.h_type) &&
                   vec_ok(p.h_out, p.ldh_out, c.h_type) && vec_ok(p.x_out, p.ldx, c.x_type) &&
                   vec_ok(c.gate_kind == MOE_GATE_ROW ? p.gate : nullptr, p.ldg, c.gate_type) &&
                   vec_ok(p.post_w, 0, c.w_type) && vec_ok(p.post_b, 0, c.w_type) && vec_ok(p.pre_w, 0, c.w_type) &&
                   vec_ok(p.pre_b, 0, c.w_type);
  if (vec) {
    bool taken = false;
    const int rc = launch_rows(p, sms, dev, &taken, s);
    if (rc || taken) return rc;
  }
  const dim3 grid((unsigned)p.m), block((unsigned)row_threads(c.dim));
  if (row_groups(c.dim) == 2) return vec ? launch_overlapped(k_norm_row<2, true>, grid, block, 0, s, p)
                          : launch_overlapped(k_norm_row<2, false>, grid, block, 0, s, p);
  return vec ? launch_overlapped(k_norm_row<4, true>, grid, block, 0, s, p)
             : launch_overlapped(k_norm_row<4, false>, grid, block, 0, s, p);
}

}  // namespace moe
