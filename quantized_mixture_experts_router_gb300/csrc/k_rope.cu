// Rotary positions, and the append of keys and values to a paged cache with the
// rotation on the way:
//   a' = g (a cos t - b sin t),  b' = g (b cos t + a sin t),  t = pos f_i
//
// Bound by bytes for many tokens and by latency for few.  A block takes a few
// tokens; a thread of it computes a pair's sine and cosine once per token into
// shared memory, and all its heads use them.  The angle is reduced in 64 bits:
// pos f / 2 pi minus its nearest whole number (exact to 2^-52 of the turns), then
// sincospi in f32.  Values move eight at a time (16-bit neighbours 16) wherever the
// head's parts begin at multiples of it (both halves' vectors in one thread), else one
// pair at a time.  Among its kind in a graph, inputs partly in L2, one row of 32 heads of 128
// takes 1.8 us, a launch, and 4096 rows of 16 heads of 192, f32 (101 MB), 17 us.  As a call
// on data that is not there it takes 22 us, 68% of a copy's rate: a thread has one unit on
// its way, and the first waits for look-ups and angles that it does not need.
#include "attn_work.cuh"

namespace moe {

namespace {

constexpr int NTHR = 256;
// SMs of the GPU that the library is built for.  It only spreads the work: asking the device would cost a call whose
// time is the host's, and another count is served as rightly.
constexpr int SMS = 152;

struct RopeArgs {
  RopeParams p;
  int tokens;          // a block's
  int pairs;           // rot_dim / 2
  int units_rot;       // rotated units of a head: vectors (interleaved) or pairs of vectors (half)
  int units;           // all units of a head
  int heads;           // of a token: queries, keys, values
  int page_shift;
  AttnGroup per_token, per_head;  // units of a token, of a head
};

template <class T>
__device__ __forceinline__ float get(T v);
template <>
__device__ __forceinline__ float get(float v) { return v; }
template <>
__device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float get(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T put(float v);
template <>
__device__ __forceinline__ float put(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }

// V values in one go: V = 8 on 16-byte boundaries, or one.
template <int V, class T>
__device__ __forceinline__ void load_v(const T* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = get<T>(*p);
  } else {
    constexpr int W = V * (int)sizeof(T) / 16;
    uint4 w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = get<T>(e[i]);
  }
}
template <int V, class T>
__device__ __forceinline__ void store_v(T* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = put<T>(f[0]);
  } else {
    constexpr int W = V * (int)sizeof(T) / 16;
    alignas(16) T e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = put<T>(f[i]);
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
  }
}

// (cos, sin) of two neighbouring pairs at once.
__device__ __forceinline__ float4 two(const float2* cs) { return *reinterpret_cast<const float4*>(cs); }

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float r = x * c - y * s;
  y = y * c + x * s;
  x = r;
}

// One unit of a head.  cs: the token's (cos, sin) per pair, or NULL for a head
// that is copied (values).
template <class IN, class OUT, int V>
__device__ __forceinline__ void do_unit(const RopeArgs& a, const IN* x, OUT* y, int u, const float2* cs) {
  const int first = a.p.c.rot_first;
  if (u < a.units_rot) {
    if (a.p.c.layout == MOE_ROPE_HALF) {
      const int i = u * V, lo = first + i, hi = lo + a.pairs;
      float s[V], t[V];
      load_v<V>(x + lo, s);
      load_v<V>(x + hi, t);
      if (cs) {
        if constexpr (V == 1) {
          turn(s[0], t[0], cs[i].x, cs[i].y);
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const float4 c = two(cs + i + j);
            turn(s[j], t[j], c.x, c.y);
            turn(s[j + 1], t[j + 1], c.z, c.w);
          }
        }
      }
      store_v<V>(y + lo, s);
      store_v<V>(y + hi, t);
    } else {
      constexpr int P = V == 1 ? 1 : V / 2;  // pairs of the unit
      const int at = first + 2 * P * u;
      float s[2 * P];
      if constexpr (V == 1) {
        s[0] = get<IN>(x[at]);
        s[1] = get<IN>(x[at + 1]);
      } else {
        load_v<2 * P>(x + at, s);
      }
      if (cs) {
        if constexpr (V == 1) {
          turn(s[0], s[1], cs[u].x, cs[u].y);
        } else {
#pragma unroll
          for (int j = 0; j < P; j += 2) {
            const float4 c = two(cs + P * u + j);
            turn(s[2 * j], s[2 * j + 1], c.x, c.y);
            turn(s[2 * j + 2], s[2 * j + 3], c.z, c.w);
          }
        }
      }
      if constexpr (V == 1) {
        y[at] = put<OUT>(s[0]);
        y[at + 1] = put<OUT>(s[1]);
      } else {
        store_v<2 * P>(y + at, s);
      }
    }
    return;
  }
  int at = (u - a.units_rot) * V;  // the values beside the rotated ones
  if (at >= first) at += 2 * a.pairs;
  float s[V];
  load_v<V>(x + at, s);
  store_v<V>(y + at, s);
}

struct Token {
  int live;                    // rows of nobody are left alone
  long long slot;              // where its key and value go in the cache, -1: nowhere
  int pos;
};

// The sequence of row t: the last b with cu[b] <= t, by a whole warp, 32
// boundaries a step; batch when t lies behind the last, -1 before the first.
__device__ __forceinline__ int find_sequence(const int* cu, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch + 1;   // among the boundaries lo .. lo + n - 1
  while (true) {
    const int step = (n + 31) / 32, i = lane * step;
    const bool le = i < n && __ldg(cu + lo + i) <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, le));
    if (hits == 0) return lo - 1;
    if (step == 1) return lo + hits - 1;
    const int from = (hits - 1) * step;
    lo += from;
    n = min(step, n - from);
  }
}

template <class IN, class OUT, int V, bool APPEND>
__global__ void __launch_bounds__(NTHR) k_rope(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float2 cs[];  // [tokens][pairs]
  __shared__ Token tok[8];
  const RopeParams& p = a.p;
  const int t0 = (int)blockIdx.x * a.tokens, nt = min(a.tokens, p.m - t0);
  grid_launch_dependents();
  grid_wait();
  if (APPEND) {
    const int w = threadIdx.x >> 5;
    if (w < nt) {
      const int t = t0 + w, b = find_sequence(p.s.cu_new, p.s.batch, t);
      Token k{0, -1, 0};
      if (b >= 0 && b < p.s.batch) {
        const int c0 = p.s.cu_new[b], n = p.s.cu_new[b + 1] - c0;
        k.pos = max(p.s.kv_len[b], 0) - n + (t - c0);
        k.live = t - c0 < n;
        if (k.live && k.pos >= 0) {
          const int page = k.pos >> a.page_shift;
          int id = -1;
          if (page < p.s.max_pages) id = p.s.table[b * p.s.ld_table + page];
          if (id >= 0 && id < p.kv.n_pages)
            k.slot = (long long)id * p.kv.page_pitch + (k.pos & (p.kv.page_size - 1)) * p.kv.token_pitch;
          else if (p.status && (threadIdx.x & 31) == 0 && blockIdx.y == 0)
            atomicOr(p.status, (unsigned)MOE_STATUS_BAD_PAGE);
        }
      }
      if ((threadIdx.x & 31) == 0) tok[w] = k;
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < nt * a.pairs; i += NTHR) {
    const int w = i / a.pairs, pr = i - w * a.pairs;
    const int pos = !APPEND || p.pos ? p.pos[t0 + w] : tok[w].pos;
    const double turns = (double)pos * p.freqs[pr] * 0.15915494309189535;  // 1 / 2 pi
    float sn, cn;
    sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
    cs[i] = make_float2(cn * p.c.magnitude, (p.c.inverse ? -sn : sn) * p.c.magnitude);
  }
  __syncthreads();
  for (int i = (int)blockIdx.y * NTHR + threadIdx.x; i < nt * a.per_token.n; i += (int)gridDim.y * NTHR) {
    const int w = a.per_token.token(i), r = i - w * a.per_token.n;
    const int h = a.per_head.token(r), u = r - h * a.per_head.n;
    const long long t = t0 + w;
    if (APPEND && !tok[w].live) continue;
    const float2* c = cs + w * a.pairs;
    if (!APPEND || h < p.heads_q) {
      do_unit<IN, OUT, V>(a, static_cast<const IN*>(p.q) + t * p.ldq + h * p.ldq_head,
                          static_cast<OUT*>(p.q_out) + t * p.ldo + h * p.ldo_head, u, c);
      continue;
    }
    if (tok[w].slot < 0) continue;
    const bool key = h < p.heads_q + p.heads_kv;
    const int hk = h - p.heads_q - (key ? 0 : p.heads_kv);
    const IN* x = static_cast<const IN*>(key ? p.k : p.v) + t * (key ? p.ldk : p.ldv) + hk * p.c.head_dim;
    OUT* y = static_cast<OUT*>(key ? p.k_cache : p.v_cache) + tok[w].slot + hk * p.kv.head_pitch;
    do_unit<IN, OUT, V>(a, x, y, u, key ? c : nullptr);
  }
}

template <class IN, class OUT, int V, bool APPEND>
int launch(const RopeArgs& a, dim3 grid, cudaStream_t s) {
  return launch_overlapped(k_rope<IN, OUT, V, APPEND>, grid, dim3(NTHR), (size_t)a.tokens * a.pairs * sizeof(float2), s, a);
}

template <class IN, class OUT, bool APPEND>
int launch_v(const RopeArgs& a, int v, dim3 grid, cudaStream_t s) {
  if constexpr (sizeof(IN) == 2)
    if (v == 16) return launch<IN, OUT, 16, APPEND>(a, grid, s);
  return v == 8 ? launch<IN, OUT, 8, APPEND>(a, grid, s) : launch<IN, OUT, 1, APPEND>(a, grid, s);
}

}  // namespace

int launch_rope(const RopeParams& p, cudaStream_t s) {
  const bool append = p.kv.page_size > 0;
  RopeArgs a{};
  a.p = p;
  const moe_v41_rope_cfg& c = p.c;
  const bool half = c.layout == MOE_ROPE_HALF;
  a.pairs = c.rot_dim / 2;
  // eight values at a time: every part of a head, and every row, begins on a multiple of eight and of 16 bytes
  auto fits = [](const void* q, int64_t pitch) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && pitch % 8 == 0; };
  bool vec = c.head_dim % 8 == 0 && c.rot_first % 8 == 0 && (half ? a.pairs : c.rot_dim) % 8 == 0 &&
             (!p.heads_q || (fits(p.q, p.ldq) && fits(p.q_out, p.ldo)));
  if (p.heads_q > 1) vec = vec && p.ldq_head % 8 == 0 && p.ldo_head % 8 == 0;
  if (append) vec = vec && fits(p.k, p.ldk) && fits(p.v, p.ldv);
  // 16-bit pairs that are neighbours: 16 values, so that as many bytes are on their way
  // as with halves (8192 x 32 heads of 128, bf16: 32 us, 35 with eight)
  const bool wide = vec && !half && c.x_type != MOE_T_F32 && c.head_dim % 16 == 0 && c.rot_first % 16 == 0 && c.rot_dim % 16 == 0;
  const int v = wide ? 16 : vec ? 8 : 1;
  a.units_rot = half || !vec ? a.pairs / (half ? v : 1) : c.rot_dim / v;
  // in place, what is not rotated stays where it is
  a.units = a.units_rot + (!append && p.q == p.q_out && c.rot_dim ? 0 : (c.head_dim - c.rot_dim) / v);
  if (!append && p.q == p.q_out && !c.rot_dim) return MOE_OK;
  a.heads = p.heads_q + 2 * p.heads_kv;
  if (append) a.page_shift = __builtin_ctz((unsigned)p.kv.page_size);
  // About four units a thread; but a token's heads are shared by several blocks while there are few tokens.
  const long long units = (long long)a.heads * a.units;
  a.tokens = (int)(units >= 512 ? 1 : 1024 / units > 8 ? 8 : 1024 / units);
  while (a.tokens > 1 && (p.m + a.tokens - 1) / a.tokens < SMS * 4) a.tokens /= 2;
  a.per_token = AttnGroup::of((int)units);
  a.per_head = AttnGroup::of(a.units);
  const int blocks = (p.m + a.tokens - 1) / a.tokens;
  long long split = (units * a.tokens + NTHR - 1) / NTHR;
  if (split * blocks > SMS * 8) split = blocks >= SMS * 8 ? 1 : (SMS * 8 + blocks - 1) / blocks;
  const dim3 grid((unsigned)blocks, (unsigned)(split < 65535 ? split : 65535));
  if (!append) {
    if (c.x_type == MOE_T_F32) return launch_v<float, float, false>(a, v, grid, s);
    if (c.x_type == MOE_T_BF16) return launch_v<__nv_bfloat16, __nv_bfloat16, false>(a, v, grid, s);
    return launch_v<__half, __half, false>(a, v, grid, s);
  }
  if (p.out_type == MOE_T_BF16) {
    if (c.x_type == MOE_T_F32) return launch_v<float, __nv_bfloat16, true>(a, v, grid, s);
    if (c.x_type == MOE_T_BF16) return launch_v<__nv_bfloat16, __nv_bfloat16, true>(a, v, grid, s);
    return launch_v<__half, __nv_bfloat16, true>(a, v, grid, s);
  }
  if (c.x_type == MOE_T_F32) return launch_v<float, __half, true>(a, v, grid, s);
  if (c.x_type == MOE_T_BF16) return launch_v<__nv_bfloat16, __half, true>(a, v, grid, s);
  return launch_v<__half, __half, true>(a, v, grid, s);
}

}  // namespace moe
