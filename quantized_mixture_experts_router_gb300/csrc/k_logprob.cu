// Log probabilities of given tokens, entropy and the top alternatives of each
// row of logits.  With z = logit / T over the allowed entries, M = max z,
// S = sum exp(z - M), U = sum exp(z - M) (z - M):
//   lse = M + log S,  logprob = z_t - lse,  entropy = log S - U / S
// (the differences are taken around M, so that large common offsets cost no
// digits).  One block per row: one pass for the largest entry, one for the
// sums, one per alternative.
#include "ops.h"

namespace moe {

namespace {

constexpr int LP_THREADS = 512;
constexpr int LP_WARPS = LP_THREADS / 32;

// 64-bit order key of an entry: larger value first, NaN below every number,
// equal values (the two zeros among them) by ascending id.  0 is no entry.
__device__ __forceinline__ unsigned long long entry_key(float x, uint32_t id) {
  uint32_t o = 0;
  if (x == x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0
    o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  }
  return ((unsigned long long)o << 32) | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const uint32_t o = (uint32_t)(key >> 32);
  if (o == 0) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_id(unsigned long long key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, T* red, F f) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < LP_WARPS; ++i) v = f(v, red[i]);
  return v;
}

__global__ void __launch_bounds__(LP_THREADS) k_token_logprobs(const LogprobParams p) {
  __shared__ unsigned long long red_k[LP_WARPS];
  __shared__ float red_f[LP_WARPS];
  __shared__ int red_i[LP_WARPS];
  const long long row = blockIdx.x;
  const int V = p.c.vocab;
  const uint32_t* bits = p.allowed ? p.allowed + row * p.ld_allowed : nullptr;
  const float inf = __uint_as_float(0x7F800000u);
  const float rt = 1.0f / p.c.temperature;
  auto ok = [&](int j) { return !bits || ((bits[j >> 5] >> (j & 31)) & 1u); };
  auto val = [&](int j) { return load_elem(p.logits, row * p.ld + j, p.c.logit_type); };
  const auto kmax = [](unsigned long long a, unsigned long long b) { return a > b ? a : b; };
  const auto add = [](float a, float b) { return a + b; };

  unsigned long long best = 0;
  for (int j = threadIdx.x; j < V; j += LP_THREADS)
    if (ok(j)) best = kmax(best, entry_key(val(j), (uint32_t)j));
  best = block_reduce(best, red_k, kmax);
  float top = best ? key_value(best) : -inf;
  if (top == -inf) top = 0.f;  // no term is above zero: the shift is free, and S = 0 says so (NaN if one is NaN)

  const int t = p.target ? p.target[row] : -1;
  const bool scored = t >= 0 && t < V;
  float xt = -inf;
  if (scored && ok(t)) xt = val(t);
  float S = 0.f, U = 0.f;
  int above = 0;
  for (int j = threadIdx.x; j < V; j += LP_THREADS) {
    if (!ok(j)) continue;
    const float x = val(j);
    above += xt == xt ? x > xt : x == x;
    const float d = (x - top) * rt;
    const float e = expf(d);
    S += e;
    if (d != -inf) U += e * d;
  }
  S = block_reduce(S, red_f, add);
  U = block_reduce(U, red_f, add);
  above = block_reduce(above, red_i, [](int a, int b) { return a + b; });
  const bool empty = S == 0.f;
  const float ls = logf(S);
  const float lse = empty ? -inf : top * rt + ls;
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[row] = lse;
    if (p.entropy) p.entropy[row] = empty ? 0.f : ls - U / S;
    const float nan = __uint_as_float(0x7FC00000u);
    if (p.logprob) p.logprob[row] = scored ? (empty ? -inf : (xt - top) * rt - ls) : (t == -1 ? 0.f : nan);
    if (p.rank) p.rank[row] = scored ? above + 1 : (t == -1 ? 0 : -1);
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.c.top_k; ++i) {
    best = 0;
    for (int j = threadIdx.x; j < V; j += LP_THREADS)
      if (ok(j)) {
        const unsigned long long k = entry_key(val(j), (uint32_t)j);
        if (k < last) best = kmax(best, k);
      }
    best = block_reduce(best, red_k, kmax);
    if (threadIdx.x == 0) {
      p.top_logprob[row * p.c.top_k + i] = best == 0 || empty ? -inf : (key_value(best) - top) * rt - ls;
      p.top_id[row * p.c.top_k + i] = best ? key_id(best) : -1;
    }
    last = best;
  }
}

}  // namespace

int launch_token_logprobs(const LogprobParams& p, cudaStream_t s) {
  k_token_logprobs<<<p.m, LP_THREADS, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
