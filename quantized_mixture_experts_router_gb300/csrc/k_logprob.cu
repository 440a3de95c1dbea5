// Log probabilities of given tokens, entropy and the top alternatives of each
// row of logits.  With z = logit / T over the allowed entries, M = max z,
// S = sum exp(z - M), U = sum exp(z - M) (z - M):
//   lse = M + log S,  logprob = (z_t - M) - log S,  entropy = log S - U / S
// (differences are taken around M before anything is rounded away, so that
// large common offsets cost no digits).
//
// Bound by one read of the logits: everything comes from a single pass.
//  - A row belongs to a cluster of 1..16 blocks (more when there are few
//    rows), a contiguous slice each; their results meet in distributed shared
//    memory.
//  - Bulk copies bring batches of 32 KB into two buffers of shared memory while
//    the threads work on the other one, so that the loads in flight cost no
//    registers.  (Units of eight entries that the row begins or ends inside are
//    read entry by entry.)
//  - A thread keeps M, S, U of its own; S and U are packed pairs of f32 (two
//    sums an instruction).  The entry-wise work beside the sums hides behind
//    one comparison of the unit's maximum with min(M, the target's logit, the
//    selection threshold).
//  - Top entries: each key (value, then lower id) is a 64-bit number.  The
//    k-th largest of the threads' maxima of the first batch bounds the k-th
//    largest key from below; the few entries that reach the bound go to a
//    buffer in shared memory, of which warps sort the best 32.  A batch that
//    overflows the buffer (rows in ascending order) raises the bound to the
//    k-th largest of what fitted and is taken again.
// Sums follow the fixed order of threads, warps and blocks; the buffer's order
// varies, its sorted content does not.
#include "ops.h"
#include "select.cuh"

namespace moe {

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int CAP = 2048;             // keys of the candidate buffer
constexpr int MAX_CLUSTER = 16;
constexpr float LOWEST = -3.4028234663852886e38f;
constexpr float FAR = -1.0e30f;       // a difference whose exponential is zero, but whose product with it is not NaN

__device__ __forceinline__ float pos_inf() { return __uint_as_float(0x7F800000u); }

__device__ __forceinline__ float key_value(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  if (o == 0) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_id(u64 key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// max that keeps a NaN of a
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// Two f32 in one register pair.
__device__ __forceinline__ u64 pack(float a, float b) {
  u64 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack(u64 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The running statistics of a set of entries.
struct Stat {
  float M, S, U;
  int above;
};

// Two sets' statistics; k: log2(e) / T.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float k) {
  Stat r;
  r.M = fmaxf(a.M, b.M);
  const float da = max_nan(a.M - r.M, FAR), db = max_nan(b.M - r.M, FAR);
  const float ea = ex2(da * k), eb = ex2(db * k);
  r.S = a.S * ea + b.S * eb;
  r.U = (a.U + a.S * da) * ea + (b.U + b.S * db) * eb;
  r.above = a.above + b.above;
  return r;
}

__device__ __forceinline__ u64 shfl_xor_u64(u64 v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// The warp's 32 keys in descending order (lane 0 the largest).
__device__ __forceinline__ u64 warp_sort(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size >> 1; o; o >>= 1) {
      const u64 w = shfl_xor_u64(v, o);
      const bool up = (lane & size) == 0;        // this run descends
      const bool low = (lane & o) == 0;
      v = (up == low) == (v > w) ? v : w;
    }
  }
  return v;
}
// The 32 largest of two descending lists, descending.
__device__ __forceinline__ u64 warp_merge(u64 a, u64 b) {
  const int lane = threadIdx.x & 31;
  b = __shfl_sync(0xffffffffu, b, 31 - lane);
  u64 v = a > b ? a : b;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const u64 w = shfl_xor_u64(v, o);
    v = ((lane & o) == 0) == (v > w) ? v : w;
  }
  return v;
}

constexpr uint32_t BATCH_BYTES = 32768;
template <int T>
constexpr int BATCH_UNITS = BATCH_BYTES / (8 * (T == MOE_T_F32 ? 4 : 2));

struct Shared {
  u64 full[2];               // a batch has landed
  unsigned failed;           // a wait ran out: the row's results are NaN
  int pushed[3];             // keys pushed in a batch, by batch number mod 3
  u64 buf[CAP];
  u64 lists[WARPS][32];
  u64 best[32];              // the block's list, read by the cluster's first block
  Stat stat[WARPS];
  Stat total;                // the block's, read by the cluster's first block
};

// The 32 largest of n keys (n >= 0) by the whole block, in lists[0],
// descending (0: none).  Ends with a barrier.
__device__ __forceinline__ void block_top(Shared& sh, const u64* keys, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 cur = 0;
  for (int i = warp * 32; i < n; i += THREADS) cur = warp_merge(cur, warp_sort(i + lane < n ? keys[i + lane] : 0));
  sh.lists[warp][lane] = cur;
  for (int s = WARPS / 2; s; s >>= 1) {
    __syncthreads();
    if (warp < s) {
      cur = warp_merge(cur, sh.lists[warp + s][lane]);
      sh.lists[warp][lane] = cur;
    }
  }
  __syncthreads();
}

// Eight entries of the row.
template <int T>
struct Unit {
  static constexpr int NV = T == MOE_T_F32 ? 2 : 1;
  uint4 v[NV];
  uint32_t ok;  // bit e: entry e is in the row and allowed
  __device__ __forceinline__ void to_f32(float (&x)[8]) const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[NV - 1].x, v[NV - 1].y, v[NV - 1].z, v[NV - 1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (T == MOE_T_F32) x[e] = __uint_as_float(w[e]);
      else if (T == MOE_T_BF16) x[e] = (e & 1) ? bf16hi(w[e / 2]) : bf16lo(w[e / 2]);
      else x[e] = half_bits_to_float((e & 1) ? w[e / 2] >> 16 : w[e / 2]);
    }
  }
};

// Where a row's units lie: unit u holds the entries 8 u - off .. 8 u - off + 7,
// so that its first byte is 16-byte aligned.
template <int T, bool MASK>
struct RowView {
  const typename Elem<T>::type* row;
  const uint32_t* bits;
  int off, V;
  __device__ __forceinline__ RowView(const LogprobParams& p, long long r) {
    row = static_cast<const typename Elem<T>::type*>(p.logits) + r * p.ld;
    bits = MASK ? p.allowed + r * p.ld_allowed : nullptr;
    constexpr int SZ = (int)sizeof(typename Elem<T>::type);
    off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / SZ;
    V = p.c.vocab;
  }
  __device__ __forceinline__ int units() const { return (off + V + 7) / 8; }
  __device__ __forceinline__ bool allowed(int j) const { return !MASK || ((__ldg(bits + (j >> 5)) >> (j & 31)) & 1u); }
  // the units that lie wholly inside the row
  __device__ __forceinline__ int inner_begin() const { return off ? 1 : 0; }
  __device__ __forceinline__ int inner_end() const { return (off + V) / 8; }
  // unit u; `at`: its place in shared memory, for inner units
  __device__ __forceinline__ Unit<T> load(int u, const uint8_t* at) const {
    Unit<T> r;
    const int j0 = 8 * u - off;
    if (j0 >= 0 && j0 + 8 <= V) {
      const uint4* q = reinterpret_cast<const uint4*>(at);
#pragma unroll
      for (int i = 0; i < Unit<T>::NV; ++i) r.v[i] = q[i];
      r.ok = 0xFFu;
      if (MASK) {  // bits j0 .. j0 + 7, of one word or two
        const int w = j0 >> 5, s = j0 & 31;
        const uint32_t lo = __ldg(bits + w), hi = s > 24 ? __ldg(bits + w + 1) : 0u;
        r.ok = __funnelshift_r(lo, hi, s) & 0xFFu;
      }
    } else {  // the row begins or ends inside
      uint32_t h[8] = {};
      r.ok = 0u;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + e;
        if (j < 0 || j >= V || !allowed(j)) continue;
        r.ok |= 1u << e;
        uint32_t v;
        if (T == MOE_T_F32) v = __ldg(reinterpret_cast<const uint32_t*>(row) + j);
        else v = (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row) + j) << (16 * (e & 1));
        const int word = T == MOE_T_F32 ? e : e >> 1;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] |= i == word ? v : 0u;
      }
      r.v[0] = make_uint4(h[0], h[1], h[2], h[3]);
      if (Unit<T>::NV == 2) r.v[Unit<T>::NV - 1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
    return r;
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared-memory object in block `rank` of the cluster.
template <class P>
__device__ __forceinline__ const P* in_block(const P* p, uint32_t rank) {
  u64 d;
  asm("mapa.u64 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<u64>(p)), "r"(rank));
  return reinterpret_cast<const P*>(d);
}

struct LogprobArgs {
  LogprobParams p;
  int cl;      // blocks per row
};

template <int T, bool MASK>
__global__ void __launch_bounds__(THREADS, 2) k_token_logprobs(const LogprobArgs a) {
  extern __shared__ __align__(128) uint8_t batches[];  // two of BATCH_BYTES
  __shared__ Shared sh;
  const LogprobParams& p = a.p;
  constexpr int BU = BATCH_UNITS<T>, B = BU / THREADS;
  constexpr uint32_t UB = BATCH_BYTES / BU;  // bytes of a unit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = p.c.top_k;
  const long long r = (long long)blockIdx.x / a.cl;
  const uint32_t rank = a.cl > 1 ? cluster_rank() : 0u;
  grid_launch_dependents();
  const RowView<T, MASK> row(p, r);
  const int units = row.units(), in0 = row.inner_begin(), in1 = row.inner_end();
  const int u0 = (int)((long long)units * rank / a.cl), u1 = (int)((long long)units * (rank + 1) / a.cl);
  const int nb = (u1 - u0 + BU - 1) / BU;
  uint64_t* full = reinterpret_cast<uint64_t*>(sh.full);
  auto inner = [&](int b, int& lo, int& hi) {  // the inner units of batch b
    lo = max(u0 + b * BU, in0);
    hi = min(min(u0 + (b + 1) * BU, u1), in1);
  };
  auto fetch = [&](int b) {  // one thread
    int lo, hi;
    inner(b, lo, hi);
    if (b >= nb || lo >= hi) return;
    const uint32_t bytes = (uint32_t)(hi - lo) * UB;
    mbar_arrive_expect_tx(full + (b & 1), bytes);
    bulk_g2s(batches + (uint32_t)(b & 1) * BATCH_BYTES + (uint32_t)(lo - u0 - b * BU) * UB,
             row.row + (8ll * lo - row.off), bytes, full + (b & 1));
  };
  if (tid == 0) {
    mbar_init(full, 1);
    mbar_init(full + 1, 1);
    fence_mbar_init();
    sh.failed = 0u;
    sh.pushed[0] = sh.pushed[1] = sh.pushed[2] = 0;
  }
  grid_wait();
  if (tid == 0) {
    fetch(0);
    fetch(1);
  }
  const uint64_t deadline = globaltimer_ns() + 2000000000ull;
  const int t = p.target ? p.target[r] : -1;
  const bool scored = t >= 0 && t < row.V;
  const float rt = 1.0f / p.c.temperature;
  const float k = 1.4426950408889634f * rt;
  const u64 k2 = pack(k, k);
  // the target's logit; +inf (nothing is above it) where no rank is asked for
  float xt = -pos_inf();
  if (scored && row.allowed(t)) xt = Elem<T>::get(row.row[t]);
  const float xr = scored && p.rank ? xt : pos_inf();
  __syncthreads();

  float M = LOWEST;
  u64 S2 = pack(0.f, 0.f), U2 = S2;
  int above = 0, n = 0;  // n: keys in the buffer
  u64 thr = 0;           // keys below it are not among the top k
  float tf = K > 0 ? -pos_inf() : pos_inf();
  for (int b = 0; b < nb; ++b) {
    const int b0 = u0 + b * BU;
    const uint8_t* batch = batches + (uint32_t)(b & 1) * BATCH_BYTES;
    {
      int lo, hi;
      inner(b, lo, hi);
      if (lo < hi && !mbar_try_wait(full + (b & 1), (uint32_t)(b >> 1) & 1u))
        mbar_wait_bounded(full + (b & 1), (uint32_t)(b >> 1) & 1u, deadline, &sh.failed);
    }
    if (b == 0 && K > 0) {
      // a first lower bound of the k-th largest key: that of the threads' maxima
      u64 best = 0;
#pragma unroll 1
      for (int i = 0; i < B; ++i) {
        const int u = b0 + i * THREADS + tid;
        if (u >= u1) break;
        const Unit<T> c = row.load(u, batch + (uint32_t)(i * THREADS + tid) * UB);
        float x[8];
        c.to_f32(x);
        float m = -pos_inf();
        int at = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (((c.ok >> e) & 1u) && x[e] >= m && (at < 0 || x[e] > m)) {
            m = x[e];
            at = e;
          }
        if (at >= 0) {
          const u64 key = rank_key(m, 8 * u - row.off + at);
          best = key > best ? key : best;
        }
      }
      sh.buf[tid] = best;
      __syncthreads();
      block_top(sh, sh.buf, THREADS);
      thr = sh.lists[0][K - 1];
      tf = thr >> 32 ? key_value(thr) : -pos_inf();
      __syncthreads();
    }
    // a unit whose maximum stays below `lim` adds to the sums alone
    float lim = fminf(M, fminf(tf, xr));
    uint32_t again = 0;  // units with candidates for the top
#pragma unroll 1
    for (int i = 0; i < B; ++i) {
      const int u = b0 + i * THREADS + tid;
      if (u >= u1) break;
      const Unit<T> c = row.load(u, batch + (uint32_t)(i * THREADS + tid) * UB);
      float x[8];
      c.to_f32(x);
      if (c.ok != 0xFFu) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (c.ok >> e) & 1u ? x[e] : -pos_inf();
      }
      const float mv = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      if (mv >= lim || thr >> 32 == 0) {
        if (mv > M) {
          const float d = fmaxf(M - mv, FAR), e = ex2(d * k);
          U2 = mul2(fma2(S2, pack(d, d), U2), pack(e, e));
          S2 = mul2(S2, pack(e, e));
          M = mv;
          lim = fminf(M, fminf(tf, xr));
        }
        if (mv > xr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) above += x[e] > xr;
        }
        if (K > 0 && (mv >= tf || thr >> 32 == 0)) again |= 1u << i;
      }
      const u64 nm = pack(-M, -M);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float d0, d1, a0, a1;
        unpack(add2(pack(x[e], x[e + 1]), nm), d0, d1);
        const u64 d = pack(max_nan(d0, FAR), max_nan(d1, FAR));
        unpack(mul2(d, k2), a0, a1);
        const u64 ee = pack(ex2(a0), ex2(a1));
        S2 = add2(S2, ee);
        U2 = fma2(ee, d, U2);
      }
    }
    if (K > 0) {
      if (tid == 0) sh.pushed[(b + 1) % 3] = 0;  // last read two barriers ago
      int* pushed = &sh.pushed[b % 3];
      for (;;) {
        for (uint32_t left = again; left; left &= left - 1) {
          const int i = __ffs(left) - 1;
          const int u = b0 + i * THREADS + tid;
          const Unit<T> c = row.load(u, batch + (uint32_t)(i * THREADS + tid) * UB);
          float x[8];
          c.to_f32(x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!((c.ok >> e) & 1u) || x[e] < tf) continue;
            const u64 key = rank_key(x[e], 8 * u - row.off + e);
            if (key < thr) continue;
            const int at = n + atomicAdd(pushed, 1);
            if (at < CAP) sh.buf[at] = key;
          }
        }
        __syncthreads();
        const int now = n + *pushed;
        if (now <= CAP / 2) {
          n = now;
          break;
        }
        // the buffer fills up: raise the bound; keep the best, or, where keys
        // were lost, the bound alone, and take the batch again
        block_top(sh, sh.buf, min(now, CAP));
        thr = sh.lists[0][K - 1];
        tf = thr >> 32 ? key_value(thr) : -pos_inf();
        if (now <= CAP) {
          if (tid < 32) sh.buf[tid] = sh.lists[0][tid];
          n = 32;
        }
        if (tid == 0) *pushed = 0;
        __syncthreads();
        if (now <= CAP) break;
      }
    } else {
      __syncthreads();
    }
    if (tid == 0) fetch(b + 2);  // every thread is done with this batch
  }

  if (sh.failed && tid == 0) {  // the copies in flight land before the block leaves
    const uint64_t d2 = globaltimer_ns() + 2000000000ull;
    for (int b = max(0, nb - 2); b < nb; ++b) {
      int lo, hi;
      inner(b, lo, hi);
      if (lo < hi) mbar_wait_bounded(full + (b & 1), (uint32_t)(b >> 1) & 1u, d2, &sh.failed);
    }
  }

  // the block's statistics and list
  Stat st;
  {
    float s0, s1, v0, v1;
    unpack(S2, s0, s1);
    unpack(U2, v0, v1);
    st = Stat{M, s0 + s1, v0 + v1, above};
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Stat w;
    w.M = __shfl_xor_sync(0xffffffffu, st.M, o);
    w.S = __shfl_xor_sync(0xffffffffu, st.S, o);
    w.U = __shfl_xor_sync(0xffffffffu, st.U, o);
    w.above = __shfl_xor_sync(0xffffffffu, st.above, o);
    // the same order on both sides
    st = (lane & o) ? join(w, st, k) : join(st, w, k);
  }
  if (lane == 0) sh.stat[warp] = st;
  __syncwarp();
  if (K > 0) {
    block_top(sh, sh.buf, n);
    if (tid < 32) sh.best[tid] = sh.lists[0][tid];
  }
  // a NaN target ranks below every number: count those
  if (scored && p.rank && xt != xt) {
    int c = 0;
    for (int j = 8 * u0 - row.off + tid; j < 8 * u1 - row.off; j += THREADS) {
      if (j < 0 || j >= row.V || !row.allowed(j)) continue;
      const float x = Elem<T>::get(row.row[j]);
      c += x == x;
    }
    atomicAdd(&sh.stat[warp].above, c);  // lane 0's zero so far: no entry is above a NaN
  }
  __syncthreads();
  if (warp == 0) {
    st = sh.stat[lane < WARPS ? lane : 0];
    if (lane >= WARPS) st = Stat{LOWEST, 0.f, 0.f, 0};
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      Stat w;
      w.M = __shfl_xor_sync(0xffffffffu, st.M, o);
      w.S = __shfl_xor_sync(0xffffffffu, st.S, o);
      w.U = __shfl_xor_sync(0xffffffffu, st.U, o);
      w.above = __shfl_xor_sync(0xffffffffu, st.above, o);
      st = (lane & o) ? join(w, st, k) : join(st, w, k);
    }
    if (sh.failed) st.S = __uint_as_float(0x7FC00000u);
    if (lane == 0) sh.total = st;
  }
  if (a.cl > 1) {
    cluster_sync();
    if (rank == 0) {
      if (warp == 0) {
        st = lane < a.cl ? *in_block(&sh.total, (uint32_t)lane) : Stat{LOWEST, 0.f, 0.f, 0};
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          Stat w;
          w.M = __shfl_xor_sync(0xffffffffu, st.M, o);
          w.S = __shfl_xor_sync(0xffffffffu, st.S, o);
          w.U = __shfl_xor_sync(0xffffffffu, st.U, o);
          w.above = __shfl_xor_sync(0xffffffffu, st.above, o);
          st = (lane & o) ? join(w, st, k) : join(st, w, k);
        }
      }
      if (K > 0) {
        u64 v = warp < a.cl ? in_block(sh.best, (uint32_t)warp)[lane] : 0;
        sh.lists[warp][lane] = v;
        for (int s = MAX_CLUSTER / 2; s; s >>= 1) {
          __syncthreads();
          if (warp < s) {
            v = warp_merge(v, sh.lists[warp + s][lane]);
            sh.lists[warp][lane] = v;
          }
        }
        __syncthreads();
      }
    }
    cluster_sync();  // no block leaves while its shared memory is read
    if (rank != 0) return;
  }
  if (warp != 0) return;
  const float inf = pos_inf(), nan = __uint_as_float(0x7FC00000u);
  const bool empty = st.S == 0.f;
  const float ls = logf(st.S);
  if (lane == 0) {
    if (p.lse) p.lse[r] = empty ? -inf : st.M * rt + ls;
    if (p.entropy) p.entropy[r] = empty ? 0.f : ls - st.U / st.S * rt;
    if (p.logprob) p.logprob[r] = scored ? (empty ? -inf : (xt - st.M) * rt - ls) : (t == -1 ? 0.f : nan);
    if (p.rank) p.rank[r] = scored ? st.above + 1 : (t == -1 ? 0 : -1);
  }
  if (lane < K) {
    const u64 key = sh.lists[0][lane];
    p.top_logprob[r * K + lane] = key == 0 || empty ? -inf : (key_value(key) - st.M) * rt - ls;
    p.top_id[r * K + lane] = key ? key_id(key) : -1;
  }
}

template <int T, bool MASK>
int launch(const LogprobArgs& a, cudaStream_t s) {
  static int attr_dev = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (attr_dev != dev) {
    if (cudaFuncSetAttribute(k_token_logprobs<T, MASK>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(k_token_logprobs<T, MASK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             2 * (int)BATCH_BYTES) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_dev = dev;
  }
  return launch_overlapped(k_token_logprobs<T, MASK>, dim3((unsigned)a.p.m * (unsigned)a.cl), dim3(THREADS),
                           2 * BATCH_BYTES, s, a, a.cl);
}

template <int T>
int launch_m(const LogprobArgs& a, cudaStream_t s) {
  return a.p.allowed ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

int launch_token_logprobs(const LogprobParams& p0, cudaStream_t s) {
  // rows a launch, so that the grid stays below 2^31 blocks
  constexpr int ROWS = 1 << 26;
  for (int r0 = 0; r0 < p0.m; r0 += ROWS) {
    LogprobArgs a{};
    a.p = p0;
    LogprobParams& p = a.p;
    p.m = p0.m - r0 < ROWS ? p0.m - r0 : ROWS;
    p.logits = static_cast<const char*>(p0.logits) + (size_t)r0 * p0.ld * type_bytes(p0.c.logit_type);
    if (p.allowed) p.allowed += (size_t)r0 * p0.ld_allowed;
    if (p.target) p.target += r0;
    if (p.logprob) p.logprob += r0;
    if (p.rank) p.rank += r0;
    if (p.lse) p.lse += r0;
    if (p.entropy) p.entropy += r0;
    if (p.top_logprob) p.top_logprob += (size_t)r0 * p0.c.top_k;
    if (p.top_id) p.top_id += (size_t)r0 * p0.c.top_k;
    // blocks per row: enough to fill the GPU twice over, while a block's slice
    // fills its threads
    const int batch = (int)BATCH_BYTES / type_bytes(p.c.logit_type);
    a.cl = 1;
    while (a.cl < MAX_CLUSTER && (long long)p.m * a.cl < 304 && p.c.vocab / (2 * a.cl) >= batch / 2) a.cl *= 2;
    int rc;
    if (p.c.logit_type == MOE_T_F32) rc = launch_m<MOE_T_F32>(a, s);
    else if (p.c.logit_type == MOE_T_BF16) rc = launch_m<MOE_T_BF16>(a, s);
    else rc = launch_m<MOE_T_F16>(a, s);
    if (rc) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
