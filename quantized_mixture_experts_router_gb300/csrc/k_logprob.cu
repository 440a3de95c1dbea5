// Log probabilities of given tokens, entropy and the top alternatives of each
// row of logits.  With z = logit / T over the allowed entries, M = max z,
// S = sum exp(z - M), U = sum exp(z - M) (z - M) / log 2:
//   lse = M + log S,  logprob = (z_t - M) - log S,  entropy = log S - U / S log 2
// (differences are taken around M before anything is rounded away, so that
// large common offsets cost no digits).
//
// Bound by one read of the logits.
//  - A row belongs to a cluster of 1..16 blocks (the fewer rows the more), a
//    contiguous slice each, whose results meet in distributed shared memory; a
//    cluster walks through several rows when there are many.
//  - Each warp streams its own pieces (4 KB of f32, 2 KB of 16 bits) of the slice
//    with bulk copies into a ring of its own, across the ends of rows, so that the
//    loads in flight cost no registers and warps meet twice a row only.  (Units of
//    eight entries that the row begins or ends inside are read entry by entry.)
//  - A thread keeps S and U of its own, around a reference that moves only when
//    an entry exceeds it by a factor of 2^8 (the first unit's maximum at first),
//    so that a warp hardly ever diverges to rescale them; they are packed pairs
//    of f32 (two sums an instruction).  Rank and reference cost one comparison
//    of the unit's maximum with min(reference + 8 bits, the target's logit).
//  - Top entries take nothing from the stream but maxima: each thread's (short
//    slices), or each piece's (long ones).  They are distinct entries,
//    so with w warps holding a value a lane the least of the warps' ceil(k / w)-th
//    largest ones bounds the k-th largest key (value, then lower id: a 64-bit
//    number) from below, and the top entries belong to the few threads or pieces
//    whose maximum reaches the bound: those are read again, what reaches the
//    bound goes to a buffer, and the places in order are counted.  Where a mask
//    leaves some warp too few values, the bound is the k-th largest of them all.
//    Where the buffer overflows (many equal entries, or a row's allowed entries
//    in few pieces), they are gone through once more, an entry a thread at a time,
//    and the bound rises whenever the buffer is nearly full.
// Sums follow the fixed order of threads, warps and blocks; the buffer's order
// varies, its sorted content does not.
// Measured: 512 f32 rows of 131072, top 20: 57 us, 4.7 TB/s (43 us and 6.2 TB/s
// without top entries; copies reach 6.8).  1000 bf16 rows of 50001, top 5: 42 us,
// 2.4 TB/s: instructions bound it, and 1000 rows over 608 blocks leave the second
// turn a third empty.  One f32 row of 131072 under a mask, top 20: 8.3 us.
#include "ops.h"
#include "select.cuh"

namespace moe {

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int CAP = 768;              // keys of the candidate buffer
constexpr int MAX_CLUSTER = 16;
constexpr int SEGS = 2 * THREADS;     // piece maxima of a row
constexpr int STAGES = 2;             // pieces of a warp's ring
// Bytes of a piece and blocks an SM holds: f32 rows are long and take few
// instructions a byte, 16-bit rows need the warps (512 f32 rows of 131072: 60 us
// with 4 KB pieces and two blocks, 66 us with 2 KB and four, when this was
// chosen; 1000 bf16 rows of 50001: 55 and 43 us).
template <int T>
constexpr uint32_t PIECE_BYTES = T == MOE_T_F32 ? 4096 : 2048;
template <int T>
constexpr int BLOCKS_PER_SM = T == MOE_T_F32 ? 2 : 4;
template <int T>
constexpr uint32_t RING_BYTES = WARPS * STAGES * PIECE_BYTES<T>;
constexpr uint64_t TIMEOUT_NS = 2000000000ull;  // of one wait for a copy
constexpr uint32_t LOST = 1u << 31;   // above any number of pieces: they are 2 KB at least
constexpr float LOWEST = -3.4028234663852886e38f;
constexpr float FAR = -256.0f;        // an exponent of two whose power is zero, but whose product with it is not NaN

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

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// S += e, U += e h with e = exp2(h), h = (x - M) k, for eight entries; CLAMP: an
// infinite h counts as FAR (the product with its e = 0 is 0 then, not NaN).  U is
// kept in h, not in x - M, so that neither FAR nor U's size depends on the
// temperature.
template <bool CLAMP, int N>
__device__ __forceinline__ void add_unit(const float (&x)[N], float M, float k, float2& S, float2& U) {
  const float2 nm = make_float2(-M, -M), kk = make_float2(k, k);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    float2 h = __fmul2_rn(__fadd2_rn(make_float2(x[e], x[e + 1]), nm), kk);
    if (CLAMP) h = make_float2(max_nan(h.x, FAR), max_nan(h.y, FAR));
    const float2 w = make_float2(ex2(h.x), ex2(h.y));
    S = __fadd2_rn(S, w);
    U = __ffma2_rn(w, h, U);
  }
}

// How many of eight entries are above r (as 1.0 each: set and packed add).
template <int N>
__device__ __forceinline__ float count_above(const float (&x)[N], float r) {
  float2 c = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    float2 s;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(s.x) : "f"(x[e]), "f"(r));
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(s.y) : "f"(x[e + 1]), "f"(r));
    c = __fadd2_rn(c, s);
  }
  return c.x + c.y;
}

// The running statistics of a set of entries.
struct Stat {
  float M, S, U;
  int above;  // entries above the target's; -1: the set could not be read
};

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

template <int T>
constexpr int PIECE_UNITS = PIECE_BYTES<T> / (8 * (T == MOE_T_F32 ? 4 : 2));

// f32 as an unsigned number of the same order (0 for "none").
__device__ __forceinline__ unsigned ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float from_ordered(unsigned o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// What one row leaves in shared memory; two rows' worth alternate.
struct RowState {
  alignas(16) u64 buf[CAP];
  u64 best[32];              // the block's list, descending
  Stat stat[WARPS];
  Stat total;                // the block's, read by the cluster's first block
  unsigned bound[WARPS];     // ordered bits of each warp's bound
  int n;                     // keys pushed (counted past CAP)
  int nhot;
  unsigned seg[SEGS];        // ordered bits of the pieces' maxima, 2^sh pieces each; zero between rows
  uint16_t hot[SEGS];        // threads or segments whose maximum reaches the bound
};

// Where a warp's copies stand: pieces of the rows its block walks through, as
// byte offsets from the 16-byte aligned address at or below a row's start.
struct Cursor {
  const uint8_t* base;
  uint32_t at, lo, hi, end;  // the next piece; the inner units; the slice's end
  int row;                   // the row of `base`
  uint32_t fetched;          // pieces so far
};

struct Shared {
  Cursor cursor[WARPS];
  u64 full[WARPS][STAGES];   // a piece has landed
  u64 lists[WARPS][32];
  RowState row[2];
  unsigned failed;           // a wait ran out: the results are NaN
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

// log2 of the pieces of a segment: at most SEGS segments.
__device__ __forceinline__ int seg_shift(int np) { return max(0, 32 - __clz((np - 1) >> 9)); }
static_assert(SEGS == 512, "seg_shift");

// Eight entries of the row.
template <int T>
struct Unit {
  static constexpr int NV = T == MOE_T_F32 ? 2 : 1;
  uint4 v[NV];
  uint32_t ok;  // bit e: entry e is in the row and allowed
  __device__ __forceinline__ void to_f32(float* x) const {
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
  __device__ __forceinline__ Unit<T> inner(const uint8_t* at) const {
    Unit<T> r;
#pragma unroll
    for (int i = 0; i < Unit<T>::NV; ++i) r.v[i] = reinterpret_cast<const uint4*>(at)[i];
    r.ok = 0xFFu;
    return r;
  }
  // unit u; `at`: its place in shared memory, for inner units
  __device__ __forceinline__ Unit<T> load(int u, const uint8_t* at) const {
    Unit<T> r;
    const int j0 = 8 * u - off;
    if (j0 >= 0 && j0 + 8 <= V) {
      r = inner(at);
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
// Not the .aligned forms: they need a warp whose threads arrive together, which
// nothing but the compiler's choice gives after a branch of one thread.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
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
  int cl, cl_log2;  // blocks per row, a power of two
};

// The lanes' statistics joined around the largest M; the sums in a butterfly,
// whose order is fixed.
__device__ __forceinline__ Stat warp_join(Stat st, float k) {
  const float M = from_ordered(__reduce_max_sync(0xffffffffu, ordered(st.M)));
  const float h = max_nan((st.M - M) * k, FAR), e = ex2(h);
  st.U = (st.U + st.S * h) * e;
  st.S *= e;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    st.S += __shfl_xor_sync(0xffffffffu, st.S, o);
    st.U += __shfl_xor_sync(0xffffffffu, st.U, o);
  }
  const bool failed = __any_sync(0xffffffffu, st.above < 0);
  st.above = failed ? -1 : (int)__reduce_add_sync(0xffffffffu, (unsigned)st.above);
  st.M = M;
  return st;
}

// The slice of a row that a block reads, in pieces of PIECE_UNITS that its
// warps take in turn.
template <int T, bool MASK>
struct Slice {
  RowView<T, MASK> row;
  int u0, u1, np;
  __device__ __forceinline__ Slice(const LogprobArgs& a, long long r, uint32_t rank) : row(a.p, r) {
    const int units = row.units();
    u0 = (int)(((long long)units * rank) >> a.cl_log2);
    u1 = (int)(((long long)units * (rank + 1)) >> a.cl_log2);
    np = (u1 - u0 + PIECE_UNITS<T> - 1) / PIECE_UNITS<T>;
  }
};

// The threads' or pieces' maxima that are to be read again, as units of the row.
template <int T, bool MASK, bool by_piece>
struct HotUnits {
  const Slice<T, MASK>& s;
  const RowState& rs;
  int per, lg;  // units of a hot thread or segment, and log2 of the next power of two
  __device__ __forceinline__ HotUnits(const Slice<T, MASK>& s, const RowState& rs) : s(s), rs(rs) {
    constexpr int B = PIECE_UNITS<T> / 32;
    per = by_piece ? PIECE_UNITS<T> << seg_shift(s.np) : (s.np + WARPS - 1) / WARPS * B;
    lg = per > 1 ? 32 - __clz(per - 1) : 0;
  }
  __device__ __forceinline__ int items() const { return rs.nhot << lg; }
  // the unit of item q, or -1
  __device__ __forceinline__ int operator()(int q) const {
    constexpr int B = PIECE_UNITS<T> / 32;
    const int h = rs.hot[q >> lg], j = q & ((1 << lg) - 1);
    const int u = s.u0 + (by_piece ? h * per + j : ((h >> 5) + WARPS * (j / B)) * PIECE_UNITS<T> + (j % B) * 32 + (h & 31));
    return j < per && u < s.u1 ? u : -1;
  }
};

// The k-th largest of the block's values, one or two a thread (0 where there are
// fewer).  The buffer is not in use yet.
template <bool TWO>
__device__ __forceinline__ unsigned kth_value(Shared& sh, RowState& rs, unsigned v0, unsigned v1, int k) {
  rs.buf[threadIdx.x] = (u64)v0 << 32;
  if (TWO) rs.buf[threadIdx.x + THREADS] = (u64)v1 << 32;
  __syncthreads();
  block_top(sh, rs.buf, (TWO ? 2 : 1) * THREADS);
  return (unsigned)(sh.lists[0][k - 1] >> 32);
}

// Where more keys than the buffer takes reach thr: fills it anew from the hot
// units, an entry of every thread at a time, and keeps the 32 largest whenever
// the next entries might not fit.  Returns the number of keys.
template <int T, bool MASK, bool by_piece>
__device__ __forceinline__ int refill(const LogprobArgs& a, Shared& sh, RowState& rs, int r, uint32_t rank, u64 thr) {
  const Slice<T, MASK> s(a, r, rank);
  const HotUnits<T, MASK, by_piece> hot(s, rs);
  const int items = hot.items();
  int n = 0;
  __syncthreads();  // every thread has read the count that brought it here
  if (threadIdx.x == 0) rs.n = 0;
  __syncthreads();
  for (int q0 = 0; q0 < items; q0 += THREADS) {
    const int q = q0 + (int)threadIdx.x, u = q < items ? hot(q) : -1;
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const int id = 8 * u - s.row.off + e;
      u64 key = 0;
      if (u >= 0 && id >= 0 && id < s.row.V && s.row.allowed(id)) key = rank_key(Elem<T>::get(s.row.row[id]), id);
      const bool in = key != 0 && key >= thr;
      if (in) rs.buf[atomicAdd(&rs.n, 1)] = key;
      n += __syncthreads_count(in);
      if (n > CAP - THREADS) {
        block_top(sh, rs.buf, n);
        thr = sh.lists[0][a.p.c.top_k - 1];
        n = 32;
        if (threadIdx.x < 32) rs.buf[threadIdx.x] = sh.lists[0][threadIdx.x];
        if (threadIdx.x == 0) rs.n = n;
        __syncthreads();
      }
    }
  }
  return n;
}
static_assert(CAP >= 2 * THREADS + 32, "an entry of every thread fits after the 32 largest");

template <int T, bool MASK, bool by_piece>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM<T>) k_token_logprobs(const __grid_constant__ LogprobArgs a) {
  extern __shared__ __align__(128) uint8_t rings[];
  __shared__ Shared sh;
  const LogprobParams& p = a.p;
  constexpr int PU = PIECE_UNITS<T>, B = PU / 32;
  constexpr uint32_t UB = PIECE_BYTES<T> / PU;  // bytes of a unit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = p.c.top_k;
  const uint32_t rank = a.cl > 1 ? cluster_rank() : 0u;
  const int step = (int)gridDim.x / a.cl, r0 = (int)blockIdx.x / a.cl;
  uint64_t* full = reinterpret_cast<uint64_t*>(sh.full[warp]);
  uint8_t* ring = rings + warp * STAGES * PIECE_BYTES<T>;
  grid_launch_dependents();
  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  if (tid == 0) {
    sh.failed = 0u;
    sh.row[0].n = sh.row[1].n = sh.row[0].nhot = sh.row[1].nhot = 0;
  }
  for (int i = tid; i < SEGS; i += THREADS) sh.row[0].seg[i] = sh.row[1].seg[i] = 0u;
  __syncthreads();
  grid_wait();
  // lane 0 copies STAGES pieces ahead
  auto fetch_next = [&]() {
    Cursor& cu = sh.cursor[warp];
    uint32_t at = cu.at;
    while (at >= cu.end) {  // this row has no more for the warp
      const int fr = cu.row + step;
      if (fr >= p.m) return;
      const Slice<T, MASK> s(a, fr, rank);
      cu.row = fr;
      cu.base = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(s.row.row) & ~uintptr_t(15));
      cu.end = (uint32_t)s.u1 * UB;
      cu.lo = (uint32_t)s.row.inner_begin() * UB;
      cu.hi = min(cu.end, (uint32_t)s.row.inner_end() * UB);
      at = (uint32_t)s.u0 * UB + (uint32_t)warp * PIECE_BYTES<T>;
      cu.at = at;
    }
    const uint32_t st = cu.fetched % STAGES;
    const uint32_t lo = max(at, cu.lo), hi = min(at + PIECE_BYTES<T>, cu.hi);
    if (lo < hi) {
      mbar_arrive_expect_tx(full + st, hi - lo);
      bulk_g2s(ring + st * PIECE_BYTES<T> + (lo - at), cu.base + lo, hi - lo, full + st);
    } else {
      mbar_arrive(full + st);  // nothing but units the row begins or ends inside
    }
    ++cu.fetched;
    cu.at = at + WARPS * PIECE_BYTES<T>;
  };
  if (lane == 0) {
    sh.cursor[warp] = Cursor{nullptr, 0u, 0u, 0u, 0u, r0 - step, 0u};
    for (int i = 0; i < STAGES; ++i) fetch_next();
  }
  const float rt = 1.0f / p.c.temperature;
  const float k = 1.4426950408889634f * rt;
  const float slack = 8.0f / k;  // at most 6e36: an entry's difference from the reference stays finite upwards

  auto target_of = [&](int r) { return p.target && r < p.m ? __ldg(p.target + r) : -1; };
  auto target_logit = [&](int r, int t) {  // a masked one counts as -inf
    const RowView<T, MASK> row(p, r);
    return t >= 0 && t < row.V && row.allowed(t) ? Elem<T>::get(row.row[t]) : -pos_inf();
  };
  int t_now = target_of(r0), t_next = target_of(r0 + step);
  float xt_now = target_logit(r0, t_now);

  // pieces so far; with LOST, one did not land in time: the warp waits and copies
  // no more, and the block's rows are NaN
  uint32_t used = 0;
  int parity = 0;
  for (int r = r0; r < p.m; r += step, parity ^= 1) {
    RowState& rs = sh.row[parity];
    const Slice<T, MASK> sl(a, r, rank);
    const RowView<T, MASK>& row = sl.row;
    const int u0 = sl.u0, u1 = sl.u1;
    const int t = t_now;
    const bool scored = t >= 0 && t < row.V;
    const float xt = xt_now;
    t_now = t_next;  // the next row's, loaded while this one is worked on
    if (r + step < p.m) xt_now = target_logit(r + step, t_now);
    t_next = target_of(r + 2 * step);
    // +inf (nothing is above it) where no rank is asked for
    const float xr = scored && p.rank ? xt : pos_inf();

    float M = LOWEST;       // the largest entry so far
    float ref = LOWEST;     // S and U are sums around it,
    float ref_hi = LOWEST;  // and it moves when an entry lies above this
    float2 S2 = make_float2(0.f, 0.f), U2 = S2;
    float above = 0.f;      // entries above the target's (at most 2^20 a thread: exact)
    for (int i0 = used < LOST ? warp : sl.np; i0 < sl.np; i0 += WARPS) {
      const int b0 = u0 + i0 * PU;
      const uint32_t st = used % STAGES;
      const uint8_t* mem = ring + st * PIECE_BYTES<T> + lane * UB;
      if (!__all_sync(0xffffffffu, mbar_try_wait(full + st, (used / STAGES) & 1u)) &&
          !__all_sync(0xffffffffu, mbar_wait_for(full + st, (used / STAGES) & 1u, TIMEOUT_NS, &sh.failed))) {
        used |= LOST;
        break;
      }
      // where every lane's maximum stays below `lim`, the units add to the
      // sums alone (the warp decides as one: both ways would cost their sum)
      float lim = fminf(ref_hi, xr), Mp = LOWEST;
      auto work = [&](const auto& x, unsigned lanes) {
        constexpr int N = (int)(sizeof(x) / sizeof(float));
        float mv = max3(x[5], x[6], x[7]), mw = max3(x[0], x[1], x[2]);
#pragma unroll
        for (int e = 8; e < N; e += 2) mv = max3(mv, x[e], x[e + 1]);
        mv = fmaxf(max3(mw, x[3], x[4]), mv);
        Mp = fmaxf(Mp, mv);
        if (__any_sync(lanes, mv >= lim)) {
          if (mv > ref_hi) {
            const float h = fmaxf((ref - mv) * k, FAR), e = ex2(h);
            U2 = make_float2((U2.x + S2.x * h) * e, (U2.y + S2.y * h) * e);
            S2 = make_float2(S2.x * e, S2.y * e);
            ref = mv;
            ref_hi = mv + slack;
            lim = fminf(ref_hi, xr);
          }
          above += count_above(x, xr);
        }
      };
      const bool plain = !MASK && b0 >= row.inner_begin() && b0 + PU <= min(u1, row.inner_end());  // whole units alone
      if (plain) {
        const float2 S0 = S2, U0 = U2;
        const float ref0 = ref;
#pragma unroll 1
        for (int i = 0; i < B; i += 2) {
          float x[16];
          row.inner(mem + (uint32_t)i * (32 * UB)).to_f32(x);
          row.inner(mem + (uint32_t)(i + 1) * (32 * UB)).to_f32(x + 8);
          work(x, 0xffffffffu);
          add_unit<false>(x, ref, k, S2, U2);
        }
        // an entry too far below the reference (-inf) has made 0 * inf of its
        // product: take the piece's sums again, with a bound on the exponent
        const float u = U2.x + U2.y, u0 = U0.x + U0.y;
        if (__any_sync(0xffffffffu, u != u && u0 == u0)) {
          const float h = fmaxf((ref0 - ref) * k, FAR), e = ex2(h);
          U2 = make_float2((U0.x + S0.x * h) * e, (U0.y + S0.y * h) * e);
          S2 = make_float2(S0.x * e, S0.y * e);
#pragma unroll 1
          for (int i = 0; i < B; ++i) {
            float x[8];
            row.inner(mem + (uint32_t)i * (32 * UB)).to_f32(x);
            add_unit<true>(x, ref, k, S2, U2);
          }
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < B; ++i) {
          const int u = b0 + i * 32 + lane;
          const unsigned lanes = __ballot_sync(0xffffffffu, u < u1);
          if (u < u1) {
            const Unit<T> c = row.load(u, mem + (uint32_t)i * (32 * UB));
            float x[8];
            c.to_f32(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (c.ok >> e) & 1u ? x[e] : -pos_inf();
            work(x, lanes);
            add_unit<true>(x, ref, k, S2, U2);
          }
          __syncwarp();
        }
      }
      M = fmaxf(M, Mp);
      if (by_piece && K > 0) {
        const int sh_seg = seg_shift(sl.np);
        const unsigned m = __reduce_max_sync(0xffffffffu, Mp > LOWEST ? ordered(Mp) : 0u);
        if (lane == 0) atomicMax(&rs.seg[i0 >> sh_seg], m);
      }
      __syncwarp();  // the warp is done with this piece
      if (lane == 0) fetch_next();
      ++used;
    }

    // the block's statistics and list
    {
      // (the sums are around ref; a warp's largest ref stands for its M)
      const Stat st = warp_join(Stat{ref, S2.x + S2.y, U2.x + U2.y, (int)above}, k);
      if (lane == 0) rs.stat[warp] = st;
    }
    // a NaN target ranks below every number: count those
    if (scored && p.rank && xt != xt) {
      int c = 0;
      for (int j = 8 * u0 - row.off + tid; j < 8 * u1 - row.off; j += THREADS) {
        if (j < 0 || j >= row.V || !row.allowed(j)) continue;
        const float x = Elem<T>::get(row.row[j]);
        c += x == x;
      }
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) rs.stat[warp].above = c;  // zero so far: no entry is above a NaN
    }
    if (K > 0) {
      const int sh_seg = seg_shift(sl.np);
      if (by_piece) __syncthreads();  // the segments' maxima are complete
      // values of distinct entries, one or two a thread; the warp's bound is its
      // nth largest lane
      const int nseg = ((sl.np - 1) >> sh_seg) + 1;
      const unsigned v0 = by_piece ? rs.seg[tid] : (M > LOWEST ? ordered(M) : 0u);
      const unsigned v1 = by_piece ? rs.seg[tid + THREADS] : 0u;
      const int busy = by_piece ? min(WARPS, (nseg + 31) >> 5) : max(1, min(WARPS, sl.np));  // warps with values
      {
        const int nth = (K + busy - 1) / busy;
        unsigned o = max(v0, v1), m = __reduce_max_sync(0xffffffffu, o);
        for (int i = 1; i < nth; ++i) {
          const unsigned at = __ballot_sync(0xffffffffu, o == m);
          if (lane == __ffs(at) - 1) o = 0u;
          m = __reduce_max_sync(0xffffffffu, o);
        }
        if (lane == 0) rs.bound[warp] = m;
      }
      if (tid < 32) rs.best[tid] = 0;
      __syncthreads();
      unsigned bound = __reduce_min_sync(0xffffffffu, lane < busy ? rs.bound[lane] : 0xFFFFFFFFu);
      if (bound == 0) bound = kth_value<by_piece>(sh, rs, v0, v1, K);
      u64 thr = (u64)bound << 32;  // keys below it are not among the top k; 0: no bound, NaN may be among them
      float tf = bound ? from_ordered(bound) : -pos_inf();
      const bool live = !by_piece || tid < nseg;
      if (live && v0 >= bound) rs.hot[atomicAdd(&rs.nhot, 1)] = (uint16_t)tid;
      if (by_piece) {
        if (tid + THREADS < nseg && v1 >= bound) rs.hot[atomicAdd(&rs.nhot, 1)] = (uint16_t)(tid + THREADS);
        rs.seg[tid] = rs.seg[tid + THREADS] = 0u;  // for the row after the next
      }
      __syncthreads();
      auto unit_at = [&](int u) {  // unit u, from global memory
        return row.load(u, reinterpret_cast<const uint8_t*>(row.row + (8ll * u - row.off)));
      };
      auto push = [&](const Unit<T>& c, int u) {
        float x[8];
        c.to_f32(x);
        uint32_t left = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) left |= (x[e] < tf ? 0u : 1u) << e;
        for (left &= c.ok; left; left &= left - 1) {
          const int e = __ffs(left) - 1, id = 8 * u - row.off + e;
          const u64 key = rank_key(Elem<T>::get(row.row[id]), id);
          if (key < thr) continue;
          const int at = atomicAdd(&rs.n, 1);
          if (at < CAP) rs.buf[at] = key;
        }
      };
      if (by_piece) {  // (hot segment, piece of it) over the warps, the loads of a piece together
        const int items = rs.nhot << sh_seg;
        for (int q = warp; q < items; q += WARPS) {
          const int i0 = (rs.hot[q >> sh_seg] << sh_seg) + (q & ((1 << sh_seg) - 1));
          const int base = u0 + i0 * PU + lane;
          Unit<T> c[B];
#pragma unroll
          for (int i = 0; i < B; ++i) {
            c[i].ok = 0u;
            if (base + i * 32 < u1) c[i] = unit_at(base + i * 32);
          }
#pragma unroll
          for (int i = 0; i < B; ++i)
            if (c[i].ok) push(c[i], base + i * 32);
        }
      } else {  // (hot thread, unit of its own) over all threads
        const HotUnits<T, MASK, false> hot(sl, rs);
        const int items = hot.items();
        for (int q = tid; q < items; q += THREADS) {
          const int u = hot(q);
          if (u >= 0) push(unit_at(u), u);
        }
      }
      __syncthreads();
      int n = rs.n;
      if (n > CAP) n = refill<T, MASK, by_piece>(a, sh, rs, r, rank, thr);
      if (n <= THREADS) {  // each key's place is the number of larger ones
        const u64 key = tid < n ? rs.buf[tid] : 0;
        if (warp * 32 < n) {
          int place = 0;
          for (int j = 0; j + 1 < n; j += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(rs.buf + j);
            place += (v.x > key) + (v.y > key);
          }
          if (n & 1) place += rs.buf[n - 1] > key;
          if (tid < n && place < 32) rs.best[place] = key;
        }
      } else {
        block_top(sh, rs.buf, n);
        if (tid < 32) rs.best[tid] = sh.lists[0][tid];
      }
    }
    __syncthreads();
    Stat st;
    if (warp == 0) {
      st = warp_join(lane < WARPS ? rs.stat[lane] : Stat{LOWEST, 0.f, 0.f, 0}, k);
      if (sh.failed) {
        st.S = __uint_as_float(0x7FC00000u);
        st.above = -1;
      }
      if (lane == 0) rs.n = rs.nhot = 0;  // for the row after the next
    }
    if (a.cl > 1) {
      if (tid == 0) rs.total = st;
      cluster_sync();
      if (rank == 0) {
        if (warp == 0)
          st = warp_join(lane < a.cl ? *in_block(&rs.total, (uint32_t)lane) : Stat{LOWEST, 0.f, 0.f, 0}, k);
        if (K > 0) {
          u64 v = warp < a.cl ? in_block(rs.best, (uint32_t)warp)[lane] : 0;
          if (warp + WARPS < a.cl) v = warp_merge(v, in_block(rs.best, (uint32_t)(warp + WARPS))[lane]);
          sh.lists[warp][lane] = v;
          for (int s = WARPS / 2; s; s >>= 1) {
            __syncthreads();
            if (warp < s) {
              v = warp_merge(v, sh.lists[warp + s][lane]);
              sh.lists[warp][lane] = v;
            }
          }
          if (warp == 0) rs.best[lane] = v;
        }
      }
      // the others' totals and lists are read before they reach the next row's
      // cluster_sync, and before they leave
      if (r + step >= p.m) cluster_sync();
    }
    if (rank == 0 && warp == 0) {
      __syncwarp();
      const float inf = pos_inf(), nan = __uint_as_float(0x7FC00000u);
      const bool empty = st.S == 0.f, failed = st.above < 0;
      const float ls = logf(st.S);
      if (lane == 0) {
        if (p.lse) p.lse[r] = empty ? -inf : st.M * rt + ls;
        if (p.entropy) p.entropy[r] = empty ? 0.f : ls - st.U / st.S * 0.69314718055994531f;
        if (p.logprob) p.logprob[r] = scored ? (empty ? -inf : (xt - st.M) * rt - ls) : (t == -1 ? 0.f : nan);
        if (p.rank) p.rank[r] = scored && !failed ? st.above + 1 : (t == -1 ? 0 : -1);
      }
      if (lane < K) {
        const u64 key = rs.best[lane];
        p.top_logprob[(long long)r * K + lane] =
            failed ? nan : key == 0 || empty ? -inf : (key_value(key) - st.M) * rt - ls;
        p.top_id[(long long)r * K + lane] = key && !failed ? key_id(key) : -1;
      }
    }
  }
  if (used >= LOST && lane == 0) {  // the warp's copies in flight land before the block leaves
    const uint64_t d2 = globaltimer_ns() + TIMEOUT_NS;
    for (uint32_t v = used - LOST; v < sh.cursor[warp].fetched; ++v)
      mbar_wait_bounded(full + v % STAGES, (v / STAGES) & 1u, d2, &sh.failed);
  }
}

template <int T, bool MASK, bool BY_PIECE>
int launch(const LogprobArgs& a, int sms, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const auto kernel = k_token_logprobs<T, MASK, BY_PIECE>;
  static PerDevice ready;
  if (ready.get(dev, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
               cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RING_BYTES<T>) == cudaSuccess;
      }) < 1)
    return MOE_ERR_CUDA;
  // as many blocks as the SMs hold; clusters of more than two blocks leave some SMs out, so
  // that their number comes from the runtime
  int clusters = BLOCKS_PER_SM<T> * sms / a.cl;
  if (a.cl > 2) {
    static PerDevice fit[MAX_CLUSTER + 1];
    clusters = fit[a.cl].get(dev, [&] {
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)a.cl;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t lc{};
      lc.gridDim = dim3((unsigned)(BLOCKS_PER_SM<T> * sms / a.cl * a.cl));
      lc.blockDim = dim3(THREADS);
      lc.dynamicSmemBytes = RING_BYTES<T>;
      lc.attrs = at;
      lc.numAttrs = 1;
      int n = 0;
      return cudaOccupancyMaxActiveClusters(&n, kernel, &lc) == cudaSuccess ? n : 0;
    });
    if (clusters < 1) return MOE_ERR_CUDA;
  }
  const int grid = (a.p.m < clusters ? a.p.m : clusters) * a.cl;
  return launch_overlapped(kernel, dim3((unsigned)grid), dim3(THREADS), RING_BYTES<T>, s, a, a.cl);
}

template <int T>
int launch_m(const LogprobArgs& a, int sms, cudaStream_t s) {
  // the maxima of pieces rather than threads: reading a thread's units again is
  // reading a little of many pieces, but the pieces' maxima cost the stream.  From 62
  // pieces a slice on for f32, 98 for 16 bits.  Measured, pieces and threads in us:
  //   f32   512 x 50000   49 pieces  35.3 32.9    bf16  1000 x 50001   49 pieces  49.9 42.7
  //         400 x 64000   63         33.9 34.8          1000 x 65536   64         59.4 53.3
  //         512 x 131072 128         57.0 72.5          1000 x 100000  98         82.2 82.7
  //                                                     1000 x 131072 128         96.3 100.3
  const int pieces = a.p.c.vocab / a.cl / (int)(PIECE_BYTES<T> / type_bytes(T));
  const bool by_piece = pieces >= (T == MOE_T_F32 ? 62 : 97);
  if (by_piece) return a.p.allowed ? launch<T, true, true>(a, sms, s) : launch<T, false, true>(a, sms, s);
  return a.p.allowed ? launch<T, true, false>(a, sms, s) : launch<T, false, false>(a, sms, s);
}

}  // namespace

int launch_token_logprobs(const LogprobParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return MOE_ERR_CUDA;
  LogprobArgs a{};
  a.p = p;
  // blocks per row: enough to fill the GPU (four blocks an SM), while a block's
  // slice has 2 KB for each of its warps
  const int piece = 2048 / type_bytes(p.c.logit_type);
  a.cl = 1;
  while (a.cl < MAX_CLUSTER && 2ll * p.m * a.cl <= 4 * sms && p.c.vocab / (2 * a.cl) >= WARPS * piece / 2) a.cl *= 2;
  while ((1 << a.cl_log2) < a.cl) ++a.cl_log2;
  if (p.c.logit_type == MOE_T_F32) return launch_m<MOE_T_F32>(a, sms, s);
  if (p.c.logit_type == MOE_T_BF16) return launch_m<MOE_T_BF16>(a, sms, s);
  return launch_m<MOE_T_F16>(a, sms, s);
}

}  // namespace moe
