// How the attention kernels cut a call into work.  An item is a tile of R rows
// (new tokens x the query heads that share a key head, token by token) of one
// sequence and key head, against the tiles of TK keys that any of its rows sees.
// The items, numbered sequence by sequence, in it head by head, in it row tile by
// row tile, make one line, of which an item takes OVER places (what it costs
// whatever its length, in key tiles) and one for each of its key tiles.  The line
// is cut into about equal runs, one for each block.  A cut near an item's end is moved
// there, each for itself, so that a run can gain at both ends: the longest has about a fifth
// more than an even share where items are many, and half as much again where there are
// as many as blocks; and one of fewer than SNAP places may come out empty.  An item that
// a cut goes through is joined by the last of its blocks to finish, in the order of the runs.
//
// Lengths are on the device, so every block works the cut out for itself.
#pragma once

#include "attn.h"

namespace moe {

constexpr int ATTN_MAX_CTAS = 152;

// Rows and keys of an item's tiles in the kernel for few rows, and in that for many.
constexpr int ATTN_ROWS_TILE = 16, ATTN_ROWS_KEYS = 32, ATTN_TILES_TILE = 256, ATTN_TILES_KEYS = 128;

// Query heads of a key head, and division of rows by them: with s = ceil(log2 n) and
// mul = floor(2^(31 + s) / n) + 1, r mul / 2^(31 + s) is off by less than 1 / n for 0 <= r < 2^31.
struct AttnGroup {
  int n;
  unsigned shift;
  unsigned long long mul;
  static AttnGroup of(int n) {
    AttnGroup g{n, 31, 0};
    while ((1ull << (g.shift - 31)) < (unsigned)n) ++g.shift;
    g.mul = (1ull << g.shift) / (unsigned)n + 1;
    return g;
  }
  __device__ __forceinline__ int token(int row) const { return (int)(((unsigned long long)(unsigned)row * mul) >> shift); }
};

// a / b, quickly where both are small
__device__ __forceinline__ long long attn_div(long long a, long long b) {
  if (((unsigned long long)a | (unsigned long long)b) >> 32) return a / b;
  return (long long)((unsigned)a / (unsigned)b);
}
__device__ __forceinline__ long long attn_warp_sum(long long v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
// of this lane's and all lower lanes' values
__device__ __forceinline__ long long attn_warp_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// One sequence: its first row, new tokens, cached tokens that can be read, and
// the first new token's position.
struct AttnSeq {
  int row0, n, len, pos0;
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
  const int c0 = p.s.cu_new[b], c1 = p.s.cu_new[b + 1], kv = max(p.s.kv_len[b], 0);
  AttnSeq q;
  q.row0 = min(max(c0, 0), p.m);
  q.n = min(max(c1, q.row0), p.m) - q.row0;
  q.len = min(kv, p.s.max_pages * p.c.kv.page_size);
  q.pos0 = kv - (c1 - q.row0);
  return q;
}

// Keys lo .. hi - 1 that rows r0 .. r1 - 1 of a sequence see between them.
struct AttnRange {
  int lo, hi;
};
__device__ __forceinline__ AttnRange attn_range(const AttnParams& p, const AttnSeq& q, const AttnGroup& group, int r0, int r1) {
  AttnRange g{0, q.len};
  if (p.c.causal) {
    g.hi = min(max(q.pos0 + group.token(r1 - 1) + 1, 0), q.len);
    if (p.c.window) g.lo = min(max(q.pos0 + group.token(r0) - p.c.window + 1, 0), g.hi);
  }
  return g;
}

template <int R_, int TK_, int OVER_, int SNAP_, int MIN_RUN_, int JOIN_>
struct AttnWork {
  static constexpr int R = R_, TK = TK_;
  static constexpr int OVER = OVER_;        // places of an item beside its key tiles
  static constexpr int SNAP = SNAP_;        // an item is cut this far from its ends at the least
  static constexpr int MIN_RUN = MIN_RUN_;  // more blocks take part only if each has so many places, or an item
  static constexpr int JOIN = JOIN_;        // what a part costs who joins them, in hundredths of a place
  static_assert(OVER >= 1 && SNAP > OVER, "every part of an item has a key tile");
  static __device__ __forceinline__ int row_tiles(const AttnSeq& q, const AttnGroup& group) {
    return q.n > 0 ? (q.n * group.n - 1) / R + 1 : 0;
  }
  static __device__ __forceinline__ AttnRange range(const AttnParams& p, const AttnSeq& q, const AttnGroup& group, int i) {
    return attn_range(p, q, group, i * R, min((i + 1) * R, q.n * group.n));
  }
  static __device__ __forceinline__ int key_tiles(const AttnRange& g) {
    return g.hi > g.lo ? (g.hi - 1) / TK + 1 - g.lo / TK : 0;
  }
  static __device__ __forceinline__ int cost(const AttnParams& p, const AttnSeq& q, const AttnGroup& group, int i) {
    return OVER + key_tiles(range(p, q, group, i));
  }
  // Places of one key head of each lane's sequence (0 where !valid), and its row tiles, by a whole warp.
  static __device__ long long seq_cost(const AttnParams& p, const AttnGroup& group, int b, bool valid, int* rows = nullptr) {
    const int lane = threadIdx.x & 31;
    AttnSeq q{};
    if (valid) q = attn_seq(p, b);
    const int nt = row_tiles(q, group);
    if (rows) *rows = nt;
    long long c = nt == 1 ? cost(p, q, group, 0) : 0;
    unsigned many = __ballot_sync(0xffffffffu, nt > 1);
    while (many) {
      const int src = __ffs((int)many) - 1;
      many &= many - 1;
      AttnSeq o;
      o.row0 = __shfl_sync(0xffffffffu, q.row0, src);
      o.n = __shfl_sync(0xffffffffu, q.n, src);
      o.len = __shfl_sync(0xffffffffu, q.len, src);
      o.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
      const int n = __shfl_sync(0xffffffffu, nt, src);
      long long sum = 0;
      for (int i = lane; i < n; i += 32) sum += cost(p, o, group, i);
      sum = attn_warp_sum(sum);
      if (lane == src) c = sum;
    }
    return c;
  }
};

// The cut, and where this block's run begins and ends.
struct AttnPlan {
  long long total;           // places of the line
  int runs;                  // blocks that have work
  long long base[2], per_head[2];  // of the sequences in which the run begins and ends: place, a head's places
  int b[2];
  long long begin, end;      // the run
  int h, i, skip;            // its first item (of sequence b[0]), and the places of it that belong to the run before
};

// The place x where an even cut would fall, moved to an item's end if that is less
// than SNAP places away: an item is cut only where both parts are worth the join.
template <int SNAP>
struct AttnCut {
  static __device__ __forceinline__ long long moved(long long x, long long begin, long long end) {
    return x - begin >= SNAP && end - x >= SNAP ? x : x - begin <= end - x ? begin : end;
  }
  // The runs that hold parts of the item begin .. end - 1: first, and how many.
  static __device__ __forceinline__ int parts(const AttnPlan& S, long long begin, long long end, int* first) {
    const long long lo = attn_div((begin + SNAP) * S.runs + S.total - 1, S.total);      // first cut inside
    const long long hi = attn_div((end - SNAP + 1) * S.runs + S.total - 1, S.total) - 1;  // last cut inside
    *first = (int)lo - 1;
    return (int)(hi - lo) + 2;
  }
};

// By all NT threads of the block; ends with a barrier.  scratch: two numbers a warp.
template <class W, int NT>
__device__ void attn_plan(const AttnParams& p, const AttnGroup& group, AttnPlan& S, long long (*scratch)[2],
                          unsigned* status) {
  using Cut = AttnCut<W::SNAP>;
  constexpr int NWARP = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int batch = p.s.batch, kh = p.c.kv.kv_heads;
  long long mine = 0, first = 0, items = 0;  // all of this thread's sequences; the first
  for (int b0 = 0; b0 < batch; b0 += NT) {
    int n = 0;
    if (blockIdx.x == 0 && b0 + tid < batch && p.s.kv_len[b0 + tid] > p.s.max_pages * p.c.kv.page_size)
      atomicOr(status, (unsigned)MOE_STATUS_BAD_PAGE);  // a length beyond the table
    const long long c = W::seq_cost(p, group, b0 + tid, b0 + tid < batch, &n) * kh;
    mine += c;
    items += (long long)n * kh;
    if (b0 == 0) first = c;
  }
  mine = attn_warp_sum(mine);
  items = attn_warp_sum(items);
  if (lane == 0) {
    scratch[warp][0] = mine;
    scratch[warp][1] = items;
  }
  __syncthreads();
  long long total = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NWARP; ++w) {
    total += scratch[w][0];
    all += scratch[w][1];
  }
  __syncthreads();
  long long most = total / W::MIN_RUN;
  // an item of T places in n parts takes T / n and then n joins: least where n^2 is T over the join's places
  if (total * W::JOIN > all * (100ll * W::MIN_RUN * W::MIN_RUN))
    most = attn_div(total, (long long)sqrtf((float)total / (float)all * (W::JOIN * 0.01f)));
  const int runs = (int)min((long long)gridDim.x, max(most, all));
  if (tid == 0) {
    S.total = total;
    S.runs = runs;
    S.begin = S.end = 0;
  }
  const int run = (int)blockIdx.x;
  if (run < runs) {
    // the items that the even cuts fall into: the run's first and the next run's
    const long long x[2] = {attn_div(total * run, runs), attn_div(total * (run + 1), runs)};
    long long base = 0;
    for (int b0 = 0; b0 < batch && base <= x[1]; b0 += NT) {
      const long long c = b0 == 0 ? first : W::seq_cost(p, group, b0 + tid, b0 + tid < batch) * kh;
      const long long s = attn_warp_scan(c);
      if (lane == 31) scratch[warp][0] = s;
      __syncthreads();
      long long before = base;
#pragma unroll
      for (int w = 0; w < NWARP; ++w) {
        if (w < warp) before += scratch[w][0];
        base += scratch[w][0];
      }
      __syncthreads();
      const long long at = before + s - c;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (at <= x[e] && x[e] < at + c) {
          S.b[e] = b0 + tid;
          S.base[e] = at;
          S.per_head[e] = attn_div(c, kh);
        }
    }
    __syncthreads();
    if (warp < 2) {
      const long long xe = warp ? x[1] : x[0];
      if (xe == total) {
        if (lane == 0) S.end = total;
      } else {
        const AttnSeq q = attn_seq(p, S.b[warp]);
        const int nt = W::row_tiles(q, group);
        long long rem = xe - S.base[warp];
        const int h = (int)attn_div(rem, S.per_head[warp]);
        rem -= h * S.per_head[warp];
        for (int i0 = 0; i0 < nt; i0 += 32) {
          const int i = i0 + lane;
          const long long c = i < nt ? W::cost(p, q, group, i) : 0;
          const long long s = attn_warp_scan(c);
          const unsigned past = __ballot_sync(0xffffffffu, rem < s);
          if (past) {
            if (lane == __ffs((int)past) - 1) {
              const long long begin = xe - (rem - (s - c)), to = Cut::moved(xe, begin, begin + c);
              if (warp == 0) {
                S.begin = to;
                S.h = h;
                S.i = i;
                S.skip = (int)(to - begin);
              } else {
                S.end = to;
              }
            }
            break;
          }
          rem -= __shfl_sync(0xffffffffu, s, 31);
        }
      }
    }
  }
  __syncthreads();
}

// The items of this block's run, one after the other; every warp that needs them
// walks for itself.
template <class W>
struct AttnWalk {
  static constexpr int R = W::R, TK = W::TK;
  const AttnParams& p;
  const AttnGroup& group;
  long long at, left;      // place of the item's part in the line; what is left of the run from there on
  int b, h, i, row_tiles;
  AttnSeq q;
  AttnRange keys;
  int tiles;               // key tiles of the item
  int skip, take;          // the part: its first place in the item and how many
  bool live;

  __device__ __forceinline__ AttnWalk(const AttnParams& p_, const AttnGroup& group_, const AttnPlan& S) : p(p_), group(group_) {
    at = S.begin;
    left = S.end - at;
    live = left > 0;
    if (!live) return;
    b = S.b[0];
    h = S.h;
    i = S.i;
    skip = S.skip;
    q = attn_seq(p, b);
    row_tiles = W::row_tiles(q, group);
    set();
    if (take == 0) next();  // the cut was moved to the item's end
  }
  __device__ __forceinline__ void set() {
    keys = W::range(p, q, group, i);
    tiles = W::key_tiles(keys);
    take = (int)min((long long)(cost() - skip), left);
  }
  __device__ __forceinline__ void next() {
    at += take;
    left -= take;
    if (left <= 0) {
      live = false;
      return;
    }
    skip = 0;
    if (++i == row_tiles) {
      i = 0;
      if (++h == p.c.kv.kv_heads) {
        h = 0;
        do {
          if (++b >= p.s.batch) {
            live = false;
            return;
          }
          q = attn_seq(p, b);
        } while (q.n == 0);
        row_tiles = W::row_tiles(q, group);
      }
    }
    set();
  }
  __device__ __forceinline__ int cost() const { return W::OVER + tiles; }
  __device__ __forceinline__ bool whole() const { return take == cost(); }
  // of the sequence's rows
  __device__ __forceinline__ int row0() const { return i * R; }
  __device__ __forceinline__ int rows() const { return min(R, q.n * group.n - i * R); }
  // key tiles of the part: a cut lies behind the item's first OVER places
  __device__ __forceinline__ int first_step() const { return skip ? skip - W::OVER : 0; }
  __device__ __forceinline__ int key_steps() const {
    return (skip + take == cost() ? tiles : skip + take - W::OVER) - first_step();
  }
  __device__ __forceinline__ int key0() const { return (keys.lo / TK + first_step()) * TK; }
  // places of the whole item
  __device__ __forceinline__ long long begin() const { return at - skip; }
  __device__ __forceinline__ long long end() const { return begin() + cost(); }
};

// Workspace of a call: status, and for each block two counters (of the item that
// begins in its run and ends behind it, one for each half of its rows) and two
// partial results (of an item that begins before its run, and of one that ends
// behind it).
struct AttnWs {
  size_t count, part, slot, total;  // byte offsets; bytes of a partial result
};
inline AttnWs attn_ws(const moe_v41_attn_cfg& c) {
  AttnWs w{};
  w.count = align256(sizeof(Ctrl));
  w.part = w.count + align256(ATTN_MAX_CTAS * 2 * 4);
  w.slot = (size_t)ATTN_TILES_TILE * (c.kv.head_dim + 2) * 4;
  w.total = align256(w.part + (size_t)ATTN_MAX_CTAS * 2 * w.slot);
  return w;
}

// What a kernel needs beside the call's parameters.
struct AttnArgs {
  CUtensorMap map_k, map_v;
  CUtensorMap map_q;       // kernel for many rows, with q_map
  AttnParams p;
  AttnGroup group;
  int page_shift, box_rows;
  float c;                 // scale log2 e
  unsigned* status;
  unsigned* count;         // [blocks][2]
  char* part;              // [blocks][2] of slot bytes each
  size_t slot;
  unsigned long long timeout_ns;
  bool q_map;              // a row tile's queries are one box: the group divides it
};
int launch_attn_rows(const AttnArgs& a, int ctas, cudaStream_t s);
int launch_attn_tiles(const AttnArgs& a, int ctas, bool* taken, cudaStream_t s);  // *taken: whether it was launched
__device__ __forceinline__ uint64_t* attn_bar(unsigned long long& b) { return reinterpret_cast<uint64_t*>(&b); }

// Bounded wait of a warp.  Once one ran out, the block's others give up as well, those under way and those to come.
__device__ __forceinline__ bool attn_wait_long(uint64_t* bar, uint32_t parity, volatile uint32_t* abort,
                                                   uint64_t timeout_ns, unsigned* status) {
  bool ok = false;
#pragma unroll 1
  for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
  if (!ok && !*abort) {
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
#pragma unroll 1
    do ok = mbar_try_wait_sleep(bar, parity, 20000u);
    while (!ok && !*abort && globaltimer_ns() < deadline);
    if (!ok) {
      atomicOr(status, (unsigned)MOE_STATUS_TIMEOUT);
      *abort = 1u;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool attn_wait(unsigned long long& bar, uint32_t parity, volatile uint32_t* abort,
                                          uint64_t timeout_ns, unsigned* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(attn_bar(bar), parity))) return true;
  return attn_wait_long(attn_bar(bar), parity, abort, timeout_ns, status);
}

template <bool BF>
__device__ __forceinline__ uint32_t attn_pack2(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The reference maximum of a row is moved only when the true one is more than this
// above it (in exponents of two), so that outputs are rescaled a few times an item;
// weights are at most 2^8.  For fp16 they are 2^6 times as large, so that those of
// 2^-31 of the largest still count.
constexpr float ATTN_SLACK = 8.0f;
template <bool BF>
constexpr float ATTN_BIAS = BF ? 0.f : 6.f;

// 2^x; 0 for -inf
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four values of a row, over n parts of its keys: part i has reference maximum and
// sum ml(i) and unscaled values o(i).
struct AttnJoined {
  float m, l;
  float4 o;
};
template <int U, class ML, class O>
__device__ __forceinline__ AttnJoined attn_join(int n, ML ml, O o) {
  AttnJoined j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
  for (int x0 = 0; x0 < n; x0 += U) {  // U parts on their way at once
    float2 v[U];
    float4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = min(x0 + i, n - 1);
      v[i] = ml(at);
      x[i] = o(at);
    }
    float top = j.m;
#pragma unroll
    for (int i = 0; i < U; ++i) top = fmaxf(top, v[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f0 = exp2_fast(j.m - ref);
    j.m = top;
    j.l *= f0;
    j.o.x *= f0;
    j.o.y *= f0;
    j.o.z *= f0;
    j.o.w *= f0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (x0 + i >= n || v[i].y == 0.f) continue;  // (0: nothing seen, its values may never have been written)
      const float f = exp2_fast(v[i].x - ref);
      j.l += f * v[i].y;
      j.o.x += f * x[i].x;
      j.o.y += f * x[i].y;
      j.o.z += f * x[i].z;
      j.o.w += f * x[i].w;
    }
  }
  return j;
}

// log sum exp of a row from its reference maximum and sum
template <bool BF>
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l) - ATTN_BIAS<BF>) * 0.69314718055994531f;
}

template <bool BF>
__device__ __forceinline__ void attn_store(const AttnArgs& a, int tok0, int h, int row, int d, const AttnJoined& j) {
  const int tok = a.group.token(row), hd = h * a.group.n + row - tok * a.group.n;
  const long long t = tok0 + tok;
  const float s = j.l == 0.f ? 0.f : 1.f / j.l;
  uint2 v;
  v.x = attn_pack2<BF>(j.o.x * s, j.o.y * s);
  v.y = attn_pack2<BF>(j.o.z * s, j.o.w * s);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.p.out) + t * a.p.ldo + (long long)hd * a.p.c.kv.head_dim + d) = v;
  if (d == 0 && a.p.lse) a.p.lse[t * a.p.ld_lse + hd] = attn_lse<BF>(j.m, j.l);
}

// Box {64 values, rows of a page, 1, 1} of the cache seen as [page][head][slot][value].
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int x, int slot, int head, int page,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Pages of a sequence, 64 at a time in two registers of a warp's lanes.
struct AttnPages {
  const int* row;
  int base, last, a, b;
  __device__ __forceinline__ int load(int i) const { return i <= last ? __ldg(row + i) : -1; }
  __device__ __forceinline__ void begin(const int* row_, int first, int last_) {
    row = row_;
    base = first;
    last = last_;
    a = load(base + (int)(threadIdx.x & 31));
    b = load(base + 32 + (int)(threadIdx.x & 31));
  }
  // from here on, pages from `first` on are asked for (at most 32 of them at once)
  __device__ __forceinline__ void advance(int first) {
    while (first - base >= 32) {
      a = b;
      base += 32;
      b = load(base + 32 + (int)(threadIdx.x & 31));
    }
  }
  // page i, by every lane for an i of its own
  __device__ __forceinline__ int at(int i) const {
    const int u = __shfl_sync(0xffffffffu, a, (i - base) & 31), v = __shfl_sync(0xffffffffu, b, (i - base) & 31);
    return i - base < 32 ? u : v;
  }
};

}  // namespace moe
