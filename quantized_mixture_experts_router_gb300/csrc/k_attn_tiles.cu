// Attention over a paged cache for many rows: chunks of prompts, whole prompts,
// several drafted tokens of many heads, cross attention.  Rows are tokens x the
// query heads that share a key head; an item is two tiles of 128 rows against
// tiles of 128 keys.
//   S = Q K^T,   P = exp2(c S - m),   O += P V   (tcgen05, f32 in tensor memory)
//
// Roles of a block (one an SM, persistent over its run of the line):
//   warps 0-3, 4-7   softmax of the first and second row tile, a row a thread: S out
//                    of tensor memory, maximum, P as 16-bit values over S, sum
//   warps 8, 9       issue the products of the first and second row tile
//   warp 10          walks through the run, tells the others its items, and copies keys
//                    (TMA boxes of a page's slots) into a ring
//   warp 11          copies queries, and values into a ring
// While one row tile is in its softmax the tensor cores work on the other.  A warp
// issues P V of a key tile and Q K of the next one behind another, as the second
// overwrites the P of the first.
// V lies in shared memory as it lies in the cache, [key][value], and is read as an
// operand whose values, not keys, are contiguous.  A row's output is rescaled only
// when its maximum has grown by more than 2^8 over the reference, which its own
// thread then does in place.
//
// Bound (times among calls of its kind in a graph) by the softmax between a tile's two
// products: at 2048 tokens over 10000 (32 heads over 8 key heads of 128, 301 GFLOP) 218 us,
// 1380 TFLOP/s, the tensor pipe busy 58% of the time; by bytes where the rows are few (five
// tokens of 16 sequences over 3000 to 7400: 79 us, 4.8 TB/s); where items are short by runs
// that come out uneven and by what an item takes beside its tiles, first copies, the end,
// joins (seven prompts of up to 2500: 105 us; the longest run has 56 places, an even share 46).
#include "attn_work.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int R = ATTN_TILES_TILE, TK = ATTN_TILES_KEYS, TR = 128;
constexpr int W_MMA = 8, W_K = 10, W_V = 11;
// An item costs about as much as three key tiles beside its own, and so does a join (with
// two or four, a window of 1000 took 59 and 55 us instead of 54).  Parts of a join cost
// half a tile each: 100 tokens over 30000 of two key heads, 69 us, 92 with as many runs
// as blocks; eight over 60000 of one, 52 and 66.
using Work = AttnWork<R, TK, 3, 6, 6, 50>;
using Walk = AttnWalk<Work>;
constexpr int NSOFT = 256, NTHR = 384;
// Registers a thread: 168 at launch; the softmax warps take what the others leave (200
// and 104 take the same time).
constexpr int REG_LAUNCH = 168, REG_SOFT = 184, REG_REST = 136;
static_assert(NSOFT * REG_SOFT + (NTHR - NSOFT) * REG_REST <= NTHR * REG_LAUNCH, "register shares exceed the launch's");
constexpr uint32_t HALF = TK * 128;  // 64 values of 128 keys or rows

template <int DH>
struct Cfg {
  static constexpr uint32_t SLOT = DH * HALF;   // keys or values of a tile; queries of a row tile
  // A key tile is done with once both row tiles' scores are, a value tile half a tile later.
  static constexpr int NK = DH == 2 ? 2 : 4, NV = DH == 2 ? 3 : 6;
  static constexpr int NS = NK + NV;
};

// One half of the softmax and issuing warps in this run's part of an item: one of
// its two row tiles, or, where there is but one, every other key tile of it.
struct Half {
  int row0, rows;       // of the item
  int lo, hi;           // keys that any of them sees
  int first, last;      // key tiles to go through, none if last < first
};
// An item as the warps need it.
struct Item {
  int number;           // of the run, from 1 on; 0: the run has ended, and nothing else is told
  int tok0, pos0, len;  // first row, its position, and the tokens of the sequence
  int row0;             // of the sequence's rows (tokens x heads of the group)
  int b, h;             // sequence, key head
  int lo, hi;           // keys that any row sees
  int from, steps;      // key tiles of the part
  int whole, slot;      // not cut; which partial result of the block otherwise
  int c0, n;            // the runs that hold its parts
  int split;            // one row tile
  Half half[2];
};
constexpr int NITEMS = 4;
// `told` counts the items that the walking warp has told, and the one that it will tell next.  Who waited too long,
// a reader for an item that is not among these or the walking warp for a reader, sets NO_MORE.  Then no other item
// is told, and as this is one word, all warps agree on the last: they meet at barriers within an item.
constexpr uint32_t NO_MORE = 0x80000000u;
constexpr int ITEM_READERS = NSOFT / 32 + 3;  // softmax, issuing and value warps

struct TilesCtl {
  unsigned long long full[10], empty[10], landed;
  unsigned long long i_full[NITEMS], i_empty[NITEMS];
  unsigned long long q_full[2], q_empty[2];     // queries of a row tile
  unsigned long long s_full[2], p_full[2];      // scores to the softmax; weights to the products
  unsigned long long o_full[2], o_free[2];      // an item's output, complete; read
  unsigned long long done[2];
  uint32_t tmem, abort, last[2], turn, told;
  Item items[NITEMS];
  alignas(16) float2 hand[TR];                              // (maximum, sum) of a row that the second half hands to the first
  AttnPlan plan;
};
template <int DH>
constexpr uint32_t SMEM_BYTES = (2 + Cfg<DH>::NS) * Cfg<DH>::SLOT + ((sizeof(TilesCtl) + 15) & ~15u);
static_assert(SMEM_BYTES<1> <= 232448 && SMEM_BYTES<2> <= 232448, "shared memory of a block");

struct Env {
  const AttnArgs& a;
  TilesCtl& C;
  __device__ __forceinline__ bool wait(unsigned long long& bar, uint32_t parity) const {
    return attn_wait(bar, parity, &C.abort, a.timeout_ns, a.status);
  }
};

// The items, one after the other, as a warp reads them.  They also come when a copy
// has not landed, so that every output is written.
struct Reader {
  const Env E;
  uint32_t n = 0;
  __device__ __forceinline__ explicit Reader(const Env& e) : E(e) {}
  __device__ __forceinline__ const Item& item() const { return E.C.items[n % NITEMS]; }
  // waits for the next, until it is told or it is certain that it will not be; whether there is one.  What lies in
  // a slot that was not told is another item's, or none.
  __device__ __forceinline__ bool get() {
    unsigned long long& bar = E.C.i_full[n % NITEMS];
    const uint32_t parity = (n / NITEMS) & 1u;
    if (!__all_sync(0xffffffffu, mbar_try_wait(attn_bar(bar), parity)))
      while (!__all_sync(0xffffffffu, mbar_wait_for(attn_bar(bar), parity, 4 * E.a.timeout_ns, E.a.status)))
        if (__shfl_sync(0xffffffffu, (int)none(), 0)) return false;
    return item().number == (int)n + 1;
  }
  // That there will be no item n.  One that is announced comes or is taken back, as the walking warp's own waits end;
  // so that the answer may change between the lanes, and the first one's counts.
  __device__ __forceinline__ bool none() const { return (atomicCAS(&E.C.told, n, n | NO_MORE) & ~NO_MORE) == n; }
  // has read it
  __device__ __forceinline__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(attn_bar(E.C.i_empty[n % NITEMS]));
    ++n;
  }
  __device__ __forceinline__ void skip_rest() {
    while (get()) done();
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void warp_arrive(unsigned long long& b) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(attn_bar(b));
}

// ------------------------------------------------------------ copies
// Key or value tiles into a ring of NS slots.
template <int DH, int NS>
struct Ring {
  const AttnArgs& a;
  const Env E;
  const CUtensorMap* map;
  const uint32_t smem;
  unsigned long long *full, *empty;
  const int br, box, half;
  uint32_t st = NS - 1, par = 0, used = 0;  // par: the phase of each slot's empty barrier that is waited for next
  AttnPages pages;

  __device__ __forceinline__ Ring(const AttnArgs& a_, TilesCtl& C, const CUtensorMap* map_, uint32_t smem_, int first)
      : a(a_), E{a_, C}, map(map_), smem(smem_), full(C.full + first), empty(C.empty + first), br(a_.box_rows),
        box((int)(threadIdx.x & 31) % (TK / a_.box_rows)), half((int)(threadIdx.x & 31) / (TK / a_.box_rows)) {}
  int lo, hi, h;  // of the item
  __device__ __forceinline__ void begin(const Item& it) {
    lo = it.lo;
    hi = it.hi;
    h = it.h;
    pages.begin(a.p.s.table + it.b * a.p.s.ld_table, max(it.from * TK, lo) >> a.page_shift, (hi - 1) >> a.page_shift);
  }
  // The boxes of the tile at `key`: whether this lane has one, of which page; all of them.
  bool mine;
  int id, slot0;
  uint32_t bytes;
  __device__ __forceinline__ void locate(int key) {
    const int k = key + box * br;
    mine = half < DH && k + br > lo && k < hi;
    slot0 = k & (a.p.c.kv.page_size - 1);
    pages.advance(max(key, lo) >> a.page_shift);
    id = pages.at(min(max(k, lo), hi - 1) >> a.page_shift);
    bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * (uint32_t)br * 128u;
    if (mine && (id < 0 || id >= a.p.c.kv.n_pages)) {
      atomicOr(a.status, (unsigned)MOE_STATUS_BAD_PAGE);
      id = a.p.c.kv.n_pages;  // outside: filled with zeros
    }
  }
  __device__ __forceinline__ bool next_slot() {
    st = st + 1 == NS ? 0 : st + 1;
    if ((used >> st) & 1u) {
      if (!E.wait(empty[st], (par >> st) & 1u)) return false;
      par ^= 1u << st;
    }
    used |= 1u << st;
    return true;
  }
  // The boxes into the slot; `bar` hears of them.
  __device__ __forceinline__ void copy(unsigned long long& bar) {
    if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(attn_bar(bar), bytes);
    __syncwarp();
    if (mine)
      tma_load_4d(smem + st * Cfg<DH>::SLOT + (uint32_t)half * HALF + (uint32_t)(box * br) * 128u, map, half * 64, slot0, h, id,
                  attn_bar(bar));
  }
  // Copies in flight land before the block can exit: each slot's last one (its full
  // barrier's phase flips with every use, as `par` does from the second use on).
  __device__ __forceinline__ void drain() {
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
#pragma unroll 1
    for (uint32_t i = 0; i < NS; ++i)
      if ((used >> i) & 1u) mbar_wait_bounded(attn_bar(full[i]), (par >> i) & 1u, deadline, a.status);
  }
};

// The walk's item, by a whole warp (each lane finds the same).
__device__ __forceinline__ Item describe(const AttnArgs& a, const AttnPlan& plan, const Walk& w, int number) {
  Item x{};
  if (!w.live) return x;
  x.number = number;
  x.tok0 = w.q.row0;
  x.pos0 = w.q.pos0;
  x.len = w.q.len;
  x.row0 = w.row0();
  x.b = w.b;
  x.h = w.h;
  x.lo = w.keys.lo;
  x.hi = w.keys.hi;
  x.from = w.key0() / TK;
  x.steps = w.key_steps();
  x.whole = w.whole();
  x.slot = w.skip ? 0 : 1;
  x.c0 = x.n = 0;
  if (!x.whole) x.n = AttnCut<Work::SNAP>::parts(plan, w.begin(), w.end(), &x.c0);
  x.split = w.rows() <= TR;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Half& t = x.half[s];
    t.row0 = x.split ? 0 : s * TR;
    t.rows = min(w.rows() - t.row0, TR);
    t.first = 0;
    t.last = -1;
    const AttnRange g = attn_range(a.p, w.q, a.group, x.row0 + t.row0, x.row0 + t.row0 + t.rows);
    t.lo = g.lo;
    t.hi = g.hi;
    if (g.hi <= g.lo) continue;
    t.first = max(g.lo / TK, x.from) + (x.split ? s : 0);
    t.last = min((g.hi - 1) / TK, x.from + x.steps - 1);
    if (x.split && ((t.last - t.first) & 1)) --t.last;
  }
  return x;
}

constexpr uint32_t NAN2 = 0x7fff7fffu;  // two NaNs, bf16 or fp16

// An item that is not told, by a whole warp: NaN, and its part counted all the same, so that the counters are ready
// for the next call.  (In rolled loops, as all code that is hardly run: the kernel's instructions fill their caches,
// and 10 KB more of them cost seven prompts 3%.)
__device__ __forceinline__ void lose(const AttnArgs& a, const Item& it) {
  const int lane = threadIdx.x & 31, D = a.p.c.kv.head_dim;
#pragma unroll 1
  for (int s = 0; s < (it.split ? 1 : 2); ++s) {
    const int first = s ? it.half[1].row0 : it.half[0].row0, end = first + (s ? it.half[1].rows : it.half[0].rows);
    if (!it.whole) {
      float* part = reinterpret_cast<float*>(a.part + (2 * (size_t)blockIdx.x + it.slot) * a.slot);
#pragma unroll 1
      for (int r = first + lane; r < end; r += 32) *reinterpret_cast<float2*>(part + 2 * r) = make_float2(0.f, NAN);
      __threadfence();
      __syncwarp();
      bool last = false;
      if (lane == 0) {
        unsigned* count = a.count + 2 * it.c0 + s;
        last = atomicAdd(count, 1u) == (unsigned)(it.n - 1);
        if (last) *count = 0u;
      }
      if (!__any_sync(0xffffffffu, last)) continue;  // (a part of NaN makes the whole of it)
    }
#pragma unroll 1
    for (int r = first + lane; r < end; r += 32) {
      const int row = it.row0 + r, tok = a.group.token(row), hd = it.h * a.group.n + row - tok * a.group.n;
      const long long t = it.tok0 + tok;
      uint16_t* out = static_cast<uint16_t*>(a.p.out) + t * a.p.ldo + (long long)hd * D;
#pragma unroll 1
      for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(out + d) = make_uint4(NAN2, NAN2, NAN2, NAN2);
      if (a.p.lse) a.p.lse[t * a.p.ld_lse + hd] = NAN;
    }
  }
}

template <int DH>
__device__ void run_k(const AttnArgs& a, TilesCtl& C, uint32_t ring) {
  Ring<DH, Cfg<DH>::NK> K(a, C, &a.map_k, ring, 0);
  bool ok = true;
  uint32_t n = 0;
  uint32_t was = 0;  // of `told`, when this item was announced (the first lane's)
  bool telling = true;
  for (Walk w(a.p, a.group, C.plan);; w.next()) {
    const bool lead = (threadIdx.x & 31) == 0;
    const uint32_t e = n % NITEMS;
    if (telling) {
      telling = __all_sync(0xffffffffu, !lead || was == n);  // not if a reader gave up before
      if (telling && n >= NITEMS) {
        telling = __all_sync(0xffffffffu, mbar_wait_for(attn_bar(C.i_empty[e]), (n / NITEMS - 1) & 1u, 4 * a.timeout_ns, a.status));
        if (!telling && lead) atomicExch(&C.told, n | NO_MORE);
      }
    }
    const Item x = describe(a, C.plan, w, (int)n + 1);
    if (!telling) {
      if (!w.live) break;
      lose(a, x);
      continue;
    }
    if (lead) {
      C.items[e] = x;
      mbar_arrive(attn_bar(C.i_full[e]));
    }
    __syncwarp();
    ++n;
    if (!w.live) break;
    if (lead) was = atomicCAS(&C.told, n, n + 1);  // announces the next; the answer comes while keys are copied
    const int steps = w.key_steps();
    if (!steps || !ok) continue;
    const Item& it = C.items[e];  // stays until this warp overwrites it
    K.begin(it);
    const int from = w.key0();
    for (int j = 0; ok && j < steps; ++j) {
      K.locate(from + j * TK);
      ok = K.next_slot();
      if (ok) K.copy(K.full[K.st]);
    }
  }
  K.drain();
}

// A row tile's queries into the swizzled layout; `full` hears of them.  By boxes of
// [tokens][heads of the group] where these make a row tile: rows that there are none
// of then hold what comes next in memory, or zeros, which concerns nobody.  Else
// piece by piece, rows and values that there are none of as zeros.
template <int DH>
__device__ __forceinline__ void copy_q(const AttnArgs& a, const Item& it, int s, uint32_t q_smem, unsigned long long& full) {
  const int lane = threadIdx.x & 31, D = a.p.c.kv.head_dim, first = it.row0 + it.half[s].row0, rows = it.half[s].rows;
  if (a.q_map) {
    if (lane == 0) {
      mbar_arrive_expect_tx(attn_bar(full), Cfg<DH>::SLOT);
      const int tok = it.tok0 + a.group.token(first);
#pragma unroll
      for (int half = 0; half < DH; ++half)
        tma_load_3d(q_smem + half * HALF, &a.map_q, half * 64, it.h * a.group.n, tok, attn_bar(full));
    }
    __syncwarp();
    return;
  }
  constexpr int CH = DH * 8;         // 16-byte pieces of a row
  constexpr int RPI = 32 / CH;       // rows an instruction of the warp covers
  const int ch = lane % CH, rr = lane / CH;
  const bool in = ch * 8 < D;
  const uint16_t* q = static_cast<const uint16_t*>(a.p.q);
#pragma unroll 1
  for (int r0 = 0; r0 < TR; r0 += 32) {
    // each lane finds one of 32 rows
    const int r = r0 + lane, row = first + r, tok = a.group.token(row);
    const long long at = (it.tok0 + tok) * a.p.ldq + (long long)(it.h * a.group.n + row - tok * a.group.n) * D;
    const long long off = r < rows ? at : -1;
#pragma unroll 4
    for (int i = 0; i < 32; i += RPI) {
      const long long o = __shfl_sync(0xffffffffu, off, i + rr);
      const bool there = o >= 0 && in;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       q_smem + (uint32_t)(ch / 8) * HALF + swz(r0 + i + rr, ch & 7)),
                   "l"(there ? q + o + ch * 8 : q), "r"(there ? 16 : 0)
                   : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(attn_bar(full));
}

// Value slots of the tile at key0 that the item's rows do not see, in steps of 16
// that hold some that they see: zeros, whatever the pages hold there.
struct Edge {
  int from[2], to[2];
  __device__ __forceinline__ Edge(int key0, int lo, int hi) {
    to[0] = lo - key0;
    from[0] = to[0] & ~15;
    from[1] = hi - key0;
    to[1] = (from[1] + 15) & ~15;
  }
  __device__ __forceinline__ bool has(int side) const { return from[side] >= 0 && to[side] <= TK && from[side] < to[side]; }
  template <int DH>
  __device__ __forceinline__ void clear(uint8_t* slot) const {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      if (!has(side)) continue;
      const int n = (to[side] - from[side]) * 8;  // 16-byte pieces of 64 values
      for (int i = threadIdx.x & 31; i < n * DH; i += 32) {
        const int half = i / n, c = i - half * n;
        *reinterpret_cast<uint4*>(slot + half * HALF + from[side] * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    fence_async_smem();
    __syncwarp();
  }
};

template <int DH>
__device__ void run_qv(const AttnArgs& a, TilesCtl& C, uint32_t q_smem, uint8_t* ring) {
  const Env E{a, C};
  Ring<DH, Cfg<DH>::NV> V(a, C, &a.map_v, smem_u32(ring), Cfg<DH>::NK);
  const int lane = threadIdx.x & 31;
  uint32_t uses[2] = {}, edges = 0;
  bool ok = true, flying = false;  // flying: a copy that `landed` was to hear of
  Reader items(E);
  for (; items.get(); items.done()) {
    const Item& it = items.item();
    if (!it.steps || !ok) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (!ok || it.half[s].last < it.half[s].first) continue;
      ok = E.wait(C.q_empty[s], (uses[s] & 1u) ^ 1u);  // passes at once the first time
      if (!ok) continue;
      ++uses[s];
      copy_q<DH>(a, it, s, q_smem + (uint32_t)s * Cfg<DH>::SLOT, C.q_full[s]);
    }
    V.begin(it);
    for (int j = 0; ok && j < it.steps; ++j) {
      const int key = (it.from + j) * TK;
      V.locate(key);
      ok = V.next_slot();
      if (!ok) break;
      const Edge e(key, it.lo, it.hi);
      if (!e.has(0) && !e.has(1)) {
        V.copy(V.full[V.st]);
        continue;
      }
      V.copy(C.landed);
      ok = E.wait(C.landed, edges++ & 1u);
      if (!ok) {
        flying = true;
        V.used &= ~(1u << V.st);
        break;
      }
      e.clear<DH>(ring + V.st * Cfg<DH>::SLOT);
      if (lane == 0) mbar_arrive(attn_bar(V.full[V.st]));
    }
  }
  V.drain();
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (uses[s]) mbar_wait_bounded(attn_bar(C.q_full[s]), (uses[s] - 1) & 1u, globaltimer_ns() + a.timeout_ns, a.status);
  if (flying) mbar_wait_bounded(attn_bar(C.landed), (edges - 1) & 1u, globaltimer_ns() + a.timeout_ns, a.status);
}

// ------------------------------------------------------------ products
// Instructions of the issuing warp count: with 100 cycles a product, which generic
// code takes, they bound the kernel at half its rate.  So descriptors are built from
// warp-uniform words, whose offsets are constants of unrolled code.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Lower and upper word of a matrix descriptor (128-byte swizzle).  Rows of 128 bytes,
// eight of them 1024 bytes.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
// K and Q: 64 values of a key or row are one swizzled row, and what is summed over.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
// V as the second operand of P V: 64 values of a key are one swizzled row, keys follow
// one another; the values, not the keys (which are summed over), are contiguous.  The
// next 64 values are HALF on.
__device__ __forceinline__ uint32_t desc_v_lo(uint32_t saddr) { return (saddr >> 4) | ((HALF >> 4) << 16); }

__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)DESC_HI << 32) | lo; }

// scores = Q K^T over KS steps of 16 values
template <int KS>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t q, uint32_t k, uint32_t id) {
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const uint32_t off = (uint32_t)(i / 4) * (HALF >> 4) + (uint32_t)(i & 3) * 2u;
    umma_f16(d, desc(q + off), desc(k + off), id, i > 0);
  }
}

// The key tiles of all items of the run, and what one half does with each.
struct Steps {
  Reader items;
  const int s;
  int k, end, lo, hi, first, last, split;
  bool live;
  __device__ __forceinline__ Steps(const Env& E, int s_) : items(E), s(s_) { item(); }
  __device__ __forceinline__ void item() {
    while (true) {
      live = items.get();
      if (!live) return;
      const Item& it = items.item();
      const int steps = it.steps;
      k = it.from;
      end = k + steps;
      lo = it.half[s].lo;
      hi = it.half[s].hi;
      first = it.half[s].first;
      last = it.half[s].last;
      split = it.split;
      items.done();
      if (steps) return;
    }
  }
  __device__ __forceinline__ void next() {
    if (++k == end) item();
  }
};

// Weights against a value tile, in steps of 16 keys that any row sees.
struct Product {
  int from, to;
  bool active, first, last;
  __device__ __forceinline__ explicit Product(const Steps& t) {
    const int key0 = t.k * TK;
    active = t.k >= t.first && t.k <= t.last && !(t.split && ((t.k - t.first) & 1));
    first = t.k == t.first;
    last = t.k == t.last;
    from = max(t.lo - key0, 0) / 16;
    to = (min(t.hi - key0, TK) + 15) / 16;
  }
};

// The tensor cores take the products of both issuing warps in turn.  Held while one
// row tile's are issued, so that they do not mix with the other's: mixed, both tiles'
// scores come at the end of all of them and both softmaxes run while the tensor
// cores have nothing (2048 tokens over 10000: 294 us, 264 with the turn when it was
// added).  Only the order depends on it, so that a warp goes ahead without it rather
// than wait for long.
__device__ __forceinline__ void turn_begin(uint32_t turn) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i) {
    uint32_t was;
    asm volatile("atom.shared.cas.b32 %0, [%1], 0, 1;" : "=r"(was) : "r"(turn) : "memory");
    if (was == 0u) return;
  }
}
__device__ __forceinline__ void turn_end(uint32_t turn) { asm volatile("st.shared.u32 [%0], 0;" ::"r"(turn) : "memory"); }

// Every slot is waited for and given back, also where this row tile has no use for
// it: a wait that left one out could take the phase before for done.
template <int DH, bool BF, int S>
__device__ __forceinline__ void run_products(const AttnArgs& a, TilesCtl& C, Steps& t, uint32_t tmem_, uint32_t ring_,
                                             uint32_t q_) {
  constexpr int NK = Cfg<DH>::NK, NV = Cfg<DH>::NV;
  const Env E{a, C};
  const uint32_t tmem = uniform(tmem_), ring = uniform(ring_), q = uniform(desc_lo(q_ + S * Cfg<DH>::SLOT));
  const uint32_t id_qk = umma_idesc(TK, BF), id_pv = umma_idesc((a.p.c.kv.head_dim + 15) & ~15, BF) | (1u << 16);
  const uint32_t turn = smem_u32(&C.turn);
  const uint32_t sp = tmem + S * 128u, o = tmem + 256u + S * (DH * 64);
  const int ksteps = (a.p.c.kv.head_dim + 15) / 16 + (DH == 2 ? 0 : 4);
  uint32_t ks = 0, vs = 0, par = 0;             // slots; the phase of each
  uint32_t uq = 0, up = 0, uo = 0;              // uses of the barriers
  auto full = [&](uint32_t slot) {
    if (!E.wait(C.full[slot], (par >> slot) & 1u)) return false;
    par ^= 1u << slot;
    return true;
  };
  auto scores = [&](uint32_t k, const Product& P) {  // by the elected thread
    switch (ksteps) {
      case 8: issue_scores<DH * 4>(sp, q, k, id_qk); break;
      case 7: issue_scores<DH * 4 - 1>(sp, q, k, id_qk); break;
      case 6: issue_scores<DH * 4 - 2>(sp, q, k, id_qk); break;
      default: issue_scores<DH * 4 - 3>(sp, q, k, id_qk);
    }
    umma_commit(attn_bar(C.s_full[S]));
    if (P.last) umma_commit(attn_bar(C.q_empty[S]));
  };
  if (!t.live) return;
  Product P(t);
  if (!full(0)) return;
  if (P.active) {
    if (!E.wait(C.q_full[S], uq++ & 1u)) return;
    tc_fence_after();
    const uint32_t k = uniform(desc_lo(ring));
    if (elect_one()) {
      scores(k, P);
      umma_commit(attn_bar(C.empty[0]));
    }
  } else if (elect_one()) {
    mbar_arrive(attn_bar(C.empty[0]));
  }
  __syncwarp();
  while (true) {
    t.next();
    const Product N(t);
    const bool more = t.live;
    ks = ks + 1 == NK ? 0 : ks + 1;
    if (more && !full(ks)) return;
    if (!full(NK + vs)) return;
    const uint32_t k = uniform(desc_lo(ring + ks * Cfg<DH>::SLOT)), v = uniform(desc_v_lo(ring + (NK + vs) * Cfg<DH>::SLOT));
    const bool straight = more && P.active && N.active && !N.first;  // the next scores of the same queries
    if (P.active) {
      if (P.first && !E.wait(C.o_free[S], (uo++ & 1u) ^ 1u)) return;  // passes at once the first time
      if (!E.wait(C.p_full[S], up++ & 1u)) return;
      tc_fence_after();
      if (elect_one()) {
        turn_begin(turn);
        if (P.from == 0 && P.to == TK / 16) {
          umma_f16_ta(o, sp, desc(v), id_pv, P.first ? 0u : 1u);
#pragma unroll
          for (int i = 1; i < TK / 16; ++i)
            umma_f16_ta(o, sp + (uint32_t)i * 8u, desc(v + (uint32_t)i * (2048u >> 4)), id_pv, 1u);
        } else {
#pragma unroll 1
          for (int i = P.from; i < P.to; ++i)
            umma_f16_ta(o, sp + (uint32_t)i * 8u, desc(v + (uint32_t)i * (2048u >> 4)), id_pv, !(P.first && i == P.from));
        }
        if (P.last) umma_commit(attn_bar(C.o_full[S]));
        if (straight) {
          scores(k, N);
          umma_commit(attn_bar(C.empty[ks]));
        }
        umma_commit(attn_bar(C.empty[NK + vs]));
        turn_end(turn);
      }
    } else if (elect_one()) {
      mbar_arrive(attn_bar(C.empty[NK + vs]));
    }
    __syncwarp();
    if (!more) return;
    if (!straight) {
      if (N.active) {
        if (N.first && !E.wait(C.q_full[S], uq++ & 1u)) return;
        tc_fence_after();
        if (elect_one()) {
          scores(k, N);
          umma_commit(attn_bar(C.empty[ks]));
        }
      } else if (elect_one()) {
        mbar_arrive(attn_bar(C.empty[ks]));
      }
      __syncwarp();
    }
    vs = vs + 1 == NV ? 0 : vs + 1;
    P = N;
  }
}

// ------------------------------------------------------------ softmax
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The loads so far are complete.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Two f32 at once.
__device__ __forceinline__ uint64_t pack_f32(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ void unpack_f32(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void tmem_ld16_later(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The scores at ts, 16 at a time, each time the next 16 on their way.  How far the loop
// is unrolled decides: beyond 32 scores the warps' instructions come from farther away
// than they are used (a prompt's chunk, 2048 tokens over 10000: 262 us with 16 scores a
// turn, 256 with 32, 250 with 64; seven prompts of up to 2500: 108, 108, 116 us).
template <class F>
__device__ __forceinline__ void each_16(uint32_t ts, F use) {
  uint32_t a[16], b[16];
  tmem_ld16_later(ts, a);
#pragma unroll 1
  for (int i = 0; i < TK; i += 32) {
    tmem_wait_ld();
    tmem_ld16_later(ts + (uint32_t)i + 16u, b);
    use(a, i);
    tmem_wait_ld();
    tmem_ld16_later(ts + ((uint32_t)i + 32u) % TK, a);  // the last time for nothing, but without a branch
    use(b, i + 16);
  }
  tmem_wait_ld();
}

// The largest of this thread's row's scores, times c.
__device__ __forceinline__ float largest(uint32_t ts, float c) {
  uint32_t v[64];
  float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int i = 0; i < TK; i += 64) {
    tmem_ld32(ts + (uint32_t)i, v);
    tmem_ld32(ts + (uint32_t)i + 32u, v + 32);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 64; j += 2) t[(j / 2) & 3] = fmaxf(fmaxf(t[(j / 2) & 3], __uint_as_float(v[j])), __uint_as_float(v[j + 1]));
  }
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c;
}

// exp2(c s - ref) of 16 scores, packed, to the columns ts .. ts + 7; added to the sums.
template <bool BF>
__device__ __forceinline__ void weigh_16(const uint32_t (&v)[16], uint32_t ts, float c, float ref, uint64_t (&sum)[2]) {
  const uint64_t c2 = pack_f32(c, c), ref2 = pack_f32(-ref, -ref);
  uint32_t p[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float x, y;
    unpack_f32(fma2(pack_f32(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), c2, ref2), x, y);
    x = exp2_fast(x);
    y = exp2_fast(y);
    sum[j & 1] = add2(sum[j & 1], pack_f32(x, y));
    p[j] = attn_pack2<BF>(x, y);
  }
  tmem_st8(ts, p);
}
__device__ __forceinline__ float total(const uint64_t (&sum)[2]) {
  float x, y;
  unpack_f32(add2(sum[0], sum[1]), x, y);
  return x + y;
}

// Scores of keys outside from .. end - 1 become -inf, where the warp's rows do not see
// all 16 of some: a pass of its own over the few columns that need it, so that every tile
// runs through the same instructions (seven prompts: 109 us; with masks in both passes,
// whose instructions are rarer and come from farther away, 122).
__device__ __forceinline__ void hide(uint32_t ts, int from, int end) {
#pragma unroll 1
  for (int i = 0; i < TK; i += 16) {
    if (!__any_sync(0xffffffffu, from > i || end < i + 16)) continue;
    // bit j: score i + j is seen
    const uint32_t lo = (uint32_t)min(max(from - i, 0), 16), hi = (uint32_t)min(max(end - i, 0), 16);
    const uint32_t seen = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    uint32_t v[16];
    if (__any_sync(0xffffffffu, seen)) {
      tmem_ld16_later(ts + (uint32_t)i, v);
      tmem_wait_ld();
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (!(seen >> j & 1u)) v[j] = 0xff800000u;
    tmem_st8(ts + (uint32_t)i, v);
    tmem_st8(ts + (uint32_t)i + 8u, v + 8);
  }
  tmem_wait_st();
}

// One key tile of this thread's row.
template <int DH, bool BF>
__device__ __forceinline__ void soft_tile(uint32_t ts, uint32_t to, int key0, int lo, int hi, float c, bool first, float& m,
                                          float& l) {
  const int from = lo - key0, end = hi - key0;  // of the tile's keys, what the row sees
  if (__any_sync(0xffffffffu, from > 0 || end < TK)) hide(ts, from, end);
  const float top = largest(ts, c);
  const bool rise = top > m + ATTN_SLACK;  // from -inf: by anything
  if (first) {
    m = top;
  } else if (__any_sync(0xffffffffu, rise)) {
    const float next = rise ? top : m, f = rise ? exp2_fast(m - next) : 1.f;
    m = next;
    l *= f;
#pragma unroll 1
    for (int i = 0; i < DH * 4; ++i) {
      uint32_t o[16];
      tmem_ld16_later(to + 16u * i, o);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st8(to + 16u * i, o);
      tmem_st8(to + 16u * i + 8u, o + 8);
    }
  }
  const float ref = (m == -INFINITY ? 0.f : m) - ATTN_BIAS<BF>;
  uint64_t sum[2] = {0, 0};
  each_16(ts, [&](uint32_t (&v)[16], int i) { weigh_16<BF>(v, ts + (uint32_t)i / 2u, c, ref, sum); });
  l += total(sum);
  tmem_wait_st();
}

// A partial result: (maximum, sum) of 256 rows, then their values, four of all rows
// after four of all rows, so that the threads of a warp write and read side by side.
__device__ __forceinline__ float4* part_values(float* part, int row, int d) {
  return reinterpret_cast<float4*>(part + 2 * R) + (d / 4) * R + row;
}

// 32 values of a row from value c0 on, times inv (a row that saw nothing, or scores of
// -inf alone: zeros).
template <bool BF>
__device__ __forceinline__ void store_32(uint16_t* out, int c0, int D, const float (&f)[32], float inv) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* g = f + 8 * i;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (inv != 0.f) {
      x.x = attn_pack2<BF>(g[0] * inv, g[1] * inv);
      x.y = attn_pack2<BF>(g[2] * inv, g[3] * inv);
      x.z = attn_pack2<BF>(g[4] * inv, g[5] * inv);
      x.w = attn_pack2<BF>(g[6] * inv, g[7] * inv);
    }
    if (c0 + 8 * i < D) *reinterpret_cast<uint4*>(out + c0 + 8 * i) = x;
  }
}

// Joins the n parts of a row tile that runs c0 .. c0 + n - 1 have left: a row's values
// first .. first + 31, and every `step` on.
// It takes what its rounds of loads that wait for one another take: maxima, sums and
// values of two parts are on their way at once.
template <bool BF>
__device__ __forceinline__ void join_row(const AttnArgs& a, int c0, int n, int row, int first, int step, uint16_t* out,
                                         float* lse) {
  const int D = a.p.c.kv.head_dim;
  auto part = [&](int x) { return reinterpret_cast<float*>(a.part + (2 * (size_t)(c0 + x) + (x ? 0 : 1)) * a.slot); };
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int d0 = first; d0 < D; d0 += step) {
    float acc[32] = {};
    m = -INFINITY;
    l = 0.f;
#pragma unroll 1
    for (int x0 = 0; x0 < n; x0 += 2) {
      float2 y[2];
      float4 v[2][8];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool is = x0 + x < n;
        float* at = part(is ? x0 + x : x0);
        y[x] = is ? __ldcg(reinterpret_cast<const float2*>(at) + row) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[x][i] = is && d0 + 4 * i < D ? __ldcg(part_values(at, row, d0 + 4 * i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const float top = fmaxf(m, fmaxf(y[0].x, y[1].x)), ref = top == -INFINITY ? 0.f : top;
      const float w = exp2_fast(m - ref);
      m = top;
      l *= w;
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] *= w;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float f = y[x].y == 0.f ? 0.f : exp2_fast(y[x].x - ref);  // (0: nothing seen)
        l += f * y[x].y;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[4 * i] = fmaf(f, v[x][i].x, acc[4 * i]);
          acc[4 * i + 1] = fmaf(f, v[x][i].y, acc[4 * i + 1]);
          acc[4 * i + 2] = fmaf(f, v[x][i].z, acc[4 * i + 2]);
          acc[4 * i + 3] = fmaf(f, v[x][i].w, acc[4 * i + 3]);
        }
      }
    }
    store_32<BF>(out, d0, D, acc, l == 0.f ? 0.f : 1.f / l);
  }
  if (lse) *lse = attn_lse<BF>(m, l);
}

template <int DH, bool BF>
__device__ void run_softmax(const AttnArgs& a, TilesCtl& C, uint32_t tmem, int s) {
  const Env E{a, C};
  const int r = threadIdx.x & 127, D = a.p.c.kv.head_dim;  // row of the row tile
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t ts = tmem + lanes + (uint32_t)s * 128u, to = tmem + lanes + 256u + (uint32_t)(s * DH * 64);
  uint32_t us = 0, uo = 0;  // uses of s_full and o_full
  bool ok = true;
  Reader items(E);
  for (; items.get(); items.done()) {
    const Item& it = items.item();
    const Half& t = it.half[s];
    const int step = it.split ? 2 : 1, first = t.first, last = t.last;
    int lo = 0, hi = INT_MAX;  // what the row sees
    if (r < t.rows) {
      const int row = it.row0 + t.row0 + r;  // of the sequence
      const AttnRange g = attn_range(a.p, AttnSeq{0, 0, it.len, it.pos0}, a.group, row, row + 1);
      lo = g.lo;
      hi = g.hi;
    }
    const bool some = first <= last;
    float m = -INFINITY, l = 0.f;
    for (int k = first; k <= last; k += step) {
      ok = ok && E.wait(C.s_full[s], us++ & 1u);
      if (!ok) break;
      tc_fence_after();
      soft_tile<DH, BF>(ts, to, k * TK, lo, hi, a.c, k == first, m, l);
      warp_arrive(C.p_full[s]);
    }
    if (some) {
      ok = ok && E.wait(C.o_full[s], uo++ & 1u);
      tc_fence_after();
    }
    if (!ok) l = NAN;
    // With one row tile the second half hands what it has to the first.
    float f0 = 1.f, f1 = 0.f;
    bool other = false;
    if (it.split) {
      if (s == 1) {
        C.hand[r] = make_float2(m, l);
        tc_fence_before();
      }
      named_bar_sync(3, NSOFT);
      float m1 = 0.f, l1 = 0.f;
      if (s == 0) {
        m1 = C.hand[r].x;
        l1 = C.hand[r].y;
        tc_fence_after();
      }
      named_bar_sync(3, NSOFT);
      if (s == 1) continue;
      other = it.half[1].first <= it.half[1].last;
      const float top = fmaxf(m, m1), ref = top == -INFINITY ? 0.f : top;
      f0 = l == 0.f ? 0.f : exp2_fast(m - ref);
      f1 = l1 == 0.f ? 0.f : exp2_fast(m1 - ref);
      l = f0 * l + f1 * l1;
      m = top;
    }
    const bool there = r < t.rows, whole = it.whole;
    float* part = reinterpret_cast<float*>(a.part + (2 * (size_t)blockIdx.x + it.slot) * a.slot);
    const int pr = t.row0 + r;
    // where a row of the item goes
    struct Place {
      uint16_t* out;
      float* lse;
    };
    auto place = [&](int at) {
      const int row = it.row0 + at, tok = a.group.token(row), hd = it.h * a.group.n + row - tok * a.group.n;
      return Place{static_cast<uint16_t*>(a.p.out) + (it.tok0 + tok) * a.p.ldo + (long long)hd * D,
                   a.p.lse ? a.p.lse + (it.tok0 + tok) * a.p.ld_lse + hd : nullptr};
    };
    const Place mine = place(pr);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t o[32];
      float f[32];
      if (some) {
        tmem_ld32(to + (uint32_t)c0, o);
        tmem_wait_ld();
      }
      const bool zero = !some || f0 == 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] = zero ? 0.f : f0 * __uint_as_float(o[j]);
      if (other) {
        tmem_ld32(to + (uint32_t)(c0 + DH * 64), o);
        tmem_wait_ld();
        if (f1 != 0.f) {
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] += f1 * __uint_as_float(o[j]);
        }
      }
      if (!ok) {
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = NAN;
      }
      if (there && whole) {
        store_32<BF>(mine.out, c0, D, f, inv);
      } else if (there) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          if (c0 + j < D) *part_values(part, pr, c0 + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
      }
      __syncwarp();
    }
    if (some) warp_arrive(C.o_free[s]);
    if (other) warp_arrive(C.o_free[1]);
    if (there) {
      if (!whole) *reinterpret_cast<float2*>(part + 2 * pr) = make_float2(m, l);
      else if (mine.lse) *mine.lse = attn_lse<BF>(m, l);
    }
    if (!whole) {
      named_bar_sync(1 + s, TR);
      if (r == 0) {
        __threadfence();
        unsigned* count = a.count + 2 * it.c0 + s;
        const bool last = atomicAdd(count, 1u) == (unsigned)(it.n - 1);
        if (last) *count = 0u;
        C.last[s] = last;
      }
      named_bar_sync(1 + s, TR);
      if (C.last[s]) {
        __threadfence();
        // where the rows are but one or two warps', the others take their share of the values
        const int warps = (t.rows + 31) / 32, shares = 4 / warps, share = (r >> 5) / warps;
        const int at = (r >> 5) % warps * 32 + (r & 31);
        if (at < t.rows && share < shares) {
          const Place to = place(t.row0 + at);
          join_row<BF>(a, it.c0, it.n, t.row0 + at, share * 32, shares * 32, to.out, share ? nullptr : to.lse);
        }
      }
      named_bar_sync(1 + s, TR);  // `last` has been read
    }
  }
}

template <int DH, bool BF>
__global__ void __launch_bounds__(NTHR, 1) k_attn_tiles(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  uint8_t* sm = raw_smem;  // on its 1024 bytes: there is no room to move it
  uint8_t* ring = sm + 2 * Cfg<DH>::SLOT;
  TilesCtl& C = *reinterpret_cast<TilesCtl*>(ring + Cfg<DH>::NS * Cfg<DH>::SLOT);
  const int warp = threadIdx.x >> 5;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg<DH>::NS; ++i) {
      mbar_init(attn_bar(C.full[i]), 1);
      mbar_init(attn_bar(C.empty[i]), 2);  // both row tiles
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(attn_bar(C.q_full[i]), 1);
      mbar_init(attn_bar(C.q_empty[i]), 1);
      mbar_init(attn_bar(C.s_full[i]), 1);
      mbar_init(attn_bar(C.p_full[i]), 4);
      mbar_init(attn_bar(C.o_full[i]), 1);
      mbar_init(attn_bar(C.o_free[i]), 4);
      mbar_init(attn_bar(C.done[i]), 1);
    }
    mbar_init(attn_bar(C.landed), 1);
    for (int i = 0; i < NITEMS; ++i) {
      mbar_init(attn_bar(C.i_full[i]), 1);
      mbar_init(attn_bar(C.i_empty[i]), ITEM_READERS);
      C.items[i].number = 0;
    }
    C.abort = C.turn = 0u;
    C.told = 1u;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&C.tmem, 512);
  grid_wait();
  attn_plan<Work, NTHR>(a.p, a.group, C.plan, reinterpret_cast<long long(*)[2]>(C.hand), a.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;

  if (warp < NSOFT / 32) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFT));
    run_softmax<DH, BF>(a, C, tmem, warp >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_REST));
    if (warp == W_K) {
      run_k<DH>(a, C, smem_u32(ring));
    } else if (warp == W_V) {
      run_qv<DH>(a, C, smem_u32(sm), ring + Cfg<DH>::NK * Cfg<DH>::SLOT);
    } else {
      Steps t(Env{a, C}, warp - W_MMA);
      if (warp == W_MMA) run_products<DH, BF, 0>(a, C, t, tmem, smem_u32(ring), smem_u32(sm));
      else run_products<DH, BF, 1>(a, C, t, tmem, smem_u32(ring), smem_u32(sm));
      if (t.live) t.items.skip_rest();  // a wait ran out
      __syncwarp();
      if (elect_one()) umma_commit(attn_bar(C.done[warp - W_MMA]));  // after every product of this thread
    }
  }
  __syncwarp();
  // no product may still be writing tensor memory when it is freed
  if (threadIdx.x < 2)
    mbar_wait_bounded(attn_bar(C.done[threadIdx.x]), 0u, globaltimer_ns() + a.timeout_ns, a.status);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DH, bool BF>
int launch(const AttnArgs& a, int ctas, bool* taken, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const auto kernel = k_attn_tiles<DH, BF>;
  static PerDevice allocated;  // registers a thread
  const int regs = allocated.get(dev, [&] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, kernel) == cudaSuccess &&
                   cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES<DH>) == cudaSuccess
               ? fa.numRegs
               : 0;
  });
  if (regs < 1) return MOE_ERR_CUDA;
  // The register trade waits until the launch holds what the shares add up to: a
  // compiler that chose another number leaves the call to the kernel for few rows.
  *taken = regs == REG_LAUNCH;
  if (!*taken) return MOE_OK;
  return launch_overlapped(kernel, dim3((unsigned)ctas), dim3(NTHR), SMEM_BYTES<DH>, s, a);
}

}  // namespace

int launch_attn_tiles(const AttnArgs& a, int ctas, bool* taken, cudaStream_t s) {
  const bool bf = a.p.c.kv.type == MOE_T_BF16;
  if (a.p.c.kv.head_dim > 64) return bf ? launch<2, true>(a, ctas, taken, s) : launch<2, false>(a, ctas, taken, s);
  return bf ? launch<1, true>(a, ctas, taken, s) : launch<1, false>(a, ctas, taken, s);
}

}  // namespace moe
