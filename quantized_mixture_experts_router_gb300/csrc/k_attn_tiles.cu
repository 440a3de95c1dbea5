// Attention over a paged cache for many rows: chunks of prompts, whole prompts,
// several drafted tokens of many heads, cross attention.  Rows are tokens x the
// query heads that share a key head; an item is two tiles of 128 rows against
// tiles of 128 keys.
//   S = Q K^T,   P = exp2(c S - m),   O += P V   (tcgen05, f32 in tensor memory)
//
// Roles of a block (one an SM, persistent over its run of key tiles):
//   warps 0-3, 4-7   softmax of the first and second row tile, a row a thread: S out
//                    of tensor memory, maximum, P as 16-bit values over S, sum
//   warp 8           issues the products; zeroes value slots that nobody sees
//   warps 9, 10      copy keys and values (TMA boxes of a page's slots) into rings
//   warp 11          copies the queries
// While one row tile is in its softmax the tensor cores work on the other:
//   Q0 K(u) | P1 V(u-1) | Q1 K(u) | P0 V(u) | Q0 K(u+1) ...
// V lies in shared memory as it lies in the cache, [key][value], and is read as an
// operand whose values, not keys, are contiguous.  A row's output is rescaled only
// when its maximum has grown by more than 2^8 over the reference, which its own
// thread then does in place.
#include "attn_work.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int R = ATTN_TILES_TILE, TK = ATTN_TILES_KEYS, TR = 128;
constexpr int W_MMA = 8, W_K = 9, W_V = 10, W_Q = 11;
// An item costs about as much as three key tiles beside its own, and so does a join.
using Work = AttnWork<R, TK, 3, 6, 6>;
using Walk = AttnWalk<Work>;
constexpr int NTHR = 384;
// Registers a thread: 168 at launch; the softmax warps take what the others leave.
constexpr int REG_LAUNCH = 168, REG_SOFT = 216, REG_REST = 72;
static_assert(256 * REG_SOFT + 128 * REG_REST <= NTHR * REG_LAUNCH, "register shares exceed the launch's");
constexpr uint32_t HALF = TK * 128;  // 64 values of 128 keys or rows

template <int DH>
struct Cfg {
  static constexpr uint32_t SLOT = DH * HALF;   // keys or values of a tile; queries of a row tile
  // A key tile is done with once both row tiles' scores are, a value tile half a tile later.
  static constexpr int NK = DH == 2 ? 2 : 4, NV = DH == 2 ? 3 : 6;
  static constexpr int NS = NK + NV;
};

struct TilesCtl {
  unsigned long long full[10], empty[10];
  unsigned long long q_full[2], q_empty[2];     // queries of a row tile
  unsigned long long s_full[2], p_full[2];      // scores to the softmax; weights to the products
  unsigned long long o_full[2], o_free[2];      // an item's output, complete; read
  unsigned long long done;
  uint32_t tmem, abort, last[2];
  AttnPlan plan;
};
template <int DH>
constexpr uint32_t SMEM_BYTES = 1024 + (2 + Cfg<DH>::NS) * Cfg<DH>::SLOT + ((sizeof(TilesCtl) + 15) & ~15u);
static_assert(SMEM_BYTES<1> <= 232448 && SMEM_BYTES<2> <= 232448, "shared memory of a block");

// What one row tile of an item does in this run's part of it.
struct Tile {
  int rows;        // rows of the tile that there are
  AttnRange keys;  // that any of them sees
  int first, end;  // key tiles to go through
  __device__ __forceinline__ Tile(const AttnArgs& a, const Walk& w, int s) {
    rows = min(max(w.rows() - s * TR, 0), TR);
    first = end = 0;
    keys = AttnRange{0, 0};
    if (rows == 0) return;
    const int r0 = w.row0() + s * TR;
    keys = attn_range(a.p, w.q, a.group, r0, r0 + rows);
    if (keys.hi <= keys.lo) return;
    const int from = w.key0() / TK, to = from + w.key_steps();
    first = max(keys.lo / TK, from);
    end = max(min((keys.hi - 1) / TK + 1, to), first);
  }
  __device__ __forceinline__ bool has(int k) const { return k >= first && k < end; }
};

struct Env {
  const AttnArgs& a;
  TilesCtl& C;
  __device__ __forceinline__ bool wait(unsigned long long& bar, uint32_t parity) const {
    return attn_wait(bar, parity, &C.abort, a.timeout_ns, a.status);
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

// ------------------------------------------------------------ keys, values
// NS slots from `ring` on, their barriers from `full` and `empty` on.
template <int DH, int NS>
__device__ void run_copies(const AttnArgs& a, TilesCtl& C, const CUtensorMap* map, uint32_t ring, unsigned long long* full,
                           unsigned long long* empty) {
  const Env E{a, C};
  const int lane = threadIdx.x & 31, br = a.box_rows, nb = TK / br;
  const int box = lane % nb, half = lane / nb;
  const uint32_t dst0 = (uint32_t)half * HALF + (uint32_t)(box * br) * 128u;
  uint32_t st = 0, par = 0, used = 0;  // par: the phase of each slot's empty barrier that is waited for next
  bool ok = true;
  for (Walk w(a.p, a.group, C.plan); ok && w.live; w.next()) {
    const int steps = w.key_steps();
    if (!steps) continue;
    AttnPages pages;
    int key = w.key0();
    pages.begin(a.p.s.table + w.b * a.p.s.ld_table, max(key, w.keys.lo) >> a.page_shift, (w.keys.hi - 1) >> a.page_shift);
    for (int j = 0; j < steps; ++j, key += TK) {
      if ((used >> st) & 1u) {
        if (!E.wait(empty[st], (par >> st) & 1u)) {
          ok = false;
          break;
        }
        par ^= 1u << st;
      }
      used |= 1u << st;
      const int k = key + box * br;
      const bool mine = half < DH && k + br > w.keys.lo && k < w.keys.hi;
      pages.advance(max(key, w.keys.lo) >> a.page_shift);
      int id = pages.at(min(max(k, w.keys.lo), w.keys.hi - 1) >> a.page_shift);
      const unsigned boxes = __ballot_sync(0xffffffffu, mine);
      if (mine && (id < 0 || id >= a.p.c.kv.n_pages)) {
        atomicOr(a.status, (unsigned)MOE_STATUS_BAD_PAGE);
        id = a.p.c.kv.n_pages;  // outside: filled with zeros
      }
      if (lane == 0) mbar_arrive_expect_tx(attn_bar(full[st]), (uint32_t)__popc(boxes) * (uint32_t)br * 128u);
      __syncwarp();
      if (mine)
        tma_load_4d(ring + st * Cfg<DH>::SLOT + dst0, map, half * 64, k & (a.p.c.kv.page_size - 1), w.h, id,
                    attn_bar(full[st]));
      st = st + 1 == NS ? 0 : st + 1;
    }
  }
  // copies in flight land before the block can exit: each slot's last one
  const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
  for (uint32_t i = 0; i < NS; ++i)
    if ((used >> i) & 1u) mbar_wait_bounded(attn_bar(full[i]), (par >> i) & 1u, deadline, a.status);
}

// ------------------------------------------------------------ queries
// The row tiles' queries into the swizzled layout, rows and values that there are
// none of as zeros.
template <int DH>
__device__ void run_q(const AttnArgs& a, TilesCtl& C, uint32_t q_smem) {
  const Env E{a, C};
  const int lane = threadIdx.x & 31, D = a.p.c.kv.head_dim;
  constexpr int CH = DH * 8;         // 16-byte pieces of a row
  constexpr int RPI = 32 / CH;       // rows an instruction of the warp covers
  const int ch = lane % CH, rr = lane / CH;
  const bool in = ch * 8 < D;
  const uint16_t* q = static_cast<const uint16_t*>(a.p.q);
  uint32_t uses[2] = {};
  for (Walk w(a.p, a.group, C.plan); w.live; w.next()) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Tile T(a, w, s);
      if (T.first >= T.end) continue;
      if (!E.wait(C.q_empty[s], (uses[s]++ & 1u) ^ 1u)) return;  // passes at once the first time
#pragma unroll 1
      for (int r0 = 0; r0 < TR; r0 += 32) {
        // each lane finds one of 32 rows
        const int r = r0 + lane, row = w.row0() + s * TR + r, tok = row / a.group;
        const long long at = (w.q.row0 + tok) * a.p.ldq + (long long)(w.h * a.group + row - tok * a.group) * D;
        const long long off = r < T.rows ? at : -1;
#pragma unroll 8
        for (int i = 0; i < 32; i += RPI) {
          const long long o = __shfl_sync(0xffffffffu, off, i + rr);
          const bool there = o >= 0 && in;
          const uint32_t dst = q_smem + (uint32_t)s * Cfg<DH>::SLOT + (uint32_t)(ch / 8) * HALF + swz(r0 + i + rr, ch & 7);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(there ? q + o + ch * 8 : q),
                       "r"(there ? 16 : 0)
                       : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(attn_bar(C.q_full[s]));
    }
  }
}

// ------------------------------------------------------------ products
// Descriptor of V as the second operand of P V: 64 values of a key are one
// swizzled row of 128 bytes, keys follow one another; the values, not the keys,
// are contiguous.  8 keys are 1024 bytes, the next 64 values HALF on.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(HALF >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// The weights of one row tile against one value tile.
struct Product {
  uint32_t slot;   // of the ring
  int from, to;    // steps of 16 keys that any row sees
  bool first, last;
};

template <int DH, bool BF>
struct Issuer {
  const AttnArgs& a;
  TilesCtl& C;
  const uint32_t tmem, ring, q_smem;
  const Env E;
  uint32_t par_full = 0;                 // phase of each slot
  uint32_t uq[2] = {}, up[2] = {}, uo[2] = {};  // uses of the barriers
  const uint32_t id_qk, id_pv;
  const int ksteps;

  __device__ __forceinline__ Issuer(const AttnArgs& a_, TilesCtl& C_, uint32_t tmem_, uint32_t ring_, uint32_t q_)
      : a(a_), C(C_), tmem(tmem_), ring(ring_), q_smem(q_), E{a_, C_}, id_qk(umma_idesc(TK, BF)),
        id_pv(umma_idesc((a_.p.c.kv.head_dim + 15) & ~15, BF) | (1u << 16)), ksteps((a_.p.c.kv.head_dim + 15) / 16) {}

  __device__ __forceinline__ bool slot_full(uint32_t st) {
    if (!E.wait(C.full[st], (par_full >> st) & 1u)) return false;
    par_full ^= 1u << st;
    return true;
  }
  __device__ __forceinline__ bool scores(int s, uint32_t kslot, bool first, bool last) {
    if (first && !E.wait(C.q_full[s], uq[s]++ & 1u)) return false;
    tc_fence_after();
    if (elect_one()) {
      const uint64_t q = umma_desc(q_smem + (uint32_t)s * Cfg<DH>::SLOT), k = umma_desc(ring + kslot * Cfg<DH>::SLOT);
#pragma unroll
      for (int i = 0; i < DH * 4; ++i)
        if (i < ksteps) {
          const uint64_t off = (uint64_t)((i / 4) * (HALF >> 4) + (i & 3) * 2);
          umma_f16(tmem + (uint32_t)s * 128u, q + off, k + off, id_qk, i > 0);
        }
      umma_commit(attn_bar(C.s_full[s]));
      if (last) umma_commit(attn_bar(C.q_empty[s]));
    }
    __syncwarp();
    return true;
  }
  // free: the value slot has no other use
  __device__ __forceinline__ bool values(int s, const Product& P, bool free) {
    if (P.first && !E.wait(C.o_free[s], (uo[s]++ & 1u) ^ 1u)) return false;  // passes at once the first time
    if (!E.wait(C.p_full[s], up[s]++ & 1u)) return false;
    tc_fence_after();
    if (elect_one()) {
      const uint64_t v = v_desc(ring + P.slot * Cfg<DH>::SLOT);
      const uint32_t o = tmem + 256u + (uint32_t)s * (DH * 64), p = tmem + (uint32_t)s * 128u;
#pragma unroll
      for (int i = 0; i < TK / 16; ++i)
        if (i >= P.from && i < P.to)
          umma_f16_ta(o, p + (uint32_t)i * 8u, v + (uint64_t)(i * (2048 >> 4)), id_pv, !(P.first && i == P.from));
      if (free) umma_commit(attn_bar(C.empty[P.slot]));
      if (P.last) umma_commit(attn_bar(C.o_full[s]));
    }
    __syncwarp();
    return true;
  }
  // Value slots of the tile at key0 that the item's rows do not see, in steps of 16
  // that hold some that they see, hold zeros from here on.
  __device__ __forceinline__ void clean(uint8_t* slot, int key0, const AttnRange& keys) {
    const int lane = threadIdx.x & 31;
    bool any = false;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      int from, to;
      if (side) {
        from = keys.hi - key0;
        to = (from + 15) & ~15;
      } else {
        to = keys.lo - key0;
        from = to & ~15;
      }
      if (from < 0 || to > TK || from >= to) continue;
      any = true;
      for (int i = lane; i < (to - from) * 8 * DH; i += 32) {
        const int half = i / ((to - from) * 8), c = i - half * ((to - from) * 8);
        *reinterpret_cast<uint4*>(slot + half * HALF + from * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (any) {
      fence_async_smem();
      __syncwarp();
    }
  }
};

template <int DH, bool BF>
__device__ __forceinline__ bool issue_all(Issuer<DH, BF>& I, uint8_t* ring_ptr) {
  constexpr int NK = Cfg<DH>::NK, NV = Cfg<DH>::NV;
  const AttnArgs& a = I.a;
  TilesCtl& C = I.C;
  uint32_t ks = NK - 1, vs = NK + NV - 1;  // slots
  bool pending = false;  // the second row tile's product of the tile before
  Product P1{};
  for (Walk w(a.p, a.group, C.plan); w.live; w.next()) {
    const int steps = w.key_steps();
    if (!steps) continue;
    const Tile T0(a, w, 0), T1(a, w, 1);
    const int from = w.key0() / TK;
    for (int k = from; k < from + steps; ++k) {
      const int key0 = k * TK;
      const bool h0 = T0.has(k), h1 = T1.has(k);
      ks = ks + 1 == NK ? 0 : ks + 1;
      vs = vs + 1 == NK + NV ? NK : vs + 1;
      auto product = [&](const Tile& T) {
        return Product{vs, max(T.keys.lo - key0, 0) / 16, (min(T.keys.hi - key0, TK) + 15) / 16, k == T.first,
                       k == T.end - 1};
      };
      if (!I.slot_full(ks)) return false;
      if (h0 && !I.scores(0, ks, k == T0.first, k == T0.end - 1)) return false;
      if (pending && !I.values(1, P1, true)) return false;
      pending = false;
      if (h1 && !I.scores(1, ks, k == T1.first, k == T1.end - 1)) return false;
      if (elect_one()) umma_commit(attn_bar(C.empty[ks]));
      __syncwarp();
      if (!I.slot_full(vs)) return false;
      I.clean(ring_ptr + vs * Cfg<DH>::SLOT, key0, w.keys);
      if (h0 && !I.values(0, product(T0), !h1)) return false;
      if (h1) {
        P1 = product(T1);
        pending = true;
      } else if (!h0) {
        if (elect_one()) umma_commit(attn_bar(C.empty[vs]));
        __syncwarp();
      }
    }
  }
  return !pending || I.values(1, P1, true);
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* w) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}

// One key tile of this thread's row.
template <int DH, bool BF>
__device__ __forceinline__ void soft_tile(uint32_t ts, uint32_t to, int key0, int lo, int hi, float c, bool first, float& m,
                                          float& l) {
  uint32_t v[TK];
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32u * i, v + 32 * i);
  tmem_wait_ld();
  const int from = lo - key0, end = hi - key0;  // of the tile's keys, what the row sees
  if (__any_sync(0xffffffffu, from > 0 || end < TK)) {
#pragma unroll
    for (int j = 0; j < TK; ++j)
      if (j < from || j >= end) v[j] = 0xff800000u;  // -inf
  }
  float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < TK; ++j) t[j & 3] = fmaxf(t[j & 3], __uint_as_float(v[j]));
  const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c;
  const bool rise = top > m + ATTN_SLACK;  // from -inf: by anything
  if (first) {
    m = top;
  } else if (__any_sync(0xffffffffu, rise)) {
    const float next = rise ? top : m;
    const float f = rise ? exp2_fast(m - next) : 1.f;
    m = next;
    l *= f;
#pragma unroll 1
    for (int i = 0; i < DH * 4; ++i) {
      uint32_t o[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]), "=r"(o[8]),
            "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
          : "r"(to + 16u * i));
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st16(to + 16u * i, o);
    }
  }
  const float ref = (m == -INFINITY ? 0.f : m) - ATTN_BIAS<BF>;
  float sum[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = exp2_fast(fmaf(__uint_as_float(v[32 * i + 2 * j]), c, -ref));
      const float y = exp2_fast(fmaf(__uint_as_float(v[32 * i + 2 * j + 1]), c, -ref));
      sum[j & 1] += x;
      sum[2 + (j & 1)] += y;
      p[j] = attn_pack2<BF>(x, y);
    }
    tmem_st16(ts + 16u * i, p);
  }
  l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  tmem_wait_st();
}

// A partial result: (maximum, sum) of 256 rows, then their values, four of all rows
// after four of all rows, so that the threads of a warp write and read side by side.
__device__ __forceinline__ float4* part_values(float* part, int row, int d) {
  return reinterpret_cast<float4*>(part + 2 * R) + (d / 4) * R + row;
}

// Eight values of a row, rounded, of each of four 8-value pieces; the four threads
// of a quad trade theirs, so that each writes a piece of every row of the quad and
// they write 64 bytes side by side.
__device__ __forceinline__ void quad_transpose(uint4 (&x)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & b) continue;
      // keeps piece (i | own bit), gives the other away
      uint4 give = up ? x[i] : x[i | b];
      give.x = __shfl_xor_sync(0xffffffffu, give.x, b);
      give.y = __shfl_xor_sync(0xffffffffu, give.y, b);
      give.z = __shfl_xor_sync(0xffffffffu, give.z, b);
      give.w = __shfl_xor_sync(0xffffffffu, give.w, b);
      if (up) x[i] = give;
      else x[i | b] = give;
    }
  }
}

// 32 values of this thread's row from value c0 on, times inv, out of the row tile's
// rows that there are; by whole warps.  off: where each row's output begins, -1 for none.
template <bool BF>
__device__ __forceinline__ void store_32(const AttnArgs& a, long long off, int c0, const float (&f)[32], float inv) {
  const int lane = threadIdx.x & 31, D = a.p.c.kv.head_dim;
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a row that saw nothing, or scores of -inf alone: zeros
    const float* g = f + 8 * i;
    x[i].x = inv == 0.f ? 0u : attn_pack2<BF>(g[0] * inv, g[1] * inv);
    x[i].y = inv == 0.f ? 0u : attn_pack2<BF>(g[2] * inv, g[3] * inv);
    x[i].z = inv == 0.f ? 0u : attn_pack2<BF>(g[4] * inv, g[5] * inv);
    x[i].w = inv == 0.f ? 0u : attn_pack2<BF>(g[6] * inv, g[7] * inv);
  }
  quad_transpose(x);  // now piece lane & 3 of the quad's rows
  const int d = c0 + 8 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long o = __shfl_sync(0xffffffffu, off, (lane & ~3) + i);
    if (o >= 0 && d < D) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.p.out) + o + d) = x[i];
  }
}

// Joins the n parts of a row tile that runs c0 .. c0 + n - 1 have left; this thread's row.
template <bool BF>
__device__ __forceinline__ void join_row(const AttnArgs& a, int c0, int n, int row, bool there, long long off, float* lse) {
  const int D = a.p.c.kv.head_dim;
  auto part = [&](int x) { return reinterpret_cast<float*>(a.part + (2 * (size_t)(c0 + x) + (x ? 0 : 1)) * a.slot); };
  auto ml = [&](int x) { return there ? __ldcg(reinterpret_cast<const float2*>(part(x)) + row) : make_float2(-INFINITY, 0.f); };
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int x = 0; x < n; ++x) m = fmaxf(m, ml(x).x);
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int x = 0; x < n; ++x) {
    const float2 v = ml(x);
    l += v.y == 0.f ? 0.f : exp2_fast(v.x - ref) * v.y;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 32) {
    float acc[32] = {};
#pragma unroll 2
    for (int x = 0; x < n; ++x) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = there && d0 + 4 * i < D ? __ldcg(part_values(part(x), row, d0 + 4 * i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float2 y = ml(x);
      const float f = y.y == 0.f ? 0.f : exp2_fast(y.x - ref);  // (0: nothing seen)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[4 * i] = fmaf(f, v[i].x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(f, v[i].y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(f, v[i].z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(f, v[i].w, acc[4 * i + 3]);
      }
    }
    store_32<BF>(a, off, d0, acc, inv);
  }
  if (there && lse) *lse = attn_lse<BF>(m, l);
}

template <int DH, bool BF>
__device__ void run_softmax(const AttnArgs& a, TilesCtl& C, uint32_t tmem, int s) {
  const Env E{a, C};
  const int wi = (threadIdx.x >> 5) & 3, tid = threadIdx.x & 127;
  const int D = a.p.c.kv.head_dim;
  const uint32_t lanes = (uint32_t)(wi * 32) << 16;
  const uint32_t ts = tmem + lanes + (uint32_t)s * 128u, to = tmem + lanes + 256u + (uint32_t)s * (DH * 64);
  uint32_t us = 0, uo = 0;  // uses of s_full and o_full
  bool ok = true;
  for (Walk w(a.p, a.group, C.plan); w.live; w.next()) {
    const Tile T(a, w, s);
    if (T.rows == 0) continue;
    const int row = w.row0() + s * TR + tid;  // of the sequence
    int lo = 0, hi = INT_MAX;
    if (tid < T.rows) {
      const AttnRange g = attn_range(a.p, w.q, a.group, row, row + 1);
      lo = g.lo;
      hi = g.hi;
    }
    float m = -INFINITY, l = 0.f;
    for (int k = T.first; k < T.end; ++k) {
      ok = ok && E.wait(C.s_full[s], us++ & 1u);
      if (!ok) break;
      tc_fence_after();
      soft_tile<DH, BF>(ts, to, k * TK, lo, hi, a.c, k == T.first, m, l);
      warp_arrive(C.p_full[s]);
    }
    const bool some = T.first < T.end;
    if (some) {
      ok = ok && E.wait(C.o_full[s], uo++ & 1u);
      tc_fence_after();
    }
    if (!ok) l = NAN;
    const bool whole = w.whole();
    float* part = reinterpret_cast<float*>(a.part + (2 * (size_t)blockIdx.x + (w.skip ? 0 : 1)) * a.slot);
    const int pr = s * TR + tid;
    const int tok = row / a.group, hd = w.h * a.group + row - tok * a.group;
    const long long t = w.q.row0 + tok;
    const bool there = tid < T.rows;
    const long long off = there ? t * a.p.ldo + (long long)hd * D : -1;
    float* lse = a.p.lse ? a.p.lse + t * a.p.ld_lse + hd : nullptr;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      float f[32];
      if (some && ok) {
        tmem_ld32(to + (uint32_t)c0, reinterpret_cast<uint32_t*>(f));
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = ok ? 0.f : NAN;
      }
      if (whole) {
        store_32<BF>(a, off, c0, f, inv);
      } else if (there) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          if (c0 + j < D) *part_values(part, pr, c0 + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
      }
    }
    if (some) warp_arrive(C.o_free[s]);
    if (there) {
      if (!whole) *reinterpret_cast<float2*>(part + 2 * pr) = make_float2(m, l);
      else if (lse) *lse = attn_lse<BF>(m, l);
    }
    if (!whole) {
      int c0;
      const int n = AttnCut<Work::SNAP>::parts(C.plan, w.begin(), w.end(), &c0);
      named_bar_sync(1 + s, TR);
      if (tid == 0) {
        __threadfence();
        unsigned* count = a.count + 2 * c0 + s;
        const bool last = atomicAdd(count, 1u) == (unsigned)(n - 1);
        if (last) *count = 0u;
        C.last[s] = last;
      }
      named_bar_sync(1 + s, TR);
      if (C.last[s]) {
        __threadfence();
        join_row<BF>(a, c0, n, pr, there, off, lse);
      }
      named_bar_sync(1 + s, TR);  // `last` has been read
    }
  }
}

template <int DH, bool BF>
__global__ void __launch_bounds__(NTHR, 1) k_attn_tiles(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  uint8_t* sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint8_t* ring = sm + 2 * Cfg<DH>::SLOT;
  TilesCtl& C = *reinterpret_cast<TilesCtl*>(ring + Cfg<DH>::NS * Cfg<DH>::SLOT);
  const int warp = threadIdx.x >> 5;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg<DH>::NS; ++i) {
      mbar_init(attn_bar(C.full[i]), 1);
      mbar_init(attn_bar(C.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(attn_bar(C.q_full[i]), 1);
      mbar_init(attn_bar(C.q_empty[i]), 1);
      mbar_init(attn_bar(C.s_full[i]), 1);
      mbar_init(attn_bar(C.p_full[i]), 4);
      mbar_init(attn_bar(C.o_full[i]), 1);
      mbar_init(attn_bar(C.o_free[i]), 4);
    }
    mbar_init(attn_bar(C.done), 1);
    C.abort = 0u;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&C.tmem, 512);
  grid_wait();
  attn_plan<Work, NTHR>(a.p, a.group, C.plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFT));
    run_softmax<DH, BF>(a, C, tmem, warp >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_REST));
    if (warp == W_MMA) {
      Issuer<DH, BF> I(a, C, tmem, smem_u32(ring), smem_u32(sm));
      issue_all<DH, BF>(I, ring);
      __syncwarp();
      if (elect_one()) umma_commit(attn_bar(C.done));  // after every product of this thread
    } else if (warp == W_K) {
      run_copies<DH, Cfg<DH>::NK>(a, C, &a.map_k, smem_u32(ring), C.full, C.empty);
    } else if (warp == W_V) {
      constexpr int NK = Cfg<DH>::NK;
      run_copies<DH, Cfg<DH>::NV>(a, C, &a.map_v, smem_u32(ring) + NK * Cfg<DH>::SLOT, C.full + NK, C.empty + NK);
    } else {
      run_q<DH>(a, C, smem_u32(sm));
    }
  }
  __syncwarp();
  // no product may still be writing tensor memory when it is freed
  if (threadIdx.x == 0) mbar_wait_bounded(attn_bar(C.done), 0u, globaltimer_ns() + a.timeout_ns, a.status);
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
