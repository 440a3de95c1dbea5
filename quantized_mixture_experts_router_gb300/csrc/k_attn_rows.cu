// Attention over a paged cache for few rows at once: single tokens, or a few
// drafted ones, of every sequence, up to 16 rows (tokens x query heads of a key
// head) an item.
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp2(c s_j - m),   s = q k_j,   c = scale log2 e
//
// Bound by the cache's bytes.  A block a SM, with warps that copy tiles of 32
// keys and values (TMA boxes of a page's slots, 128-byte swizzle) into one ring
// and eight warps that take the tiles in turn, each with its own running maximum,
// sum and output (rows x values, in registers), so that no barrier is passed
// between tiles; they are joined at the end of an item.  Products are mma.sync
// m16n8k16: with at most 16 rows the 128-row tiles of tcgen05 would be mostly
// empty, and p would have to pass through tensor memory; here it goes from the
// accumulators of the first product straight into the operands of the second.
//
// Measured in a graph: one token over 131000 (64 heads over 8 key heads of 128, 537 MB) 89 us, 89%
// of a copy's rate; 60 of 40 to 7300 tokens each 76 us (84%), the longest run 11% over an even
// share; one over 700, 11.3 us: the cut 2.5, the first box 1.5, its tile, the end of an item and
// the join.  Heads above 64 values take all 168 registers and spill 16 to 28 bytes.
#include "attn_work.cuh"

namespace moe {

namespace {

constexpr int R = ATTN_ROWS_TILE, TK = ATTN_ROWS_KEYS;
constexpr int NW = 8;                      // warps that compute
constexpr int NP = 4;                      // warps that copy
constexpr int NTHR = (NW + NP) * 32;
// An item costs about as much as six tiles from memory beside its own, a join twice
// that; a block's warps work on eight tiles at once, so that a run of fewer is no
// shorter.  Eight parts are joined at once; one costs half a tile (one token over 131000,
// 16 heads on one key head: 34 us, 39 with as many runs as blocks, 49 with four at once).
using Work = AttnWork<R, TK, 6, 12, 8, 50>;
using Walk = AttnWalk<Work>;
constexpr uint32_t HALF = TK * 128;        // 64 values of a tile's keys
constexpr uint32_t QHALF = R * 128;        // 64 values of an item's queries

template <int DH>
struct Cfg {
  static constexpr int D = DH * 64;        // values of a head, rounded up
  static constexpr uint32_t STAGE = 2 * DH * HALF;
  // Every stage belongs to one warp (a multiple of their number): a warp that waited
  // for a stage's next use while another's was still on its way would take that
  // use's phase for done, as a phase's parity tells it from its neighbours alone.
  static constexpr int NS = DH == 2 ? NW : 2 * NW;
  static_assert(NS % NW == 0, "a stage is one warp's");
  static constexpr int OPITCH = D + 8;     // floats of a row of a warp's output in shared memory
};

template <int DH>
struct Shared {
  alignas(1024) uint8_t ring[Cfg<DH>::NS * Cfg<DH>::STAGE];
  alignas(1024) uint8_t q[2][DH * QHALF];  // queries of this item and the next
  alignas(16) float o[NW][R][Cfg<DH>::OPITCH];
  alignas(16) float ml[NW][R][2];
  unsigned long long full[Cfg<DH>::NS], empty[Cfg<DH>::NS];
  unsigned long long q_full[2], q_empty[2];
  AttnPlan plan;
  uint32_t abort, last;
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += A B: A 16 rows x 16, B 16 x 8
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------ the copying warps
// Rows pw, pw + NP, ... of the item's queries, by the copying warp pw, in the
// swizzled layout; rows and values that there are none of are zeros.  The barrier
// hears of the copies when they have landed.
template <int DH>
__device__ __forceinline__ void copy_q(const AttnArgs& a, const Walk& w, uint32_t q_smem, int pw, unsigned long long& full) {
  constexpr int CH = DH * 8, RPI = 32 / CH;  // 16-byte pieces of a row; rows an instruction of the warp covers
  const int lane = threadIdx.x & 31, ch = lane % CH, D = a.p.c.kv.head_dim, rows = w.rows();
#pragma unroll
  for (int i = 0; i < R / NP; i += RPI) {
    const int r = pw + NP * (i + lane / CH), row = w.row0() + r, tok = a.group.token(row);
    const bool there = r < rows && ch * 8 < D;
    const uint16_t* src = static_cast<const uint16_t*>(a.p.q);
    if (there) src += (w.q.row0 + tok) * a.p.ldq + (long long)(w.h * a.group.n + row - tok * a.group.n) * D + ch * 8;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     q_smem + (uint32_t)(ch / 8) * QHALF + (uint32_t)r * 128u + (uint32_t)(((ch & 7) ^ (r & 7)) << 4)),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full)) : "memory");
}

// Tile u is copying warp u % NP's, which always fills the same stages.  A warp takes
// some 250 ns a tile, and 100 cycles more for each box of a small page.
template <int DH>
__device__ void run_copies(const AttnArgs& a, Shared<DH>& S, int pw) {
  constexpr int NS = Cfg<DH>::NS;
  static_assert(NS % NP == 0, "a stage is one copying warp's");
  const int lane = threadIdx.x & 31;
  const int br = a.box_rows, nb = TK / br;
  const int box = lane % nb, half = lane / nb % DH, val = lane / nb / DH;
  const uint32_t ring = smem_u32(S.ring);
  const uint32_t dst0 = (uint32_t)(val * DH + half) * HALF + (uint32_t)(box * br) * 128u;
  uint32_t st = (uint32_t)pw, par = 0, used = 0;  // par: the phase of each stage's empty barrier that is waited for next
  uint32_t u = 0;                                 // tiles of the run so far
  uint32_t items = 0;                             // with keys, so far
  bool ok = true;
  for (Walk w(a.p, a.group, S.plan); ok && w.live; w.next()) {
    const int steps = w.key_steps();
    if (!steps) continue;
    if (items >= 2 && !attn_wait(S.q_empty[items & 1], (items / 2 - 1) & 1u, &S.abort, a.timeout_ns, a.status)) break;
    copy_q<DH>(a, w, smem_u32(S.q[items & 1]), pw, S.q_full[items & 1]);
    ++items;
    const int first = (int)((uint32_t)(pw + NP - (int)(u % NP)) % NP);  // this warp's first tile of the item
    u += (uint32_t)steps;
    if (first >= steps) continue;
    AttnPages pages;
    int key = w.key0() + first * TK;
    pages.begin(a.p.s.table + w.b * a.p.s.ld_table, max(key, w.keys.lo) >> a.page_shift, (w.keys.hi - 1) >> a.page_shift);
    for (int j = first; j < steps; j += NP, key += NP * TK) {
      const int k = key + box * br;
      const bool mine = val < 2 && k + br > w.keys.lo && k < w.keys.hi;
      pages.advance(max(key, w.keys.lo) >> a.page_shift);
      int id = pages.at(min(max(k, w.keys.lo), w.keys.hi - 1) >> a.page_shift);
      const unsigned boxes = __ballot_sync(0xffffffffu, mine);
      if (mine && (id < 0 || id >= a.p.c.kv.n_pages)) {
        atomicOr(a.status, (unsigned)MOE_STATUS_BAD_PAGE);
        id = a.p.c.kv.n_pages;  // outside: filled with zeros
      }
      if ((used >> st) & 1u) {
        // a stage that was given back because its copies have not landed is not used again
        if (!attn_wait(S.empty[st], (par >> st) & 1u, &S.abort, a.timeout_ns, a.status) ||
            *(volatile uint32_t*)&S.abort) {
          ok = false;
          break;
        }
        par ^= 1u << st;
      }
      used |= 1u << st;
      if (lane == 0) mbar_arrive_expect_tx(attn_bar(S.full[st]), (uint32_t)__popc(boxes) * (uint32_t)br * 128u);
      __syncwarp();
      if (mine)
        tma_load_4d(ring + st * Cfg<DH>::STAGE + dst0, val ? &a.map_v : &a.map_k, half * 64,
                    k & (a.p.c.kv.page_size - 1), w.h, id, attn_bar(S.full[st]));
      st = st + NP >= NS ? (uint32_t)pw : st + NP;
    }
  }
  // Copies in flight land before the block can exit: each stage's last one (its full
  // barrier's phase flips with every use, as `par` does from the second use on).
  const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
  for (uint32_t i = 0; i < NS; ++i)
    if ((used >> i) & 1u) mbar_wait_bounded(attn_bar(S.full[i]), (par >> i) & 1u, deadline, a.status);
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------- the computing warps
// The item's queries as operands of the first product.
template <int DH>
__device__ __forceinline__ void load_q(uint32_t q_smem, uint32_t (&qf)[DH * 4][4]) {
  const int lane = threadIdx.x & 31, row = lane & 15, c = lane >> 4;
#pragma unroll
  for (int ks = 0; ks < DH * 4; ++ks)
    ldmatrix4(q_smem + (uint32_t)(ks / 4) * QHALF + (uint32_t)row * 128u + (uint32_t)((((ks & 3) * 2 + c) ^ (row & 7)) << 4),
              qf[ks]);
}

// One tile of keys against the rows.  lo, hi: what each of the lane's two rows
// sees; m, l: reference maximum and this lane's part of the sum.
template <int DH, bool BF>
__device__ __forceinline__ void do_tile(const uint32_t base, int key, const AttnRange& keys, bool masked,
                                        const int (&lo)[2], const int (&hi)[2], float c, const uint32_t (&qf)[DH * 4][4],
                                        float (&o)[DH * 8][4], float (&m)[2], float (&l)[2]) {
  const int lane = threadIdx.x & 31, t = lane & 3;
  const int mi = lane >> 3, r8 = lane & 7;
  float s[4][4] = {};
  {
    const int row = (mi >> 1) * 8 + r8;  // key of the tile's first 16
    const uint32_t kb = base + (uint32_t)row * 128u;
#pragma unroll
    for (int ks = 0; ks < DH * 4; ++ks) {
      const uint32_t off = (uint32_t)(ks / 4) * HALF + (((uint32_t)((ks & 3) * 2 + (mi & 1)) ^ (uint32_t)r8) << 4);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t b[4];
        ldmatrix4(kb + off + kk * 16 * 128, b);
        mma<BF>(s[2 * kk], qf[ks], b[0], b[1]);
        mma<BF>(s[2 * kk + 1], qf[ks], b[2], b[3]);
      }
    }
  }
  if (masked) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = key + 8 * n + 2 * t + (e & 1);
        if (k < lo[e >> 1] || k >= hi[e >> 1]) s[n][e] = -INFINITY;
      }
  }
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
  bool rise = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
    top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2)) * c;
    rise |= top[i] > m[i] + ATTN_SLACK;  // from -inf: by anything
  }
  if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float to = fmaxf(m[i], top[i]);
      const float f = to == m[i] ? 1.f : exp2_fast(m[i] - to);
      m[i] = to;
      l[i] *= f;
#pragma unroll
      for (int n = 0; n < DH * 8; ++n) {
        o[n][2 * i] *= f;
        o[n][2 * i + 1] *= f;
      }
    }
  }
  uint32_t pf[2][4];
  {
    const float ref[2] = {(m[0] == -INFINITY ? 0.f : m[0]) - ATTN_BIAS<BF>, (m[1] == -INFINITY ? 0.f : m[1]) - ATTN_BIAS<BF>};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[i] = exp2_fast(fmaf(s[n][i], c, -ref[i >> 1]));
        l[i >> 1] += e[i];
      }
      pf[n >> 1][2 * (n & 1)] = attn_pack2<BF>(e[0], e[1]);
      pf[n >> 1][2 * (n & 1) + 1] = attn_pack2<BF>(e[2], e[3]);
    }
  }
  // values of slots that none of the rows sees may be anything: zeros
  const bool edge = key < keys.lo || key + TK > keys.hi;
  const uint32_t vb = base + DH * HALF + (uint32_t)((mi & 1) * 8 + r8) * 128u;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
    if (edge) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = key + 16 * kk + 8 * j + 2 * t;
        keep[j] = (k >= keys.lo && k < keys.hi ? 0xffffu : 0u) | (k + 1 >= keys.lo && k + 1 < keys.hi ? 0xffff0000u : 0u);
      }
    }
#pragma unroll
    for (int n = 0; n < DH * 4; ++n) {
      uint32_t b[4];
      ldmatrix4t(vb + kk * 16 * 128 + (uint32_t)(n / 4) * HALF + (((uint32_t)((n & 3) * 2 + (mi >> 1)) ^ (uint32_t)r8) << 4),
                 b);
      mma<BF>(o[2 * n], pf[kk], b[0] & keep[0], b[1] & keep[1]);
      mma<BF>(o[2 * n + 1], pf[kk], b[2] & keep[0], b[3] & keep[1]);
    }
  }
}

// Joins the n parts of an item's rows that runs c0 .. c0 + n - 1 have left, U at once.  Most items that are cut have
// two: asking for eight whatever there are took 11.6 us for one token over 700 and 76.2 for 60 of 40 to 7300, as
// many as there are 11.4 and 75.8.
template <int U, bool BF>
__device__ __forceinline__ void join_parts(const AttnArgs& a, int c0, int n, int tok0, int h, int row0, int rows) {
  const int D = a.p.c.kv.head_dim, d4 = D / 4;
  auto at = [&](int x) { return reinterpret_cast<const float*>(a.part + (2 * (size_t)(c0 + x) + (x ? 0 : 1)) * a.slot); };
  for (int i = threadIdx.x; i < rows * d4; i += NW * 32) {
    const int r = i / d4, d = (i - r * d4) * 4;
    const AttnJoined v = attn_join<U>(
        n, [&](int x) { return __ldcg(reinterpret_cast<const float2*>(at(x)) + r); },
        [&](int x) { return __ldcg(reinterpret_cast<const float4*>(at(x) + R * 2 + r * D + d)); });
    attn_store<BF>(a, tok0, h, row0 + r, d, v);
  }
}

template <int DH, bool BF>
__device__ void run_rows(const AttnArgs& a, Shared<DH>& S) {
  constexpr int NS = Cfg<DH>::NS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int D = a.p.c.kv.head_dim, d4 = D / 4;
  const uint32_t ring = smem_u32(S.ring);
  uint32_t u = 0;      // tiles of the run so far; tile u is warp u % NW's, in stage u % NS
  uint32_t items = 0;  // with keys, so far
  bool ok = true;      // until a wait runs out: then every phase from there on is in doubt
  for (Walk w(a.p, a.group, S.plan); w.live; w.next()) {
    const int steps = w.key_steps(), rows = w.rows();
    uint32_t j = (uint32_t)(warp + NW - (int)(u % NW)) % NW;  // this warp's first tile of the item
    if (j < (uint32_t)steps) {
      uint32_t qf[DH * 4][4];
      float o[DH * 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {};
      ok = attn_wait(S.q_full[items & 1], (items / 2) & 1u, &S.abort, a.timeout_ns, a.status) && ok;
      load_q<DH>(smem_u32(S.q[items & 1]), qf);
      int lo[2], hi[2], lo_all = 0, hi_all = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 2) + 8 * i;
        lo[i] = hi[i] = 0;
        if (r < rows) {
          const AttnRange g = attn_range(a.p, w.q, a.group, w.row0() + r, w.row0() + r + 1);
          lo[i] = g.lo;
          hi[i] = g.hi;
        }
      }
      // what every row sees
      lo_all = attn_range(a.p, w.q, a.group, w.row0() + rows - 1, w.row0() + rows).lo;
      hi_all = attn_range(a.p, w.q, a.group, w.row0(), w.row0() + 1).hi;
      for (; j < (uint32_t)steps; j += NW) {
        const uint32_t st = (u + j) % NS, par = ((u + j) / NS) & 1u;
        const int key = w.key0() + (int)j * TK;
        ok = attn_wait(S.full[st], par, &S.abort, a.timeout_ns, a.status) && ok;
        if (ok)
          do_tile<DH, BF>(ring + st * Cfg<DH>::STAGE, key, w.keys, key < lo_all || key + TK > hi_all, lo, hi, a.c, qf, o,
                          m, l);
        else
          l[0] = l[1] = NAN;
        __syncwarp();
        if (lane == 0) mbar_arrive(attn_bar(S.empty[st]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const int r = (lane >> 2) + 8 * i;
        if (r < rows) {
          if ((lane & 3) == 0) {
            S.ml[warp][r][0] = m[i];
            S.ml[warp][r][1] = l[i];
          }
#pragma unroll
          for (int n = 0; n < DH * 8; ++n)
            *reinterpret_cast<float2*>(&S.o[warp][r][8 * n + 2 * (lane & 3)]) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
        }
      }
    } else if (lane < rows) {
      S.ml[warp][lane][0] = -INFINITY;
      S.ml[warp][lane][1] = 0.f;
    }
    u += (uint32_t)steps;
    if (steps) {
      __syncwarp();
      if (lane == 0) mbar_arrive(attn_bar(S.q_empty[items & 1]));
      ++items;
    }
    named_bar_sync(1, NW * 32);
    const bool whole = w.whole();
    // A copying warp that gave up leaves its arrivals out: from there on a phase of the queries' barrier is not one
    // item's, and a warp that had waited for nothing yet may have taken other queries for this item's.  `abort` is
    // set before such a phase ends, as it ends only after this block's warps have given an item back whose queries
    // were not all there.  (A stage's barrier hears of one copying warp, and one computing warp waits for its
    // every use in turn.)
    const bool gone = *(volatile uint32_t*)&S.abort != 0u;
    float* part = reinterpret_cast<float*>(a.part + (2 * (size_t)blockIdx.x + (w.skip ? 0 : 1)) * a.slot);
    for (int i = tid; i < rows * d4; i += NW * 32) {
      const int r = i / d4, d = (i - r * d4) * 4;
      AttnJoined v = attn_join<1>(
          NW, [&](int x) { return *reinterpret_cast<const float2*>(S.ml[x][r]); },
          [&](int x) { return *reinterpret_cast<const float4*>(&S.o[x][r][d]); });
      if (gone) v.l = NAN;
      if (whole) {
        attn_store<BF>(a, w.q.row0, w.h, w.row0() + r, d, v);
      } else {
        *reinterpret_cast<float4*>(part + (size_t)R * 2 + r * D + d) = v.o;
        if (d == 0) *reinterpret_cast<float2*>(part + 2 * r) = make_float2(v.m, v.l);
      }
    }
    if (!whole) {
      int c0;
      const int n = AttnCut<Work::SNAP>::parts(S.plan, w.begin(), w.end(), &c0);
      named_bar_sync(1, NW * 32);
      if (tid == 0) {
        __threadfence();
        const bool last = atomicAdd(a.count + 2 * c0, 1u) == (unsigned)(n - 1);
        if (last) a.count[2 * c0] = 0u;
        S.last = last;
      }
      named_bar_sync(1, NW * 32);
      if (S.last) {
        __threadfence();
        if (n <= 2) join_parts<2, BF>(a, c0, n, w.q.row0, w.h, w.row0(), rows);
        else join_parts<8, BF>(a, c0, n, w.q.row0, w.h, w.row0(), rows);
      }
    }
    named_bar_sync(1, NW * 32);
  }
}

template <int DH, bool BF>
__global__ void __launch_bounds__(NTHR, 1) k_attn_rows(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  Shared<DH>& S = *reinterpret_cast<Shared<DH>*>(raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u));
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Cfg<DH>::NS; ++i) {
      mbar_init(attn_bar(S.full[i]), 1);
      mbar_init(attn_bar(S.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(attn_bar(S.q_full[i]), NP * 32);
      mbar_init(attn_bar(S.q_empty[i]), NW);
    }
    S.abort = 0u;
    fence_mbar_init();
  }
  grid_wait();
  attn_plan<Work, NTHR>(a.p, a.group, S.plan, reinterpret_cast<long long(*)[2]>(S.ml), a.status);
  if (threadIdx.x < NW * 32) run_rows<DH, BF>(a, S);
  else run_copies<DH>(a, S, (int)(threadIdx.x >> 5) - NW);
}

template <int DH, bool BF>
int launch(const AttnArgs& a, int ctas, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const auto kernel = k_attn_rows<DH, BF>;
  constexpr int SMEM = (int)sizeof(Shared<DH>) + 1024;
  static_assert(SMEM <= 232448, "shared memory of a block");
  static PerDevice ready;
  if (ready.get(dev, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) == cudaSuccess;
      }) < 1)
    return MOE_ERR_CUDA;
  return launch_overlapped(kernel, dim3((unsigned)ctas), dim3(NTHR), (size_t)SMEM, s, a);
}

}  // namespace

int launch_attn_rows(const AttnArgs& a, int ctas, cudaStream_t s) {
  const bool bf = a.p.c.kv.type == MOE_T_BF16;
  if (a.p.c.kv.head_dim > 64) return bf ? launch<2, true>(a, ctas, s) : launch<2, false>(a, ctas, s);
  return bf ? launch<1, true>(a, ctas, s) : launch<1, false>(a, ctas, s);
}

}  // namespace moe
