// Products with 4-bit weights and group scales for many tokens, as a
// persistent tcgen05 kernel over tiles of 128 weight rows x up to 256 tokens:
//   out[t, r] = sum_groups s[r, j] sum_{k in j} (q[r, k] - z[r, j]) x[t, k]
//
//   A  q - z, exact in bf16 and fp16, written by the dequantising warps into
//      tensor memory (lane = row), so that shared memory carries B alone.
//   B  x as it is, by TMA (128-byte swizzle), 64 or 128 k a stage.
// A group's products accumulate into a fresh tensor-memory accumulator; the
// epilogue warps drain it, multiply by the row's f32 scale and add it to
// running sums in registers.  So no weight is rounded and the scale costs one
// FMA per group and output.  Two or three accumulators of 128 tokens take
// turns (a tile of more than 128 tokens is two halves that share each A stage),
// so that one is drained while the tensor cores fill the others.
//
// x, at 256 tokens a tile, is the larger operand by far (a weight has four
// bits).  Every block loads its own copy; blocks that run at the same time walk
// through the same k of the same few token tiles, so that x comes from L2
// (pairs of blocks that each loaded half and copied it to both: 515 us where
// this takes 497).
//
// The running sums of 128 outputs per thread need more registers than an even
// split of the register file: the warpgroups trade them (setmaxnreg).
//
// Measured: 512 tokens, 131072 x 5120, groups of 128: 498 us in a graph, 1.38
// PFLOP/s (a library bf16 product reaches 1.92); groups of 64: 772 us.  The
// hand-overs between the warps that dequantise, issue and drain bound it.
#include <cudaTypedefs.h>

#include "internal.h"
#include "ops.h"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int TM = 128;            // weight rows per tile
constexpr int TN = 256;            // tokens per tile, at most
constexpr int HALF = 128;          // tokens per accumulator
constexpr int KS = 64;             // k per swizzled 128-byte row of x
constexpr int RAW_K = 128;         // k per raw stage
constexpr int BBOX = 64;           // tokens per B copy
constexpr uint32_t B_SUB = TN * KS * 2;       // 64 k of all tokens
constexpr uint32_t RAW_STAGE = TM * RAW_K / 2;
constexpr int NSR = 4;             // raw stages

// Groups of 128: stages of 128 k and two accumulators; a drain and its two
// hand-overs fit behind the other half's MMAs (a group has to lie in one stage).
// Shorter groups: stages of 64 k leave tensor memory for a third accumulator,
// which doubles the time for a drain.  512 tokens, 131072 x 5120, and the same
// with stages of 128 k: groups of 32, 1400 us and 1963; of 64, 772 and 760, but
// 225 and 226 for 1000 tokens, 20000 x 4096.
template <int G>
struct Cfg {
  static constexpr int KC = G == 128 ? 128 : 64;   // k per stage of A and B
  static constexpr int SUBS = KC / KS;
  static constexpr int NS = G == 128 ? 3 : 4;      // stages of the A and B rings, which move together
  static constexpr int NACC = G == 128 ? 2 : 3;    // accumulators
  static constexpr uint32_t B_STAGE = SUBS * B_SUB;
  static constexpr uint32_t A_COLS = KC / 2;       // tensor-memory columns of an A stage
  static constexpr uint32_t A_COL0 = NACC * HALF;
  static_assert(A_COL0 + NS * A_COLS <= 512, "tensor memory");
};
constexpr int MAX_NS = 4, MAX_NACC = 3;
constexpr int NEW = 8;             // epilogue warps 0-7: tokens 0-63 (0-3) and 64-127 (4-7) of each half
constexpr int NDW = 8;             // dequantising warps 8-15: the even (8-11) and odd (12-15) 64 k
constexpr int W_TMA = 16, W_MMA = 17, W_RAW = 18;
constexpr int NTHR = 640;
// Registers per thread: 96 at launch; the shares add up to the launch's total.
constexpr int REG_LAUNCH = 96, REG_EPI = 176, REG_DEQ = 40, REG_REST = 48;
static_assert(256 * REG_EPI + 256 * REG_DEQ + 128 * REG_REST <= NTHR * REG_LAUNCH, "register shares exceed the launch's");

struct Q4GemmArgs {
  CUtensorMap map_w;               // w as bytes [n][k / 2], box {64 bytes, 128 rows}
  CUtensorMap map_x;               // x [m][k], box {64 values, 64 rows}
  Q4Params p;
  int tn;                          // tokens per tile: 64, 128 or 256
  int nt, tiles;                   // token tiles; all tiles
  unsigned* status;
  unsigned long long timeout_ns;
};

struct GemmCtl {
  unsigned long long full[MAX_NS];    // a stage's A and B are there
  unsigned long long empty[MAX_NS];   // the MMAs are done with them
  unsigned long long r_full[NSR], r_empty[NSR];
  unsigned long long acc_full[MAX_NACC], acc_empty[MAX_NACC];
  unsigned long long done;
  uint32_t tmem;
  uint32_t abort;
};

template <int G>
constexpr uint32_t SMEM_BYTES = 1024 + Cfg<G>::NS * Cfg<G>::B_STAGE + NSR * RAW_STAGE + ((sizeof(GemmCtl) + 15) & ~15u);
static_assert(SMEM_BYTES<128> <= 232448 && SMEM_BYTES<64> <= 232448, "stages exceed the shared memory of a block");

__device__ __forceinline__ uint64_t* bp(unsigned long long& b) { return reinterpret_cast<uint64_t*>(&b); }

// Bounded wait of one thread; on a timeout the block's abort flag is set and
// every later wait of the block returns false at once.
struct Waiter {
  GemmCtl& C;
  uint64_t timeout_ns;  // of one wait
  unsigned* status;
  __device__ __forceinline__ bool one(unsigned long long& bar, uint32_t parity) const {
    if (mbar_try_wait(bp(bar), parity)) return true;
    if (*reinterpret_cast<volatile uint32_t*>(&C.abort)) return false;
    if (mbar_wait_for(bp(bar), parity, timeout_ns, status)) return true;
    *reinterpret_cast<volatile uint32_t*>(&C.abort) = 1u;
    return false;
  }
  __device__ __forceinline__ bool warp(unsigned long long& bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, one(bar, parity));
  }
};

__device__ __forceinline__ void warp_arrive(unsigned long long& b) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bp(b));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

// A place in a ring: the index, and the phase of each entry in a bit.
template <int N>
struct Place {
  uint32_t i, phases;
  __device__ __forceinline__ uint32_t parity() const { return (phases >> i) & 1u; }
  __device__ __forceinline__ void next() {
    phases ^= 1u << i;
    i = i + 1 == N ? 0u : i + 1;
  }
};

struct Tile {
  int row0, tok0, n;  // n: tokens, rounded up to 16; rows past the end compute zeros
};
__device__ __forceinline__ Tile tile_of(const Q4GemmArgs& a, int t) {
  Tile T;
  const int mt = t / a.nt, nt = t - mt * a.nt;  // neighbouring blocks share weight rows
  T.row0 = mt * TM;
  T.tok0 = nt * a.tn;
  T.n = (min(a.tn, a.p.m - T.tok0) + 15) & ~15;
  return T;
}

// ------------------------------------------------------------ TMA issuers
__device__ void run_raw(const Q4GemmArgs& a, GemmCtl& C, uint32_t raw_smem, const Waiter& wt) {
  const int chunks = (a.p.k + RAW_K - 1) / RAW_K;
  uint32_t u = 0;
  for (int t = (int)blockIdx.x; t < a.tiles; t += (int)gridDim.x) {
    const Tile T = tile_of(a, t);
    for (int c = 0; c < chunks; ++c, ++u) {
      const uint32_t st = u % NSR;
      if (u >= NSR && !wt.one(C.r_empty[st], (u / NSR - 1) & 1u)) goto out;
      mbar_arrive_expect_tx(bp(C.r_full[st]), RAW_STAGE);
      tma_load_2d(raw_smem + st * RAW_STAGE, &a.map_w, c * (RAW_K / 2), T.row0, bp(C.r_full[st]));
    }
  }
out:
  // copies still in flight land before the block can exit
  const uint64_t d2 = globaltimer_ns() + a.timeout_ns;
  for (uint32_t v = u > NSR ? u - NSR : 0u; v < u; ++v)
    mbar_wait_bounded(bp(C.r_full[v % NSR]), (v / NSR) & 1u, d2, a.status);
}

// A and B stage j of the ring holds chunks j, j + NS, ... of every tile, so that
// the roles' loops unroll to fixed stages; `par` holds a stage's phase in bit j.
template <int G>
__device__ void run_x(const Q4GemmArgs& a, GemmCtl& C, uint32_t b_smem, const Waiter& wt) {
  constexpr int KC = Cfg<G>::KC, NS = Cfg<G>::NS, SUBS = Cfg<G>::SUBS;
  const int chunks = (a.p.k + KC - 1) / KC;
  uint32_t par = 0, used = 0;
  for (int t = (int)blockIdx.x; t < a.tiles; t += (int)gridDim.x) {
    const Tile T = tile_of(a, t);
    const int nbox = (T.n + BBOX - 1) / BBOX;
    uint32_t st = 0;
    for (int c = 0; c < chunks; ++c) {
      if (!wt.one(C.empty[st], ((par >> st) & 1u) ^ 1u)) goto out;  // passes at once the first time
      mbar_arrive_expect_tx(bp(C.full[st]), (uint32_t)nbox * BBOX * KC * 2);
      for (int r = 0; r < SUBS * nbox; ++r) {  // (64 tokens, 64 k)
        const int sub = r % SUBS, box = r / SUBS;
        const uint32_t dst = b_smem + st * Cfg<G>::B_STAGE + (uint32_t)sub * B_SUB + (uint32_t)box * (BBOX * 128);
        tma_load_2d(dst, &a.map_x, c * KC + sub * KS, T.tok0 + box * BBOX, bp(C.full[st]));
      }
      par ^= 1u << st;
      used |= 1u << st;
      st = st + 1 == NS ? 0 : st + 1;
    }
  }
out:
  const uint64_t d2 = globaltimer_ns() + a.timeout_ns;
  for (uint32_t st = 0; st < NS; ++st)
    if ((used >> st) & 1u) mbar_wait_bounded(bp(C.full[st]), ((par >> st) & 1u) ^ 1u, d2, a.status);
}

// ------------------------------------------------------------ MMA issuer
// The whole warp walks the loop, so that addresses and descriptors are uniform
// values, and one elected thread issues.  The instructions of this warp per
// MMA count: a round of NS chunks is unrolled, with fixed stages and offsets.
// Every use of an accumulator takes the next one of the ring.
template <bool BF, int G, int NH>
__device__ __forceinline__ bool mma_tile(const Q4GemmArgs& a, GemmCtl& C, uint32_t tmem, uint64_t bdesc0,
                                         const Waiter& wt, int n, int chunks, uint32_t& full_par,
                                         Place<Cfg<G>::NACC>& pc) {
  constexpr int KC = Cfg<G>::KC, NS = Cfg<G>::NS;
  constexpr int GPC = KC / G;        // groups per chunk
  constexpr int STEPS = G / 16;      // MMA steps of a group
  const uint32_t id0 = umma_idesc(min(n, HALF), BF), id1 = umma_idesc(NH == 2 ? n - HALF : 16, BF);
  const int last_groups = GPC == 1 ? 1 : (a.p.k - (chunks - 1) * KC + G - 1) / G;  // groups of the last chunk
#pragma unroll 1
  for (int c0 = 0; c0 < chunks; c0 += NS) {
    asm volatile("" : "+l"(bdesc0), "+r"(tmem));  // offsets are added in place, not kept in registers over the loop
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      if (c0 + st >= chunks) break;
#pragma unroll
      for (int gi = 0; gi < GPC; ++gi) {
        if (gi > 0 && c0 + st == chunks - 1 && gi >= last_groups) break;
        const bool frees = gi == GPC - 1 || (c0 + st == chunks - 1 && gi + 1 >= last_groups);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if (h == 0 && gi == 0 && !wt.warp(C.full[st], (full_par >> st) & 1u)) return false;
          // two halves and two accumulators: the half names its own
          const uint32_t reg = NH == 2 && Cfg<G>::NACC == 2 ? (uint32_t)h : pc.i;
          if (!wt.warp(C.acc_empty[reg], ((pc.phases >> reg) & 1u) ^ 1u)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + reg * HALF, id = h ? id1 : id0;
            // k past the end of the row meets zeros of x (the copies fill them in)
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
              const int step = gi * STEPS + i;
              umma_f16_ta(d, tmem + Cfg<G>::A_COL0 + st * Cfg<G>::A_COLS + step * 8,
                          bdesc0 + (uint64_t)((st * Cfg<G>::B_STAGE + (step / 4) * B_SUB + h * HALF * 128) >> 4) +
                              2u * (step % 4),
                          id, i > 0);
            }
            umma_commit(bp(C.acc_full[reg]));
            if (h == NH - 1 && frees) umma_commit(bp(C.empty[st]));  // the stage is free once these are done
          }
          pc.next();
        }
      }
      full_par ^= 1u << st;
    }
  }
  return true;
}

template <bool BF, int G>
__device__ void run_mma(const Q4GemmArgs& a, GemmCtl& C, uint32_t tmem, uint32_t b_smem, const Waiter& wt) {
  const int chunks = (a.p.k + Cfg<G>::KC - 1) / Cfg<G>::KC;
  const uint64_t bdesc0 = umma_desc(b_smem);
  uint32_t full_par = 0;
  Place<Cfg<G>::NACC> pc{0u, 0u};
  for (int t = (int)blockIdx.x; t < a.tiles; t += (int)gridDim.x) {
    const Tile T = tile_of(a, t);
    pc.i = 0u;  // every tile begins with the first accumulator
    const bool ok = T.n > HALF ? mma_tile<BF, G, 2>(a, C, tmem, bdesc0, wt, T.n, chunks, full_par, pc)
                               : mma_tile<BF, G, 1>(a, C, tmem, bdesc0, wt, T.n, chunks, full_par, pc);
    if (!ok) break;
  }
  __syncwarp();
  if (elect_one()) umma_commit(bp(C.done));  // after every MMA this thread issued
}

// --------------------------------------------------------- dequantisers
__device__ __forceinline__ uint32_t h2_sub(uint32_t v, uint32_t z, bool bf) {
  if (bf) {
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), *reinterpret_cast<__nv_bfloat162*>(&z));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  const __half2 d = __hsub2(*reinterpret_cast<__half2*>(&v), *reinterpret_cast<__half2*>(&z));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Eight codes of a word as four pairs (k, k + 1) of q - z: the code in the
// mantissa of 128 (bf16) or 1024 (fp16), whose unit step holds it, minus
// zz = that base + z in both halves.
template <bool BF>
__device__ __forceinline__ void expand8(uint32_t w, uint32_t zz, uint32_t* o) {
  constexpr uint32_t BASE = BF ? 0x43434343u : 0x64646464u;
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const uint32_t a = __byte_perm(lo, hi, 0x5140u), b = __byte_perm(lo, hi, 0x7362u);  // codes 0-3, 4-7 in order
  o[0] = h2_sub(__byte_perm(a, BASE, 0x4140u), zz, BF);
  o[1] = h2_sub(__byte_perm(a, BASE, 0x4342u), zz, BF);
  o[2] = h2_sub(__byte_perm(b, BASE, 0x4140u), zz, BF);
  o[3] = h2_sub(__byte_perm(b, BASE, 0x4342u), zz, BF);
}

// Warps 8-11 write the even 64 k, warps 12-15 the odd ones; thread = weight row.
template <bool BF, int G>
__device__ void run_dequant(const Q4GemmArgs& a, GemmCtl& C, uint32_t tmem, const uint8_t* raw, const Waiter& wt) {
  const Q4Params& p = a.p;
  const int w = (threadIdx.x >> 5) - NEW, lane = threadIdx.x & 31;
  const int hi = w >> 2, quarter = w & 3, r = quarter * 32 + lane;
  constexpr int KC = Cfg<G>::KC, NS = Cfg<G>::NS;
  const int raws = (p.k + RAW_K - 1) / RAW_K;
  const uint32_t base = BF ? 0x43004300u : 0x64006400u;
  const uint32_t acol = tmem + ((uint32_t)(quarter * 32) << 16) + Cfg<G>::A_COL0 + (KC == 128 ? (uint32_t)hi * 32u : 0u);
  uint32_t ru = 0, par = 0;  // raw stages walked; phases of the A stages
  for (int t = (int)blockIdx.x; t < a.tiles; t += (int)gridDim.x) {
    const Tile T = tile_of(a, t);
    const uint8_t* zrow = p.zeros && T.row0 + r < p.n ? p.zeros + (size_t)(T.row0 + r) * p.ng : nullptr;
    uint32_t as = KC == 128 ? 0u : (uint32_t)hi;
    for (int rc = 0; rc < raws; ++rc, ++ru) {
      const int k0 = rc * RAW_K + hi * KS;
      const uint32_t rs = ru % NSR;
      uint32_t zz[2];  // 32 k each: one group at most
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = k0 + 32 * j;
        zz[j] = base + (p.zeros ? (zrow && k < p.k ? (uint32_t)__ldg(zrow + k / p.group) : 0u) : 8u) * 0x00010001u;
      }
      if (!wt.warp(C.r_full[rs], (ru / NSR) & 1u)) return;
      if (KC == 64 && k0 >= p.k) {  // the row ends in the first half
        if (lane == 0) mbar_arrive(bp(C.r_empty[rs]));
        continue;
      }
      // 64-byte rows, 16-byte piece j of row r at j ^ (r / 2 % 4)
      const uint8_t* row = raw + rs * RAW_STAGE + r * 64;
      uint4 v[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) v[j] = *reinterpret_cast<const uint4*>(row + (((2 * hi + j) ^ ((r >> 1) & 3)) << 4));
      if (!wt.warp(C.empty[as], ((par >> as) & 1u) ^ 1u)) return;
      par ^= 1u << as;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t o[16];
        expand8<BF>(v[j].x, zz[j], o);
        expand8<BF>(v[j].y, zz[j], o + 4);
        expand8<BF>(v[j].z, zz[j], o + 8);
        expand8<BF>(v[j].w, zz[j], o + 12);
        tmem_st8(acol + as * Cfg<G>::A_COLS + j * 16, o);
        tmem_st8(acol + as * Cfg<G>::A_COLS + j * 16 + 8, o + 8);
      }
      tmem_wait_st();
      warp_arrive(C.full[as]);
      // The raw stage goes back only now that its codes have been used: a load that
      // has merely been issued may still be on its way when the next copy lands.
      if (lane == 0) mbar_arrive(bp(C.r_empty[rs]));
      as = KC == 128 ? (as + 1 == NS ? 0u : as + 1) : (as + 2) % NS;
    }
  }
}

// ------------------------------------------------------------- epilogue
// 32 consecutive columns of the warp's lanes; complete after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
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

// R[p] += s * accumulator column col + p for this warp's 64 columns, if it has
// any (columns past the tile's tokens hold leftovers, and are never stored);
// the accumulator is handed back as soon as it has been read.
__device__ __forceinline__ void drain(uint32_t col, int np, float s, float (&R)[64], unsigned long long& empty) {
  if (np > 0) {
    uint32_t v[32];
    tmem_ld32(col, v);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) R[j] = fmaf(s, __uint_as_float(v[j]), R[j]);
    tmem_ld32(col + 32u, v);
    tmem_wait_ld();
    warp_arrive(empty);
#pragma unroll
    for (int j = 0; j < 32; ++j) R[32 + j] = fmaf(s, __uint_as_float(v[j]), R[32 + j]);
  } else {
    warp_arrive(empty);
  }
}

// Tokens tok0 .. tok0 + 63 of one row (those that exist): a warp's stores of a
// token are contiguous.  One comparison, one addition and one store an output:
// the code is unrolled over the registers and its length is what it costs.
template <int T>
__device__ __forceinline__ void store_cols_t(char* out, uint32_t off, uint32_t step, int count, const float (&R)[64]) {
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    if (j < count) *reinterpret_cast<typename Elem<T>::type*>(out + off) = Elem<T>::put(R[j]);
    off += step;
  }
}
__device__ __forceinline__ void store_cols(const Q4Params& p, int row0, int r, int tok0, int np, const float (&R)[64]) {
  const int count = row0 + r < p.n ? min(np, p.m - tok0) : 0;
  const int sz = type_bytes(p.out_type);
  char* out = static_cast<char*>(p.out) + ((long long)tok0 * p.ldo + row0) * sz;
  const uint32_t off = (uint32_t)(r * sz), step = (uint32_t)p.ldo * (uint32_t)sz;  // 64 rows of out span less than 4 GB
  if (p.out_type == MOE_T_F32) store_cols_t<MOE_T_F32>(out, off, step, count, R);
  else if (p.out_type == MOE_T_BF16) store_cols_t<MOE_T_BF16>(out, off, step, count, R);
  else store_cols_t<MOE_T_F16>(out, off, step, count, R);
}

// A 16-bit load that stays where it is written (the compiler would move it next
// to its use, behind the wait that is to hide it).
__device__ __forceinline__ uint32_t load_u16_here(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

template <int G>
__device__ void run_epilogue(const Q4GemmArgs& a, GemmCtl& C, uint32_t tmem, const Waiter& wt) {
  const Q4Params& p = a.p;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int set = w >> 2, quarter = w & 3;
  const uint32_t col = tmem + ((uint32_t)(quarter * 32) << 16) + 64u * set;
  Place<Cfg<G>::NACC> pc{0u, 0u};
  for (int t = (int)blockIdx.x; t < a.tiles; t += (int)gridDim.x) {
    const Tile T = tile_of(a, t);
    const int row = T.row0 + quarter * 32 + lane;
    const uint16_t* srow = p.scales + (size_t)min(row, p.n - 1) * p.ng;
    const int np0 = min(64, min(T.n, HALF) - 64 * set), np1 = min(64, T.n - HALF - 64 * set);  // <= 0: none
    float R0[64], R1[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) R0[j] = R1[j] = 0.f;
    pc.i = 0u;
    uint32_t next = load_u16_here(srow);
    for (int g = 0; g < p.ng; ++g) {
      const float s = p.scale_type == MOE_T_BF16 ? __uint_as_float(next << 16) : half_bits_to_float(next);
      if (g + 1 < p.ng) next = load_u16_here(srow + g + 1);
      if (!wt.warp(C.acc_full[pc.i], pc.parity())) return;
      tc_fence_after();
      drain(col + pc.i * HALF, np0, s, R0, C.acc_empty[pc.i]);
      pc.next();
      if (T.n > HALF) {
        if (!wt.warp(C.acc_full[pc.i], pc.parity())) return;
        tc_fence_after();
        drain(col + pc.i * HALF, np1, s, R1, C.acc_empty[pc.i]);
        pc.next();
      }
    }
    store_cols(p, T.row0, quarter * 32 + lane, T.tok0 + 64 * set, np0, R0);
    if (T.n > HALF) store_cols(p, T.row0, quarter * 32 + lane, T.tok0 + HALF + 64 * set, np1, R1);
  }
}

// ---------------------------------------------------------------- kernel
template <bool BF, int G>
__global__ void __launch_bounds__(NTHR, 1) k_q4_gemm(const __grid_constant__ Q4GemmArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  uint8_t* sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint8_t* raw = sm + Cfg<G>::NS * Cfg<G>::B_STAGE;
  GemmCtl& C = *reinterpret_cast<GemmCtl*>(raw + NSR * RAW_STAGE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < Cfg<G>::NS; ++i) {
      mbar_init(bp(C.full[i]), 1 + NDW / 2 * Cfg<G>::SUBS);  // the copy of x and the warps that write A
      mbar_init(bp(C.empty[i]), 1);
    }
    for (int i = 0; i < NSR; ++i) {
      mbar_init(bp(C.r_full[i]), 1);
      mbar_init(bp(C.r_empty[i]), NDW);
    }
    for (int i = 0; i < Cfg<G>::NACC; ++i) {
      mbar_init(bp(C.acc_full[i]), 1);
      mbar_init(bp(C.acc_empty[i]), NEW);
    }
    mbar_init(bp(C.done), 1);
    C.abort = 0u;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&C.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;
  const uint32_t b_smem = smem_u32(sm), r_smem = smem_u32(raw);
  grid_wait();
  const Waiter wt{C, a.timeout_ns, a.status};

  if (warp < NEW) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_EPI));
    run_epilogue<G>(a, C, tmem, wt);
  } else if (warp < NEW + NDW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_DEQ));
    run_dequant<BF, G>(a, C, tmem, raw, wt);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_REST));
    if (warp == W_MMA) run_mma<BF, G>(a, C, tmem, b_smem, wt);
    else if (warp == W_TMA && lane == 0) run_x<G>(a, C, b_smem, wt);
    else if (warp == W_RAW && lane == 0) run_raw(a, C, r_smem, wt);
  }
  __syncwarp();
  // no MMA may still be writing tensor memory when it is freed: the issuer's
  // final commit follows its last MMA (bounded wait, a fresh deadline)
  if (warp == 0 && lane == 0) mbar_wait_bounded(bp(C.done), 0u, globaltimer_ns() + a.timeout_ns, a.status);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool BF, int G>
int launch_gemm(const Q4GemmArgs& a, int sms, bool* taken, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const auto kernel = k_q4_gemm<BF, G>;
  static PerDevice allocated;  // registers a thread
  const int regs = allocated.get(dev, [&] {
    cudaFuncAttributes fa{};
    return cudaFuncGetAttributes(&fa, kernel) == cudaSuccess &&
                   cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES<G>) == cudaSuccess
               ? fa.numRegs
               : 0;
  });
  if (regs < 1) return MOE_ERR_CUDA;
  // The register trade waits until the launch holds what the shares add up to: a
  // compiler that gave the kernel other than REG_LAUNCH leaves the call to the
  // passes of eight tokens.
  *taken = regs == REG_LAUNCH;
  if (!*taken) return MOE_OK;
  const int grid = a.tiles < sms ? a.tiles : sms;
  return launch_overlapped(kernel, dim3((unsigned)grid), dim3(NTHR), SMEM_BYTES<G>, s, a);
}

}  // namespace

int launch_q4_gemm(const Q4Params& p, unsigned* status, int sms, bool* taken, cudaStream_t s) {
  Q4GemmArgs a{};
  if (!make_map_2d(&a.map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, (uint64_t)p.k / 2, (uint64_t)p.n, (uint64_t)p.k / 2,
                   RAW_K / 2, TM, 64) ||
      !make_map_2d(&a.map_x, CU_TENSOR_MAP_DATA_TYPE_UINT16, p.x, (uint64_t)p.k, (uint64_t)p.m, (uint64_t)p.ldx * 2, KS,
                   BBOX, 128))
    return MOE_ERR_CUDA;
  a.p = p;
  a.status = status;
  a.timeout_ns = 2000000000ull;
  const int mt = (p.n + TM - 1) / TM;
  // The widest tile reads and expands each weight row least often, but leaves
  // SMs idle when there are few tiles.  A chunk costs about as much beside its
  // MMAs as the MMAs of 256 tokens do, whatever the width.
  long long best = -1;
  for (int tn = TN; tn >= 64; tn /= 2) {
    const int nt = (p.m + tn - 1) / tn;
    const long long cost = (((long long)mt * nt + sms - 1) / sms) * (tn + 256);
    if (best < 0 || cost < best) {
      best = cost;
      a.tn = tn;
      a.nt = nt;
    }
  }
  a.tiles = mt * a.nt;
  const bool bf = p.x_type == MOE_T_BF16;
  if (p.group == 128) return bf ? launch_gemm<true, 128>(a, sms, taken, s) : launch_gemm<false, 128>(a, sms, taken, s);
  if (p.group == 64) return bf ? launch_gemm<true, 64>(a, sms, taken, s) : launch_gemm<false, 64>(a, sms, taken, s);
  return bf ? launch_gemm<true, 32>(a, sms, taken, s) : launch_gemm<false, 32>(a, sms, taken, s);
}

}  // namespace moe
