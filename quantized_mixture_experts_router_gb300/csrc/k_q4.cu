// Products with 4-bit weights and group scales, up to eight tokens a pass:
//   out[t, r] = sum_groups s[r, j] sum_{k in j} (q[r, k] - z[r, j]) x[t, k]
//
// Bound by the weights' bytes as long as a code costs few instructions, so
// both are kept small.
//  - Work is cut into boxes of 32 rows x 256 codes (4 KB).  The boxes of all
//    rows, numbered row tile by row tile, are dealt to the blocks and within a
//    block to its warps in equal contiguous runs, so that any n and k fill
//    every SM to within one box per warp.
//  - Each warp streams its own run: TMA copies of whole boxes (128-byte
//    swizzle) into a ring of its own, no barrier with other warps.
//  - A lane of ldmatrix receives eight consecutive codes of a row as one word.
//    Masked in pairs, codes are fp16 numbers as they stand: 0x000q is
//    q 2^-24 and 0x00q0 is 16 q 2^-24, both subnormal and exact, which the
//    tensor cores (m16n8k16, rows x tokens, f32 sums) take at full rate.  One
//    shift and four masks per eight codes, no conversion; and one packed
//    subtraction a pair takes z off, exactly.  (Taking z sum x off the group's
//    sum instead would be cheaper by it, but a large x that meets a code equal
//    to its zero would leave the rounding of two large sums where its product
//    is 0.)  No weight is ever rounded: the scale multiplies the group's sum.
//  - x is laid out in shared memory once per block as fp16, scaled by a power
//    of two per token that brings its largest value to 2^14..2^15.  The entries
//    that meet 16 q are scaled by 1/16 more: of those, fp16 holds bf16 values
//    down to 2^-28 of the largest exactly, fp16 values down to 2^-25, and the
//    rest is off by at most 2^-35 of the largest; of the others all three are
//    2^-4 of that.  A token with an infinity or a NaN is computed term by term
//    instead.
//  - A row tile shared by several warps of a block is joined in shared memory,
//    one shared by several blocks through the workspace; the last to arrive
//    adds all the parts in the order of the runs, so that the result does not
//    depend on which one that was.
// Measured: 131072 x 5120, one token: 55 us, 6.3 TB/s (copies reach 6.8).  Eight
// tokens, 131072 x 5120, groups of 32: 84 us, where instructions bound it.  50001 x
// 2336, five tokens, zeros: 19.3 us, 3.2 TB/s.  512 x 5120, one token: 5.4 us, of which
// about 3 are the launch, x and the first box's latency one after the other.
#include <cudaTypedefs.h>

#include "ops.h"

namespace moe {

namespace {

constexpr int BOX_ROWS = 32;
constexpr int BOX_K = 256;
constexpr uint32_t BOX_BYTES = BOX_ROWS * BOX_K / 2;
constexpr int MAX_WARPS = 20, MIN_WARPS = 8;
constexpr int MAX_CTAS = 152;
constexpr int MAX_STAGES = 4;
constexpr int PREFETCH = 1;                    // boxes a warp sends for before the stream's previous kernel has ended
constexpr int PART = BOX_ROWS * DECODE_MAX_M;  // floats of one partial tile
constexpr uint32_t SMEM_MAX = 232448;

// n / d for 0 <= n < 2^31 by one multiplication: with s = ceil(log2 d) and
// mul = floor(2^(31+s) / d) + 1 the error n (mul d - 2^(31+s)) / (d 2^(31+s)) < 1 / d.
struct FastDiv {
  unsigned d, shift;
  unsigned long long mul;
  static FastDiv of(unsigned d) {
    FastDiv f{d, 31, 0};
    while ((1ull << (f.shift - 31)) < d) ++f.shift;
    f.mul = (1ull << f.shift) / d + 1;
    return f;
  }
  __device__ __forceinline__ int operator()(int n) const { return (int)(((unsigned long long)(unsigned)n * mul) >> shift); }
};

// `total` items dealt to `runs` contiguous runs, the first (total % runs) one
// longer: where run u begins, and the run that holds item f.
struct Deal {
  int per, rem;
  FastDiv dper, dper1;
  static Deal of(int total, int runs) {
    const int per = total / runs;
    return Deal{per, total % runs, FastDiv::of((unsigned)(per ? per : 1)), FastDiv::of((unsigned)per + 1u)};
  }
  __device__ __forceinline__ int begin(int u) const { return u * per + min(u, rem); }
  __device__ __forceinline__ int run_of(int f) const {
    const int cut = rem * (per + 1);
    return f < cut ? dper1(f) : rem + dper(f - cut);
  }
};

struct Q4Args {
  CUtensorMap map;           // w as bytes [n][k / 2], box {128 bytes, 32 rows}
  Q4Params p;                // m <= 8 tokens of this pass
  int nb;                    // boxes per row tile
  FastDiv dnb, dwarps;       // division by nb, by the warps of a block
  Deal deal;                 // boxes (or whole row tiles) to blocks
  bool by_tile;              // blocks are dealt whole row tiles
  int stages;                // ring depth of a warp
  bool vec;                  // a box's scales (and zeros) of a row are one aligned load
  unsigned* status;
  unsigned* count;           // [blocks] boxes of the row tile that runs over the block's end; zero between calls
  float* part;               // [blocks][2][PART]
  unsigned long long timeout_ns;
};

// Shared memory of a block behind the warps' rings.
struct Q4Ctl {
  unsigned long long bar[MAX_WARPS][MAX_STAGES];
  unsigned count[MAX_WARPS];             // boxes stored of the row tile that runs over the warp's end
  unsigned amax[DECODE_MAX_M];           // f32 bits of the largest |x|
  unsigned bad;                          // bit t: token t holds an infinity or a NaN
};
constexpr uint32_t CTL_BYTES = (sizeof(Q4Ctl) + 15) & ~15u;

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += A B, A 16 rows x 16 k, B 16 k x 8 tokens, fp16 with f32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bits_f32(uint32_t v16, int t) {
  return t == MOE_T_BF16 ? __uint_as_float(v16 << 16) : half_bits_to_float(v16);
}

__device__ __forceinline__ void tma_box(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_box(const void* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// The power of two that scales a token: its largest value's exponent e, held
// where 2^(14 - e) and 2^e are f32 numbers.
__device__ __forceinline__ int token_exp(unsigned amax_bits) { return max((int)(amax_bits >> 23) - 127, -112); }

// One output of a token that holds an infinity or a NaN, by a whole warp.
__device__ __noinline__ float dot_by_terms(const Q4Params& p, int row, int tok) {
  const int lane = threadIdx.x & 31;
  float acc = 0.f;
  for (int k = lane; k < p.k; k += 32) {
    const size_t g = (size_t)row * p.ng + k / p.group;
    const int q = (p.w[(size_t)row * (p.k / 2) + (k >> 1)] >> (4 * (k & 1))) & 15;
    const float w = (float)(q - (p.zeros ? (int)p.zeros[g] : 8)) * bits_f32(p.scales[g], p.scale_type);
    acc = fmaf(w, bits_f32(p.x[tok * p.ldx + k], p.x_type), acc);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}

// A lane's part of a row tile: rows g + 8 i (i < 4, g = lane / 4), tokens 2t
// and 2t + 1 (t = lane % 4): value 2 i + j is (row g + 8 i, token 2 t + j).
__device__ __forceinline__ void store_tile(const Q4Params& p, const Q4Ctl& C, int tile, const float (&v)[8]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int tok = 2 * t + j;
    if (tok >= p.m) continue;
    const float e = __uint_as_float((uint32_t)(token_exp(C.amax[tok]) + 127) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = tile * BOX_ROWS + g + 8 * i;
      // the sums hold q 2^-24 and x 2^(14 - e)
      if (row < p.n) store_elem(p.out, tok * p.ldo + row, p.out_type, v[2 * i + j] * 0x1.0p10f * e);
    }
  }
  if (C.bad) {
    __syncwarp();
    for (int tok = 0; tok < p.m; ++tok) {
      if (!((C.bad >> tok) & 1u)) continue;
      for (int r = tile * BOX_ROWS; r < min(p.n, (tile + 1) * BOX_ROWS); ++r) {
        const float d = dot_by_terms(p, r, tok);
        if (lane == 0) store_elem(p.out, tok * p.ldo + r, p.out_type, d);
      }
    }
  }
}

// The scales (and zeros) of one box, of a lane's four rows g + 8 i.
template <int G, bool ZEROS>
struct BoxScales {
  static constexpr int NG = BOX_K / G;
  static constexpr int NS = NG / 2, NZ = (NG + 3) / 4;
  uint32_t s[4][NS];  // two 16-bit scales a word
  uint32_t z[4][NZ];
  // sp, zp: the lane's first row's first group of the box; stride: elements from
  // row to row g + 8; rows, groups: how many of the lane's four rows, and of the
  // box's groups, there are (a scale past them is 0).
  template <bool VEC>
  __device__ __forceinline__ void load(const uint16_t* sp, const uint8_t* zp, int stride, int rows, int groups) {
    if (rows == 4 && groups >= NG) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* q = sp + i * stride;
        const uint8_t* zq = zp + i * stride;
        if (VEC) {
          if (NG == 2) {
            s[i][0] = __ldg(reinterpret_cast<const uint32_t*>(q));
            if (ZEROS) z[i][0] = __ldg(reinterpret_cast<const uint16_t*>(zq));
          } else if (NG == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
            s[i][0] = v.x;
            s[i][NS - 1] = v.y;
            if (ZEROS) z[i][0] = __ldg(reinterpret_cast<const uint32_t*>(zq));
          } else {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
            s[i][0] = v.x;
            s[i][1 % NS] = v.y;
            s[i][2 % NS] = v.z;
            s[i][NS - 1] = v.w;
            if (ZEROS) {
              const uint2 u = __ldg(reinterpret_cast<const uint2*>(zq));
              z[i][0] = u.x;
              z[i][NZ - 1] = u.y;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < NS; ++j)
            s[i][j] = (uint32_t)__ldg(q + 2 * j) | ((uint32_t)__ldg(q + 2 * j + 1) << 16);
          if (ZEROS) {
#pragma unroll
            for (int j = 0; j < NZ; ++j) {
              z[i][j] = (uint32_t)__ldg(zq + 4 * j) | ((uint32_t)__ldg(zq + 4 * j + 1) << 8);
              if (NG >= 4)
                z[i][j] |= ((uint32_t)__ldg(zq + 4 * j + 2) << 16) | ((uint32_t)__ldg(zq + 4 * j + 3) << 24);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < NS; ++j) s[i][j] = 0u;
#pragma unroll
        for (int j = 0; j < NZ; ++j) z[i][j] = 0u;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          if (i < rows && j < groups) {
            s[i][j / 2] |= (uint32_t)__ldg(sp + i * stride + j) << (16 * (j & 1));
            if (ZEROS) z[i][j / 4] |= (uint32_t)__ldg(zp + i * stride + j) << (8 * (j & 3));
          }
        }
      }
    }
  }
};

// a - b in both halves, as fp16 numbers
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// One box: acc += s (q - z) x over its chunks of 32 k (all eight, or the first
// `chunks`).  buf: the lane's row in the ring slot, its swizzle folded in; xb:
// the lane's x of the box's first chunk.
template <int G, bool ZEROS, bool WHOLE>
__device__ __forceinline__ void do_box(int scale_type, const BoxScales<G, ZEROS>& sc, uint32_t buf, uint32_t xb,
                                       uint32_t xchunk, int chunks, float (&acc)[8]) {
  constexpr int CPG = G / 32;  // chunks per group
#pragma unroll
  for (int gi = 0; gi < BOX_K / G; ++gi) {
    if (!WHOLE && gi * CPG >= chunks) break;
    uint32_t z[4];  // of the lane's rows, in both halves
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z[i] = ZEROS ? __byte_perm(sc.z[i][gi / 4], 0u, 0x4040u + 0x0101u * (gi & 3)) : 0x00080008u;
    float c[2][4] = {};
#pragma unroll
    for (int cj = 0; cj < CPG; ++cj) {
      const int ch = gi * CPG + cj;
      if (WHOLE || ch < chunks) {
        uint32_t w[4], xv[4];
        ldmatrix4(buf ^ (uint32_t)(ch << 4), w);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(xv[0]), "=r"(xv[1]), "=r"(xv[2]), "=r"(xv[3])
                     : "r"(xb + (uint32_t)ch * xchunk));
#pragma unroll
        for (int h = 0; h < 2; ++h)  // codes 0, 4 and 1, 5 of each word, then 2, 6 and 3, 7
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t wa = h ? w[2 * i] >> 8 : w[2 * i], wb = h ? w[2 * i + 1] >> 8 : w[2 * i + 1];
            const uint32_t za = z[2 * i], zb = z[2 * i + 1];
            const uint32_t a[4] = {sub2(wa & 0x000F000Fu, za), sub2(wb & 0x000F000Fu, zb),
                                   sub2(wa & 0x00F000F0u, za << 4), sub2(wb & 0x00F000F0u, zb << 4)};
            mma16816(c[i], a, xv[2 * h], xv[2 * h + 1]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t sw = sc.s[i][gi / 2];
      const float s = bits_f32((gi & 1) ? sw >> 16 : sw & 0xFFFFu, scale_type);
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[2 * i + j] = fmaf(s, c[i >> 1][2 * (i & 1) + j], acc[2 * i + j]);
    }
  }
}

// x of the pass, which copy_x brings into shared memory as it is, in place to
// the form the tensor cores read (see the head of the file): 16-byte pieces
// (chunk of 32 k, token, quarter), the eight values as pairs (0,4) (1,5) (2,6)
// (3,7), the order the masked codes come in.
__device__ __forceinline__ uint32_t x_piece(int m, int tok, int q) {
  return (uint32_t)((((q >> 2) * m + tok) << 2) + (q & 3)) * 16u;
}

__device__ __forceinline__ void copy_x(const Q4Params& p, uint32_t xs) {
  const int pieces = p.k / 8;
  for (int tok = 0; tok < p.m; ++tok)
    for (int q = threadIdx.x; q < pieces; q += blockDim.x)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(xs + x_piece(p.m, tok, q)),
                   "l"(p.x + tok * p.ldx + 8 * q)
                   : "memory");
}

// Eight x of type XT as f32.
template <int XT>
__device__ __forceinline__ void x_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (XT == MOE_T_BF16) {
      f[2 * i] = bf16lo(w[i]);
      f[2 * i + 1] = bf16hi(w[i]);
    } else {
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = q.x;
      f[2 * i + 1] = q.y;
    }
  }
}

template <int XT>
__device__ __forceinline__ void stage_x_t(const Q4Params& p, Q4Ctl& C, uint8_t* xp) {
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int pieces = p.k / 8;
  // warps share the tokens out
  const int tok = warp % p.m, first = warp / p.m * 32 + lane, step = ((nthr >> 5) - tok + p.m - 1) / p.m * 32;
  {  // each token's largest magnitude (the patterns order like the magnitudes)
    uint32_t mx = 0u;
#pragma unroll 4
    for (int q = first; q < pieces; q += step) {
      const uint4 v = *reinterpret_cast<const uint4*>(xp + x_piece(p.m, tok, q));
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
    }
    const unsigned b = __reduce_max_sync(0xffffffffu, max(mx >> 16, mx & 0xFFFFu));
    if (lane == 0) atomicMax(&C.amax[tok], __float_as_uint(bits_f32(b, XT)));
  }
  __syncthreads();
  // an infinity or a NaN anywhere: those tokens are computed by terms
  if (tid < p.m && C.amax[tid] >= 0x7F800000u) atomicOr(&C.bad, 1u << tid);
  const float e = __uint_as_float((uint32_t)(14 - token_exp(C.amax[tok]) + 127) << 23), e16 = e * 0.0625f;
#pragma unroll 2
  for (int q = first; q < pieces; q += step) {
    uint4* ptr = reinterpret_cast<uint4*>(xp + x_piece(p.m, tok, q));
    float f[8];
    x_f32<XT>(*ptr, f);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // odd pairs meet 16 q
      const __half2 h = __floats2half2_rn(f[j] * ((j & 1) ? e16 : e), f[j + 4] * ((j & 1) ? e16 : e));
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *ptr = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ void stage_x(const Q4Params& p, Q4Ctl& C, uint8_t* xp) {
  if (p.x_type == MOE_T_BF16) stage_x_t<MOE_T_BF16>(p, C, xp);
  else stage_x_t<MOE_T_F16>(p, C, xp);
}

template <int G, bool ZEROS, bool VEC>
__global__ void __launch_bounds__(MAX_WARPS * 32, 1) k_q4_rows(const __grid_constant__ Q4Args a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  const uint32_t base0 = smem_u32(raw_smem);
  const uint32_t pad = (1024u - (base0 & 1023u)) & 1023u;
  const Q4Params& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  // shared memory: the warps' rings, the control block, a partial tile per
  // warp, x
  uint8_t* ringp = raw_smem + pad + (uint32_t)(warp * a.stages) * BOX_BYTES;
  const uint32_t ring = smem_u32(ringp);
  uint8_t* q = raw_smem + pad + (uint32_t)(W * a.stages) * BOX_BYTES;
  Q4Ctl& C = *reinterpret_cast<Q4Ctl*>(q);
  const int pairs = (p.m + 1) / 2;
  const int part_ld = pairs * 64;  // floats of a partial tile
  float* parts = reinterpret_cast<float*>(q + CTL_BYTES);
  uint8_t* xp = q + CTL_BYTES + (uint32_t)(W * part_ld) * 4;
  uint64_t* barp = reinterpret_cast<uint64_t*>(C.bar[warp]);

  // everything up to here and the barriers needs no memory of the stream: it
  // may run while the kernel before this one ends
  grid_launch_dependents();
  const int unit = a.by_tile ? a.nb : 1;
  const int cf0 = a.deal.begin(blockIdx.x) * unit, cf1 = a.deal.begin(blockIdx.x + 1) * unit;  // the block's boxes
  const int wper = a.dwarps(cf1 - cf0), wrem = cf1 - cf0 - wper * W;  // dealt to its warps
  auto wbegin = [&](int u) { return cf0 + u * wper + min(u, wrem); };
  const int f0 = wbegin(warp), f1 = wbegin(warp + 1);
  int it = a.dnb(f0), ib = f0 - it * a.nb, ist = 0, left = f1 - f0;  // the box to copy next, one lane's
  int tile = it, b = ib;                                             // the box at hand
  if (lane == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(barp + i, 1);
    fence_mbar_init();
    if (warp == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&a.map) : "memory");
  }
  if (threadIdx.x < MAX_WARPS) C.count[threadIdx.x] = 0u;
  if (threadIdx.x < DECODE_MAX_M) C.amax[threadIdx.x] = 0u;
  if (threadIdx.x == 0) C.bad = 0u;
  // the first boxes start towards L2 (which every earlier write goes through)
  if (lane == 0) {
    int pt = it, pb = ib;
    for (int i = 0; i < PREFETCH && i < left; ++i) {
      prefetch_box(&a.map, pb * (BOX_K / 2), pt * BOX_ROWS);
      if (++pb == a.nb) {
        pb = 0;
        ++pt;
      }
    }
  }
  __syncthreads();
  grid_wait();
  // x first, all of it: its few bytes would otherwise queue behind the weights
  copy_x(p, smem_u32(xp));
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  auto issue = [&]() {
    mbar_arrive_expect_tx(barp + ist, BOX_BYTES);
    tma_box(ring + (uint32_t)ist * BOX_BYTES, &a.map, ib * (BOX_K / 2), it * BOX_ROWS, smem_u32(barp + ist));
    if (++ib == a.nb) {
      ib = 0;
      ++it;
    }
    if (++ist == a.stages) ist = 0;
    --left;
  };
  // one box a warp keeps the memory busy while x is laid out, and is issued sooner than all
  if (lane == 0 && left > 0) issue();
  constexpr int NGB = BOX_K / G;
  BoxScales<G, ZEROS> sc, sc_next;
  // scales (and zeros) of the box that is loaded next
  const uint16_t* sp = p.scales + (size_t)(tile * BOX_ROWS + g) * p.ng + b * NGB;
  const uint8_t* zp = p.zeros + (ZEROS ? (size_t)(tile * BOX_ROWS + g) * p.ng + b * NGB : 0);
  auto load_scales = [&](BoxScales<G, ZEROS>& to, int tl, int bx) {
    const int rows = p.n - tl * BOX_ROWS >= BOX_ROWS ? 4 : max(0, (p.n - tl * BOX_ROWS - g + 7) >> 3);
    to.template load<VEC>(sp, zp, 8 * p.ng, rows, p.ng - bx * NGB);
  };
  if (f0 < f1) load_scales(sc, tile, b);
  stage_x(p, C, xp);
  if (lane == 0)
    for (int i = 1; i < a.stages && left > 0; ++i) issue();
  __syncthreads();
  if (f0 >= f1) return;

  // a lane past the tokens reads token 0's values: its columns are never stored
  const uint32_t xlane = smem_u32(xp) + (uint32_t)((g < p.m ? g : 0) * 64 + t * 16);
  const uint32_t xchunk = (uint32_t)p.m * 64u;
  const uint32_t alane = (uint32_t)lane * 128u + (uint32_t)((lane & 7) << 4);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  const int whole = p.k / BOX_K;  // boxes of a row tile with all their chunks
  const int first_tile = tile;
  int st = 0, b0 = b;             // ring slot; where this row tile's share of the run began
  uint32_t phase = 0;
  // Cleared when a wait runs out: from then on the warp copies and waits no more,
  // and its sums are NaN, which join the other parts like any others, so that
  // every count ends where it began.
  bool ok = true;
  for (int f = f0; f < f1; ++f) {
    const bool wrap = b + 1 == a.nb;
    const int tile1 = wrap ? tile + 1 : tile, b1 = wrap ? 0 : b + 1;
    const int hop = wrap ? BOX_ROWS * p.ng - b * NGB : NGB;
    sp += hop;
    if (ZEROS) zp += hop;
    if (f + 1 < f1) load_scales(sc_next, tile1, b1);
    if (ok && !__all_sync(0xffffffffu, mbar_try_wait(barp + st, phase)) &&
        !__all_sync(0xffffffffu, mbar_wait_for(barp + st, phase, a.timeout_ns, a.status))) {
      ok = false;
      if (lane == 0) {  // the copies in flight land first
        const uint64_t d2 = globaltimer_ns() + a.timeout_ns;
        for (int e = f; e < f1 - left; ++e)
          mbar_wait_bounded(barp + (e - f0) % a.stages, (uint32_t)((e - f0) / a.stages) & 1u, d2, a.status);
        left = 0;
      }
      __syncwarp();
    }
    const uint32_t buf = ring + (uint32_t)st * BOX_BYTES + alane;
    const uint32_t xb = xlane + (uint32_t)(b * (BOX_K / 32)) * xchunk;
    if (b < whole) do_box<G, ZEROS, true>(p.scale_type, sc, buf, xb, xchunk, BOX_K / 32, acc);
    else do_box<G, ZEROS, false>(p.scale_type, sc, buf, xb, xchunk, (p.k - b * BOX_K) / 32, acc);
    __syncwarp();  // every lane has read the box before the ring slot is refilled
    if (lane == 0 && left > 0) issue();
    sc = sc_next;
    if (++st == a.stages) {
      st = 0;
      phase ^= 1u;
    }
    if (wrap || f + 1 == f1) {  // the run leaves this row tile
      if (!ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __uint_as_float(0x7FC00000u);
      }
      const int mine = b + 1 - b0;
      if (mine == a.nb) {
        store_tile(p, C, tile, acc);
      } else {
        // parts of the tile that the run began in lie behind the control
        // block; those of a second one in the ring, which is empty by then
        const int tf0 = tile * a.nb, tf1 = tf0 + a.nb;
        const int share = min(tf1, cf1) - max(tf0, cf0);  // the block's boxes of this row tile
        bool last = true;
        if (mine < share) {
          // the warps that hold them: from the one whose run reaches over the
          // tile's first box here
          int w0 = warp, w1 = warp;
          if (tf0 <= cf0) w0 = 0;
          while (wbegin(w0) > max(tf0, cf0)) --w0;
          if (tf1 >= cf1) w1 = min(W, cf1 - cf0) - 1;
          while (w1 + 1 < W && wbegin(w1 + 1) < min(tf1, cf1)) ++w1;
          const bool cut = wbegin(w0) < tf0;  // only the first run can have begun in an earlier tile
          float* dst = (first_tile == tile ? parts + warp * part_ld : reinterpret_cast<float*>(ringp)) + (t * 8 + g) * 8;
          if (t < pairs) {
            *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
          }
          __threadfence_block();
          __syncwarp();
          unsigned before = 0;
          if (lane == 0) before = atomicAdd(&C.count[w0], (unsigned)mine);
          before = __shfl_sync(0xffffffffu, before, 0);
          last = before + (unsigned)mine == (unsigned)share;
          if (last) {
            __threadfence_block();
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.f;
            if (t < pairs) {
#pragma unroll 4
              for (int v = w0; v <= w1; ++v) {
                const float* src = (cut && v == w0 ? reinterpret_cast<const float*>(ringp + (v - warp) * a.stages * (int)BOX_BYTES)
                                                   : parts + v * part_ld) +
                                   (t * 8 + g) * 8;
                const float4 q0 = *reinterpret_cast<const float4*>(src);
                const float4 q1 = *reinterpret_cast<const float4*>(src + 4);
                acc[0] += q0.x; acc[1] += q0.y; acc[2] += q0.z; acc[3] += q0.w;
                acc[4] += q1.x; acc[5] += q1.y; acc[6] += q1.z; acc[7] += q1.w;
              }
            }
          }
        }
        if (last && share < a.nb) {  // the same between the blocks that share the row tile
          const int c0 = a.deal.run_of(tf0), c1 = a.deal.run_of(tf1 - 1);
          float* dst = a.part + ((size_t)blockIdx.x * 2 + (cf0 >= tf0 ? 0 : 1)) * PART + (t * 8 + g) * 8;
          if (t < pairs) {
            __stcg(reinterpret_cast<float4*>(dst), make_float4(acc[0], acc[1], acc[2], acc[3]));
            __stcg(reinterpret_cast<float4*>(dst + 4), make_float4(acc[4], acc[5], acc[6], acc[7]));
          }
          __threadfence();
          __syncwarp();
          unsigned before = 0;
          if (lane == 0) before = atomicAdd(a.count + c0, (unsigned)share);
          before = __shfl_sync(0xffffffffu, before, 0);
          last = before + (unsigned)share == (unsigned)a.nb;
          if (last) {
            __threadfence();
            if (lane == 0) a.count[c0] = 0u;  // ready for the next call
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.f;
            if (t < pairs) {
#pragma unroll 4
              for (int v = c0; v <= c1; ++v) {
                const float* src = a.part + ((size_t)v * 2 + (a.deal.begin(v) >= tf0 ? 0 : 1)) * PART + (t * 8 + g) * 8;
                const float4 q0 = __ldcg(reinterpret_cast<const float4*>(src));
                const float4 q1 = __ldcg(reinterpret_cast<const float4*>(src + 4));
                acc[0] += q0.x; acc[1] += q0.y; acc[2] += q0.z; acc[3] += q0.w;
                acc[4] += q1.x; acc[5] += q1.y; acc[6] += q1.z; acc[7] += q1.w;
              }
            }
          }
        }
        if (last) store_tile(p, C, tile, acc);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      b0 = 0;
    }
    tile = tile1;
    b = b1;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

struct Ws {
  size_t ctrl, count, part, total;
};
Ws q4_ws() {
  Ws w{};
  w.ctrl = 0;
  w.count = align256(sizeof(Ctrl));
  w.part = w.count + align256(MAX_CTAS * 4);
  w.total = w.part + (size_t)MAX_CTAS * 2 * PART * 4;
  return w;
}

// Shared memory beside the rings.
uint32_t fixed_bytes(int tokens, int k, int warps) {
  const uint32_t pairs = (uint32_t)(tokens + 1) / 2;
  return 1024 + CTL_BYTES + (uint32_t)warps * pairs * 256 + (uint32_t)tokens * k * 2;
}

template <int G, bool ZEROS, bool VEC>
int launch_rows(const Q4Args& a, unsigned grid, int warps, uint32_t smem, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const auto kernel = k_q4_rows<G, ZEROS, VEC>;
  static PerDevice ready;
  if (ready.get(dev, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_MAX) == cudaSuccess;
      }) < 1)
    return MOE_ERR_CUDA;
  return launch_overlapped(kernel, dim3(grid), dim3((unsigned)warps * 32), smem, s, a);
}

template <int G>
int launch_rows_z(const Q4Args& a, unsigned grid, int warps, uint32_t smem, cudaStream_t s) {
  if (a.vec) return a.p.zeros ? launch_rows<G, true, true>(a, grid, warps, smem, s)
                              : launch_rows<G, false, true>(a, grid, warps, smem, s);
  return a.p.zeros ? launch_rows<G, true, false>(a, grid, warps, smem, s)
                   : launch_rows<G, false, false>(a, grid, warps, smem, s);
}

}  // namespace

bool make_map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t cols, uint64_t rows,
                 uint64_t pitch, uint32_t box_cols, uint32_t box_rows, int swizzle) {
  auto fn = encode_fn();
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {pitch};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t es[2] = {1, 1};
  return fn && fn(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t q4_workspace_bytes(const moe_v41_q4_cfg&) { return q4_ws().total; }

int launch_q4_linear(const Q4Params& p0, void* ws, cudaStream_t s) {
  Q4Args a{};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return MOE_ERR_CUDA;
  const Ws w = q4_ws();
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.status = &reinterpret_cast<Ctrl*>(base + w.ctrl)->status;
  // More than eight tokens: passes of eight over the weights (5 us each, 0.1 ns for
  // each value of x that is laid out, and the weights at 6.0, 5.5 or 4.5 TB/s for
  // groups of 128, 64 and 32) against tiles of 128 rows (3 us, and 0.5, 0.84 or 1.4
  // us for each 128 k of the tiles an SM takes).  Measured, passes and tiles in us:
  //   131072 x 5120   16 tokens  125 142 (groups of 128)  168 398 (of 32)
  //                   24 tokens  187 142                  251 397
  //                   48 tokens  373 142                  501 397
  //   5120 x 2304      9 tokens   13.5 12.0                14.1 28.1
  //                   32 tokens   30.4 12.0                32.1 28.3
  // (The tiles address out by 32-bit offsets within a tile: not for pitches above
  // 2^24.)
  auto fits = [&](int wps, int toks) {
    return fixed_bytes(toks, p0.k, wps) + (uint32_t)wps * 2 * BOX_BYTES <= SMEM_MAX;
  };
  if (p0.m > DECODE_MAX_M && p0.ldo <= (1 << 24)) {
    int per_pass = DECODE_MAX_M;
    while (per_pass > 1 && !fits(MIN_WARPS, per_pass)) --per_pass;
    const long long passes = (p0.m + per_pass - 1) / per_pass, bytes = (long long)p0.n * p0.k / 2;
    const int tbs10 = p0.group == 128 ? 60 : p0.group == 64 ? 55 : 45;         // weights in a pass: TB/s times ten
    const int ns_chunk = p0.group == 128 ? 500 : p0.group == 64 ? 840 : 1400;  // 128 k of a tile
    const long long ns_passes = passes * (5000 + bytes / (100 * tbs10)) + (long long)p0.m * p0.k / 10;
    const long long ns_tiles = 3000 + (long long)ns_chunk * (((p0.n + 127) / 128 + sms - 1) / sms) * ((p0.k + 127) / 128);
    if (ns_tiles < ns_passes) {
      bool taken = false;
      const int rc = launch_q4_gemm(p0, a.status, sms, &taken, s);
      if (rc || taken) return rc;
    }
  }
  if (!make_map_2d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p0.w, (uint64_t)p0.k / 2, (uint64_t)p0.n, (uint64_t)p0.k / 2,
                   BOX_K / 2, BOX_ROWS, 128))
    return MOE_ERR_CUDA;
  a.count = reinterpret_cast<unsigned*>(base + w.count);
  a.part = reinterpret_cast<float*>(base + w.part);
  a.timeout_ns = 2000000000ull;
  const int ngb = BOX_K / p0.group;  // groups per box
  a.vec = p0.ng % ngb == 0 && reinterpret_cast<uintptr_t>(p0.scales) % (2 * ngb) == 0 &&
          reinterpret_cast<uintptr_t>(p0.zeros) % ngb == 0;
  a.nb = (p0.k + BOX_K - 1) / BOX_K;
  a.dnb = FastDiv::of((unsigned)a.nb);
  const int tiles = (p0.n + BOX_ROWS - 1) / BOX_ROWS, total = tiles * a.nb;
  sms = min(sms, MAX_CTAS);
  for (int t0 = 0; t0 < p0.m;) {
    // x of the pass's tokens stays in shared memory beside two boxes per warp:
    // 20 warps while it leaves them room, else 16, 12 or 8, else fewer tokens
    int warps = MAX_WARPS, tokens = min(p0.m - t0, DECODE_MAX_M);
    while (warps > MIN_WARPS && !fits(warps, tokens)) warps -= 4;
    while (tokens > 1 && !fits(warps, tokens)) --tokens;
    const uint32_t fixed = fixed_bytes(tokens, p0.k, warps);
    a.stages = min(MAX_STAGES, (int)((SMEM_MAX - fixed) / ((uint32_t)warps * BOX_BYTES)));
    // Whole row tiles per block save the join between blocks, about as long as a
    // box of a warp or two; blocks that share row tiles are more even.  By tile and
    // shared, where the warps' boxes differ by 0: 4608 x 5120, eight tokens, groups of
    // 32, 10.3 and 13.1 us; by 1: 6000 x 6144, one token, 8.5 and 9.0; by 2: 7168 x
    // 18432, 19.0 and 17.4; by 3: 1024 x 16384, 10.7 and 8.0; by 6: 512 x 32768, 17.9
    // and 9.1.
    const int even = (total + sms * warps - 1) / (sms * warps);
    const int by_tile = ((tiles + sms - 1) / sms * a.nb + warps - 1) / warps;
    a.by_tile = by_tile <= even + 1;
    const int ctas = min(sms, a.by_tile ? tiles : total);
    a.deal = Deal::of(a.by_tile ? tiles : total, ctas);
    a.dwarps = FastDiv::of((unsigned)warps);
    a.p = p0;
    a.p.m = tokens;
    a.p.x = p0.x + (size_t)t0 * p0.ldx;
    a.p.out = static_cast<char*>(p0.out) + (size_t)t0 * p0.ldo * type_bytes(p0.out_type);
    const uint32_t smem = fixed + (uint32_t)(warps * a.stages) * BOX_BYTES;
    int rc;
    if (p0.group == 128) rc = launch_rows_z<128>(a, (unsigned)ctas, warps, smem, s);
    else if (p0.group == 64) rc = launch_rows_z<64>(a, (unsigned)ctas, warps, smem, s);
    else rc = launch_rows_z<32>(a, (unsigned)ctas, warps, smem, s);
    if (rc) return rc;
    t0 += tokens;
  }
  return MOE_OK;
}

}  // namespace moe
