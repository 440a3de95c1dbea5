// Which kernel an attention call takes, and what both are given.
#include "attn_work.cuh"

namespace moe {

namespace {

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

// The cache as [n_pages][kv_heads][page_size][head_dim] in boxes of 64 values x
// box_rows slots (128-byte swizzle); values past head_dim read zero.
bool make_cache_map(CUtensorMap* m, const moe_v41_kv_cfg& c, const void* base, int box_rows) {
  auto fn = encode_fn();
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                              (cuuint64_t)c.n_pages};
  // a pitch that is never stepped by may be anything to the caller, but not to the map
  const cuuint64_t strides[3] = {(cuuint64_t)c.token_pitch * 2, (cuuint64_t)(c.kv_heads > 1 ? c.head_pitch : c.head_dim) * 2,
                                 (cuuint64_t)(c.n_pages > 1 ? c.page_pitch : c.head_dim) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [m][heads][head_dim] in boxes of 64 values x group heads x the tokens
// that make 128 rows with them.
bool make_query_map(CUtensorMap* m, const AttnParams& p, int group) {
  auto fn = encode_fn();
  const cuuint64_t d = (cuuint64_t)p.c.kv.head_dim, h = (cuuint64_t)p.c.heads;
  const cuuint64_t dims[3] = {d, h, (cuuint64_t)p.m};
  const cuuint64_t strides[2] = {d * 2, (p.m > 1 ? (cuuint64_t)p.ldq : d * h) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p.q), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t attn_workspace_bytes(const moe_v41_attn_cfg& c) { return attn_ws(c).total; }

int launch_paged_attention(const AttnParams& p, int max_new, void* ws, cudaStream_t s) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return MOE_ERR_CUDA;
  const moe_v41_kv_cfg& kv = p.c.kv;
  const AttnWs w = attn_ws(p.c);
  uint8_t* base = static_cast<uint8_t*>(ws);
  AttnArgs a{};
  a.p = p;
  a.group = AttnGroup::of(p.c.heads / kv.kv_heads);
  a.page_shift = __builtin_ctz((unsigned)kv.page_size);
  a.c = p.c.scale * 1.4426950408889634f;
  a.status = &reinterpret_cast<Ctrl*>(base)->status;
  a.count = reinterpret_cast<unsigned*>(base + w.count);
  a.part = reinterpret_cast<char*>(base + w.part);
  a.slot = w.slot;
  a.timeout_ns = 2000000000ull;
  const int ctas = sms < ATTN_MAX_CTAS ? sms : ATTN_MAX_CTAS;
  auto maps = [&](int keys) {
    a.box_rows = min(kv.page_size, keys);
    return make_cache_map(&a.map_k, kv, p.k_cache, a.box_rows) && make_cache_map(&a.map_v, kv, p.v_cache, a.box_rows);
  };
  // Up to 16 rows of a key head (tokens of a sequence x heads) or more.  Both sides, 8 heads
  // a key head: two tokens of 16 sequences over 6000, 45 us by the kernel for few rows and
  // 51 by the other; four, 64 and 52; eight, 135 and 54; two of 64 sequences over 600, 50
  // and 61; four, 89 and 61.
  if ((long long)max_new * a.group.n > ATTN_ROWS_TILE) {
    if (!maps(ATTN_TILES_KEYS)) return MOE_ERR_CUDA;
    a.q_map = 128 % a.group.n == 0 && p.ldq < (int64_t(1) << 38);
    if (a.q_map && !make_query_map(&a.map_q, p, a.group.n)) return MOE_ERR_CUDA;
    bool taken = false;
    const int rc = launch_attn_tiles(a, ctas, &taken, s);
    if (rc || taken) return rc;
  }
  return maps(ATTN_ROWS_KEYS) ? launch_attn_rows(a, ctas, s) : MOE_ERR_CUDA;
}

}  // namespace moe
