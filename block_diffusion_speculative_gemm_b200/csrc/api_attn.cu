// C ABI of the target-side attention operators: rotation table, per-head norms
// with rotation, paged append, and attention of a chunk over paged K/V.
#include <math.h>

#include <algorithm>

#include <nvtx3/nvToolsExt.h>

#include "attn_paged.cuh"
#include "internal.h"

using namespace dflash;

namespace {

struct NvtxCall {
  explicit NvtxCall(const char* name) { nvtxRangePushA(name); }
  ~NvtxCall() { nvtxRangePop(); }
};

bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

int32_t* err_word(void* ws) { return static_cast<int32_t*>(ws); }

// A [n_rows][heads][hd] operand whose rows are `stride` elements apart.
bool rows_ok(const void* p, int64_t stride, int heads, int hd, int esz) {
  return p && aligned(p, 16) && stride >= (int64_t)heads * hd && stride * esz % 16 == 0;
}

int elem_size(int dtype) {
  return dtype == DFLASH_F32 ? 4 : dtype == DFLASH_BF16 || dtype == DFLASH_F16 ? 2 : 0;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, 256)) return DFLASH_EINVAL;
  return have < need ? DFLASH_EWORKSPACE : DFLASH_OK;
}

int check_pool(const void* k_pool, const void* v_pool, int cache_dtype, int n_kv, int n_pages,
               int page_size, const int32_t* page_table, int max_pages) {
  if (!k_pool || !v_pool || !page_table || n_pages < 1 || max_pages < 1 || page_size < 1)
    return DFLASH_EINVAL;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return DFLASH_EINVAL;
  if (cache_dtype != DFLASH_BF16 && cache_dtype != DFLASH_F16)
    return cache_dtype == DFLASH_F32 ? DFLASH_EUNSUPPORTED : DFLASH_EINVAL;
  // a key tile is made of whole pages or lies inside one
  if (page_size != 16 && page_size != 32 && page_size % 64 != 0) return DFLASH_EUNSUPPORTED;
  if ((int64_t)n_pages * n_kv * page_size > 0x7fffffffLL) return DFLASH_EUNSUPPORTED;
  if ((int64_t)max_pages * page_size > (1LL << 30)) return DFLASH_EUNSUPPORTED;
  return DFLASH_OK;
}

// Rows of an item tile: the average request's rows decide.  Either kernel is correct for
// any mix of lengths; 256 is the tcgen05 kernel's pair of query tiles.  With 4 rows
// (32 requests of one token, 4 query heads a key head) the mma.sync kernel takes 50 us
// and the tcgen05 kernel 53, 256 of them 380 and 400, one request of one token 13 and
// 18; with 32 rows (32 blocks of 8) the former 86 and the latter 55, with 64 rows (4
// blocks of 16 behind 32768 keys) 314 and 94.  The average is not the best choice where
// one chunk stands among many single tokens: 63 and a chunk of 128 behind 4096 keys take
// 203 us in the kernel chosen and 182 in the other, 255 and a chunk of 512 978 and 812.
int pick_tile_rows(int batch, int n_rows, int G) {
  const int64_t rows = std::max<int64_t>(((int64_t)n_rows + batch - 1) / batch * G, G);
  return rows <= 16 ? 16 : 256;
}

struct AttnLayout {
  int tile_rows;
  size_t join, part_o, part_ml, end;
};

AttnLayout attn_layout(int batch, int n_rows, int G, int hd) {
  AttnLayout L;
  L.tile_rows = pick_tile_rows(batch, n_rows, G);
  const int ctas = L.tile_rows == 256 ? attn_paged_umma_ctas() : attn_paged_ctas();
  const size_t rows = (size_t)2 * ctas * L.tile_rows;
  L.join = kHeader;
  L.part_o = (L.join + attn_paged_join_bytes() + 255) & ~size_t(255);
  L.part_ml = L.part_o + rows * hd * 4;
  L.end = (L.part_ml + rows * 8 + 255) & ~size_t(255);
  return L;
}

// cos and sin of p * base^(-2i/hd), evaluated in double precision, stored fp32.
__global__ void rope_rows_kernel(float* __restrict__ table, int max_pos, int half, double base) {
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t n = (int64_t)max_pos * half;
  if (idx >= n) return;
  const double ang = (double)(idx / half) * pow(base, -(double)(idx % half) / half);
  table[idx] = (float)cos(ang);
  table[n + idx] = (float)sin(ang);
}

}  // namespace

extern "C" int dflash_rope_table(float* table, int max_pos, int head_dim, double base,
                                 void* stream) {
  NvtxCall nvtx_("dflash_rope_table");
  if (!table || !aligned(table, 16) || max_pos < 1 || head_dim < 2 || head_dim % 2 ||
      !(base > 0.0) || !isfinite(base))
    return DFLASH_EINVAL;
  const int64_t n = (int64_t)max_pos * (head_dim / 2);
  if ((n + 255) / 256 > 0x7fffffffLL) return DFLASH_EUNSUPPORTED;
  rope_rows_kernel<<<(unsigned)((n + 255) / 256), 256, 0, (cudaStream_t)stream>>>(
      table, max_pos, head_dim / 2, base);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ECUDA;
}

extern "C" int dflash_qk_norm_rope(const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, int dtype, const void* g_q, const void* g_k,
                                   float eps, const float* rope, int max_pos,
                                   const int32_t* cu_rows, const int32_t* start_pos, int batch,
                                   int n_rows, int n_q, int n_kv, int head_dim, void* q_out,
                                   int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                   void* ws, size_t ws_bytes, void* stream) {
  NvtxCall nvtx_("dflash_qk_norm_rope");
  if (batch < 1 || n_rows < 0 || n_q < 0 || n_kv < 0 || n_q + (int64_t)n_kv < 1 ||
      n_q + (int64_t)n_kv > 65535)
    return DFLASH_EINVAL;
  const int e = elem_size(dtype);
  if (!e || !(eps >= 0.f) || !isfinite(eps)) return DFLASH_EINVAL;
  if (head_dim != 64 && head_dim != 128) return DFLASH_EUNSUPPORTED;
  if (n_rows == 0) return DFLASH_OK;
  if (!cu_rows || !start_pos) return DFLASH_EINVAL;
  if (n_q && (!rows_ok(q, q_stride, n_q, head_dim, e) ||
              !rows_ok(q_out, q_out_stride, n_q, head_dim, e)))
    return DFLASH_EINVAL;
  if (n_kv && (!rows_ok(k, k_stride, n_kv, head_dim, e) ||
               !rows_ok(k_out, k_out_stride, n_kv, head_dim, e)))
    return DFLASH_EINVAL;
  if (!aligned(g_q, 16) || !aligned(g_k, 16) || !aligned(rope, 16)) return DFLASH_EINVAL;
  if (rope && max_pos < 1) return DFLASH_EINVAL;
  if (const int st = check_ws(ws, ws_bytes, kHeader)) return st;
  return launch_qk_norm_rope(q, q_stride, k, k_stride, dtype, g_q, g_k, eps, rope, max_pos,
                             cu_rows, start_pos, batch, n_rows, n_q, n_kv, head_dim, q_out,
                             q_out_stride, k_out, k_out_stride, err_word(ws),
                             (cudaStream_t)stream);
}

extern "C" int dflash_kv_append_paged(const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, int dtype, const void* g_k, float eps,
                                      const float* rope, int max_pos, const int32_t* cu_rows,
                                      const int32_t* start_pos, int batch, int n_rows, int n_kv,
                                      int head_dim, void* k_pool, void* v_pool, int cache_dtype,
                                      int n_pages, int page_size, const int32_t* page_table,
                                      int max_pages, void* ws, size_t ws_bytes, void* stream) {
  NvtxCall nvtx_("dflash_kv_append_paged");
  if (batch < 1 || n_rows < 0 || n_kv < 1 || n_kv > 32767) return DFLASH_EINVAL;
  const int e = elem_size(dtype);
  if (!e || !(eps >= 0.f) || !isfinite(eps)) return DFLASH_EINVAL;
  if (head_dim != 64 && head_dim != 128) return DFLASH_EUNSUPPORTED;
  if (n_rows == 0) return DFLASH_OK;
  if (!cu_rows || !start_pos || !rows_ok(k, k_stride, n_kv, head_dim, e) ||
      !rows_ok(v, v_stride, n_kv, head_dim, e))
    return DFLASH_EINVAL;
  if (!aligned(g_k, 16) || !aligned(rope, 16) || (rope && max_pos < 1)) return DFLASH_EINVAL;
  if (const int st = check_pool(k_pool, v_pool, cache_dtype, n_kv, n_pages, page_size, page_table,
                                max_pages))
    return st;
  if (const int st = check_ws(ws, ws_bytes, kHeader)) return st;
  KvPages pg;
  pg.table = page_table;
  pg.max_pages = max_pages;
  pg.page = page_size;
  pg.n_pages = n_pages;
  return launch_kv_append_paged(k, k_stride, v, v_stride, dtype, g_k, eps, rope, max_pos, cu_rows,
                                start_pos, batch, n_rows, n_kv, head_dim, k_pool, v_pool,
                                cache_dtype, pg, err_word(ws), (cudaStream_t)stream);
}

extern "C" size_t dflash_attention_paged_workspace_size(int batch, int n_rows, int n_q, int n_kv,
                                                        int head_dim) {
  if (batch < 0 || n_rows < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv || n_q / n_kv > 64 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  if (batch == 0 || n_rows == 0) return kHeader;
  if (batch > kPagedMaxBatch || n_rows > kPagedMaxRows) return 0;
  // The kernel goes by the average request, and the one for longer requests needs more:
  // as for one request that has all rows, so that the workspace of the largest batch and
  // row count serves every call with fewer of either.
  return attn_layout(1, n_rows, n_q / n_kv, head_dim).end;
}

extern "C" int dflash_attention_paged(const void* q, int64_t q_stride, int dtype,
                                      const int32_t* cu_rows, const int32_t* start_pos,
                                      const int32_t* kv_len, int batch, int n_rows, int n_q,
                                      int n_kv, int head_dim, const void* k_pool,
                                      const void* v_pool, int n_pages, int page_size,
                                      const int32_t* page_table, int max_pages, float scale,
                                      int causal, int window, void* out, int64_t out_stride,
                                      float* lse, void* ws, size_t ws_bytes, void* stream) {
  NvtxCall nvtx_("dflash_attention_paged");
  if (batch < 1 || n_rows < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv) return DFLASH_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale) || window < 0) return DFLASH_EINVAL;
  if (!elem_size(dtype)) return DFLASH_EINVAL;
  if (dtype == DFLASH_F32 || (head_dim != 64 && head_dim != 128) || n_q / n_kv > 64 ||
      batch > kPagedMaxBatch || n_rows > kPagedMaxRows)
    return DFLASH_EUNSUPPORTED;
  if (n_rows == 0) return DFLASH_OK;
  if (!cu_rows || !start_pos || !rows_ok(q, q_stride, n_q, head_dim, 2) ||
      !rows_ok(out, out_stride, n_q, head_dim, 2) || !aligned(lse, 4))
    return DFLASH_EINVAL;
  if (const int st =
          check_pool(k_pool, v_pool, dtype, n_kv, n_pages, page_size, page_table, max_pages))
    return st;
  const int G = n_q / n_kv;
  const AttnLayout L = attn_layout(batch, n_rows, G, head_dim);
  if (const int st = check_ws(ws, ws_bytes, L.end)) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  PagedAttnArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.cu = cu_rows;
  a.start = start_pos;
  a.kv_len = kv_len;
  a.batch = batch;
  a.n_rows = n_rows;
  a.nq = n_q;
  a.nkv = n_kv;
  a.G = G;
  a.table = page_table;
  a.max_pages = max_pages;
  a.page = page_size;
  a.n_pages = n_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal != 0;
  a.window = window;
  a.out = out;
  a.out_stride = out_stride;
  a.wide_out = aligned(out, 32) && out_stride % 16 == 0;
  a.lse = lse;
  a.tile_rows = L.tile_rows;
  a.ipq = std::min(L.tile_rows, 128) / G;
  a.ipt = L.tile_rows == 256 ? 2 * a.ipq : a.ipq;
  a.part_o = reinterpret_cast<float*>(base + L.part_o);
  a.part_ml = reinterpret_cast<float*>(base + L.part_ml);
  a.cnt = reinterpret_cast<unsigned*>(base + kCntOff);
  a.err = err_word(ws);
  a.by_g = FastDiv(G);
  a.by_ipt = FastDiv(a.ipt);
  a.by_page = FastDiv(page_size);
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  if (L.tile_rows == 256)
    return launch_attn_paged_umma(a, head_dim, dtype, base + L.join, (cudaStream_t)stream);
  return launch_attn_paged(a, head_dim, dtype, (cudaStream_t)stream);
}
