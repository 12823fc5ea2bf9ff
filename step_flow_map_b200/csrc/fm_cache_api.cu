// C ABI of the target's paged key/value cache: argument checks, variant
// choice and launches of append, attention and eviction.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "flashmap.h"
#include "fm_host.cuh"
#include "fm_cache.cuh"
#include "fm_cache_attn.cuh"
#include "fm_cache_decode.cuh"
#include "fm_cache_tc.cuh"
#include "fm_cache_weights.cuh"

using fm::bf16;

namespace {

constexpr int64_t MAX_ROWS = 1 << 24;      // new rows of a call, rows of a sequence

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// 4-byte numbers on the device: a misaligned address would be a fault there.
template <typename... P>
fm_status check_aligned4(const char* names, P... p) {
  if ((((uintptr_t)p | ...) & 3) != 0) return set_err(FM_ERR_ARG, "%s must be 4-byte aligned", names);
  return FM_OK;
}

fm_status check_cache(const fm_paged_cache* c) {
  if (!c || !c->k || !c->v || !c->page_table) return set_err(FM_ERR_ARG, "NULL argument");
  if (c->dtype != FM_F32 && c->dtype != FM_BF16)
    return set_err(FM_ERR_ARG, "unknown dtype %d", c->dtype);
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->table_stride < 1)
    return set_err(FM_ERR_ARG, "sizes must be positive");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return set_err(FM_ERR_UNSUPPORTED, "page_size %d is not 16, 32, 64 or 128", c->page_size);
  if (c->head_dim != 64 && c->head_dim != 128 && !(c->head_dim == 32 && c->dtype == FM_F32))
    return set_err(FM_ERR_UNSUPPORTED, "head_dim %d is not 64 or 128 (or 32 in fp32)", c->head_dim);
  if (c->n_kv_heads > 1024)
    return set_err(FM_ERR_UNSUPPORTED, "n_kv_heads %d exceeds 1024", c->n_kv_heads);
  // rows of the whole cache and of one table row are 31-bit numbers
  if ((int64_t)c->n_pages * c->n_kv_heads > (int64_t)0x7fffffff / c->page_size ||
      c->table_stride > MAX_ROWS / c->page_size)
    return set_err(FM_ERR_UNSUPPORTED, "cache too large: pages x heads x page_size must stay below "
                   "2^31, table_stride x page_size at most 2^24");
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->pos) || ((uintptr_t)c->weight & 3) ||
      ((uintptr_t)c->page_table & 3))
    return set_err(FM_ERR_ARG, "k, v and pos must be 16-byte aligned, weight and page_table 4-byte");
  return FM_OK;
}

fm::CacheView view(const fm_paged_cache* c) {
  fm::CacheView v;
  v.n_pages = c->n_pages;
  v.ps_log2 = __builtin_ctz((unsigned)c->page_size);
  v.n_kv = c->n_kv_heads;
  v.table_stride = c->table_stride;
  v.k = c->k;
  v.v = c->v;
  v.pos = c->pos;
  v.weight = c->weight;
  v.table = c->page_table;
  return v;
}

int esize(const fm_paged_cache* c) { return c->dtype == FM_F32 ? 4 : 2; }

fm_status check_rows(const fm_paged_cache* c, int T, int B, int n_heads) {
  if (T < 0 || B < 1 || n_heads < 1) return set_err(FM_ERR_ARG, "sizes must be positive");
  if (B > FM_MAX_CALL_SEQS)
    return set_err(FM_ERR_UNSUPPORTED, "B=%d exceeds %d sequences", B, FM_MAX_CALL_SEQS);
  if (T > MAX_ROWS) return set_err(FM_ERR_UNSUPPORTED, "T=%d exceeds 2^24 rows", T);
  if (n_heads > 4096) return set_err(FM_ERR_UNSUPPORTED, "n_heads %d exceeds 4096", n_heads);
  if (n_heads % c->n_kv_heads)
    return set_err(FM_ERR_ARG, "n_heads %d is not a multiple of n_kv_heads %d", n_heads,
                   c->n_kv_heads);
  if (n_heads / c->n_kv_heads > 128)
    return set_err(FM_ERR_UNSUPPORTED, "more than 128 query heads per key/value head");
  return FM_OK;
}

// A row stride holds the row and keeps every row 16-byte aligned.
fm_status check_stride(const fm_paged_cache* c, const char* name, const void* p, int64_t stride,
                       int heads, int T) {
  if (!p) return set_err(FM_ERR_ARG, "NULL %s", name);
  if (!aligned16(p) || (stride * esize(c)) % 16)
    return set_err(FM_ERR_ARG, "%s rows must be 16-byte aligned", name);
  if ((T > 1 && stride < (int64_t)heads * c->head_dim) || stride < 0 || stride > ((int64_t)1 << 32))
    return set_err(FM_ERR_ARG, "%s row stride %lld is too short for %d heads or out of range", name,
                   (long long)stride, heads);
  return FM_OK;
}

// Rows of `width` bytes, `stride` bytes apart.
struct RowSet {
  uintptr_t at;
  int64_t stride, width;
  int64_t n;
  uintptr_t end() const { return at + (uintptr_t)((n - 1) * stride + width); }
};
RowSet row_set(const fm_paged_cache* c, const void* p, int64_t stride, int heads, int T) {
  return {(uintptr_t)p, stride * esize(c), (int64_t)heads * c->head_dim * esize(c), T};
}
int64_t floor_div(int64_t x, int64_t y) { return x / y - (x % y < 0); }
// Whether two sets of as many rows share a byte.  Slices of one buffer lie row
// by row between one another, so their extents may meet though they share
// nothing.
bool overlap(const RowSet& a, const RowSet& b) {
  if (a.at >= b.end() || b.at >= a.end()) return false;
  if (a.n == 1) return true;
  if (a.stride == b.stride) {
    // row i of a meets row i + k of b iff -b.width < d + k stride < a.width
    const int64_t d = (int64_t)(b.at - a.at);
    const int64_t lo = floor_div(-b.width - d, a.stride) + 1, hi = -floor_div(d - a.width, a.stride) - 1;
    return std::max(lo, 1 - a.n) <= std::min(hi, a.n - 1);
  }
  for (int64_t i = 0, j = 0; i < a.n && j < b.n;) {   // in the order of the addresses
    const uintptr_t x = a.at + (uintptr_t)(i * a.stride), y = b.at + (uintptr_t)(j * b.stride);
    if (x < y + (uintptr_t)b.width && y < x + (uintptr_t)a.width) return true;
    x < y ? ++i : ++j;
  }
  return false;
}

// SM count of the current device, asked once per device.
fm_status device_sms(int* sms) {
  static std::mutex mu;
  static int known[64];
  int dev = 0;
  FM_CUDA(cudaGetDevice(&dev));
  std::lock_guard<std::mutex> lock(mu);
  int& k = known[dev & 63];
  if (!k) FM_CUDA(cudaDeviceGetAttribute(&k, cudaDevAttrMultiProcessorCount, dev));
  *sms = k;
  return FM_OK;
}

#define FM_LAUNCH_OK(what, expr)                                                          \
  do {                                                                                    \
    cudaError_t e_ = (expr);                                                              \
    if (e_ != cudaSuccess)                                                                \
      return set_err(FM_ERR_CUDA, what " launch failed: %s", cudaGetErrorString(e_));     \
  } while (0)

}  // namespace

// ------------------------------------------------------------------ append
namespace {
template <typename T, int DH>
fm_status launch_append(const fm::AppendArgs& a, cudaStream_t st) {
  auto kernel = a.interleaved ? fm::k_cache_append<T, DH, true> : fm::k_cache_append<T, DH, false>;
  FM_LAUNCH_OK("cache append",
               fm::launch_pdl(kernel, dim3((unsigned)((a.T + a.tok - 1) / a.tok)),
                              dim3(fm::CA_THREADS), 0, st, a));
  return FM_OK;
}
}  // namespace

extern "C" fm_status fm_cache_append(const fm_paged_cache* c, const fm_append_args* a,
                                     fm_stream stream) {
  FM_TRY(check_cache(c));
  if (!a) return set_err(FM_ERR_ARG, "NULL argument");
  FM_TRY(check_rows(c, a->T, a->B, a->n_heads));
  if (!a->cu_rows || !a->kv_len) return set_err(FM_ERR_ARG, "NULL argument");
  FM_TRY(check_aligned4("cu_rows, kv_len and q_pos", a->cu_rows, a->kv_len, a->q_pos));
  if (a->rot_dim < 0 || a->rot_dim > c->head_dim || a->rot_dim % 16)
    return set_err(FM_ERR_ARG, "rot_dim %d is not a multiple of 16 up to head_dim %d", a->rot_dim,
                   c->head_dim);
  if (a->rot_dim > 0 && !a->inv_freq) return set_err(FM_ERR_ARG, "NULL inv_freq");
  if ((uintptr_t)a->inv_freq & 7) return set_err(FM_ERR_ARG, "inv_freq must be 8-byte aligned");
  if (!(a->eps >= 0.f) || a->eps > 1e30f) return set_err(FM_ERR_ARG, "eps must be finite and >= 0");
  if (!aligned16(a->q_gain) || !aligned16(a->k_gain))
    return set_err(FM_ERR_ARG, "gains must be 16-byte aligned");
  if (c->pos && !a->q_pos)
    return set_err(FM_ERR_ARG, "a cache with positions needs q_pos");
  if (a->T == 0) return FM_OK;
  FM_TRY(check_stride(c, "q", a->q, a->q_stride, a->n_heads, a->T));
  FM_TRY(check_stride(c, "k", a->k, a->k_stride, c->n_kv_heads, a->T));
  FM_TRY(check_stride(c, "v", a->v, a->v_stride, c->n_kv_heads, a->T));
  FM_TRY(check_stride(c, "q_out", a->q_out, a->q_out_stride, a->n_heads, a->T));
  // a row's values are loaded while the row before it is stored, keys and values
  // by other threads than its queries: only a row in its own place is safe
  const RowSet qo = row_set(c, a->q_out, a->q_out_stride, a->n_heads, a->T);
  const bool in_place = a->q_out == a->q && (a->T == 1 || a->q_out_stride == a->q_stride);
  if ((!in_place && overlap(qo, row_set(c, a->q, a->q_stride, a->n_heads, a->T))) ||
      overlap(qo, row_set(c, a->k, a->k_stride, c->n_kv_heads, a->T)) ||
      overlap(qo, row_set(c, a->v, a->v_stride, c->n_kv_heads, a->T)))
    return set_err(FM_ERR_ARG, "q_out overlaps q, k or v (only q itself with its stride is allowed)");
  fm::AppendArgs k;
  k.c = view(c);
  k.T = a->T;
  k.B = a->B;
  k.n_heads = a->n_heads;
  k.q = a->q;
  k.k = a->k;
  k.v = a->v;
  k.qs = a->q_stride;
  k.ks = a->k_stride;
  k.vs = a->v_stride;
  k.os = a->q_out_stride;
  k.qg = a->q_gain;
  k.kg = a->k_gain;
  k.eps = a->eps;
  k.inv_freq = a->inv_freq;
  k.rot = a->rot_dim;
  k.interleaved = a->interleaved != 0;
  k.cu = a->cu_rows;
  k.kv_len = a->kv_len;
  k.q_pos = a->q_pos;
  k.q_out = a->q_out;
  int sms = 0;
  FM_TRY(device_sms(&sms));
  k.tok = std::max(1, std::min(fm::CA_MAX_TOK, a->T / (4 * sms)));
  cudaStream_t st = (cudaStream_t)stream;
  if (c->dtype == FM_BF16)
    return c->head_dim == 128 ? launch_append<bf16, 128>(k, st) : launch_append<bf16, 64>(k, st);
  if (c->head_dim == 128) return launch_append<float, 128>(k, st);
  return c->head_dim == 64 ? launch_append<float, 64>(k, st) : launch_append<float, 32>(k, st);
}

// ------------------------------------------------------------------ attention
namespace {

// What a call runs and where its workspace parts lie.
struct AttnPlan {
  // k_cache_decode up to 16 packed rows of a key/value head (its MMA's M); past
  // that bf16: k_cache_attn_tc, in pairs of 128-row tiles past 128 rows; fp32:
  // k_cache_attn_simt
  enum { DECODE, TC_ONE, TC_PAIR, SIMT } kind = SIMT;
  int qt = 0, rt = 0, tile_rows = 0, ov = 0, grid = 0;   // rows of a partial; see CacheAttnArgs
  int64_t tiles = 0;
  int score_units = 0;
  size_t o_first = 0, o_tile = 0, o_join = 0, o_lse = 0, o_scores = 0, o_ml = 0, o_part = 0, total = 0;
};

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

fm_status check_attention(const fm_paged_cache* c, const fm_attention_args* a) {
  FM_TRY(check_cache(c));
  if (!a) return set_err(FM_ERR_ARG, "NULL argument");
  FM_TRY(check_rows(c, a->T, a->B, a->n_heads));
  if (a->max_rows < 1 || a->max_kv < 1) return set_err(FM_ERR_ARG, "sizes must be positive");
  if (a->max_kv > MAX_ROWS) return set_err(FM_ERR_UNSUPPORTED, "max_kv %d exceeds 2^24", a->max_kv);
  if (a->window < 0 || a->sinks < 0)
    return set_err(FM_ERR_ARG, "window and sinks must not be negative");
  if (a->accumulate && !c->weight) return set_err(FM_ERR_ARG, "accumulate needs cache->weight");
  return FM_OK;
}

fm_status plan_attention(const fm_paged_cache* c, const fm_attention_args* a, AttnPlan* p) {
  int sms = 0;
  FM_TRY(device_sms(&sms));
  const int64_t G = a->n_heads / c->n_kv_heads;
  const int64_t rows = a->max_rows * G;
  p->kind = rows <= 16 ? AttnPlan::DECODE : AttnPlan::SIMT;
  p->qt = p->rt = p->tile_rows = rows <= 16 ? fm::CD_QT : fm::CS_QT;
  // resident CTAs: shared memory holds one of the fp32 kernels of width 128 per SM
  p->grid = (c->dtype == FM_F32 && c->head_dim == 128 ? 1 : 2) * sms;
  if (c->dtype == FM_BF16) {
    if (rows > 16) {
      // whole queries per 128-row tile, so that one TMA box brings them
      p->rt = (int)(128 / G * G);
      const bool pair = rows > p->rt;
      p->kind = pair ? AttnPlan::TC_PAIR : AttnPlan::TC_ONE;
      p->qt = pair ? 256 : 128;
      p->tile_rows = pair ? 2 * p->rt : p->rt;
      p->ov = 4;
      p->grid = sms;
    }
  }
  p->tiles = ((int64_t)a->T * G) / p->tile_rows + a->B;
  // units are 31-bit numbers
  const int64_t kb = p->kind == AttnPlan::TC_ONE || p->kind == AttnPlan::TC_PAIR ? fm::CT_KB : fm::CD_KB;
  if (p->tiles * c->n_kv_heads >= 0x7fffffff / (a->max_kv / kb + p->ov + 2))
    return set_err(FM_ERR_UNSUPPORTED, "T=%d rows over max_kv %d: more than 2^31 blocks of work", a->T,
                   a->max_kv);
  size_t at = 256;
  p->o_first = at;
  at = up256(at + (size_t)(p->tiles + 1) * sizeof(int));
  p->o_tile = at;
  at = up256(at + (size_t)p->tiles * 2 * sizeof(int4));
  p->o_join = at;
  at = up256(at + (size_t)p->grid * 2 * sizeof(int4));
  p->o_lse = at;
  if (a->accumulate) at = up256(at + (size_t)a->T * a->n_heads * sizeof(float));
  // scores of few packed rows are kept for the weights, unit by unit (see
  // score_at): no more units than max_kv allows, or than the cache has rows for
  // (no page is in two tables of a call that writes weights), so they take 1/32
  // of the keys' and values' bytes at four packed rows of width 128 in bf16, 1/8
  // at sixteen.  (64 sequences of which one has 65,536 rows, the others 2,048: 24 MB
  // against 512 MB by max_kv alone, in the same time.)
  p->o_scores = at;
  if (a->accumulate && rows <= 16) {
    const int64_t bytes = fm::CD_KB * rows * (int64_t)sizeof(float);
    const int64_t blocks = std::min((int64_t)a->B * ((a->max_kv + fm::CD_KB - 1) / fm::CD_KB),
                                    (int64_t)c->n_pages * c->page_size / fm::CD_KB + a->B);
    p->score_units = (int)(blocks * c->n_kv_heads);
    at = up256(at + (size_t)(p->score_units * bytes));
  }
  p->o_ml = at;
  at = up256(at + (size_t)p->grid * 2 * p->qt * sizeof(float2));
  p->o_part = at;
  at = up256(at + (size_t)p->grid * 2 * p->qt * c->head_dim * sizeof(float));
  p->total = at;
  return FM_OK;
}

template <int DH>
fm_status launch_simt(const fm::CacheAttnArgs& k, const AttnPlan& p, cudaStream_t st) {
  using C = fm::CsCfg<DH>;
  FM_CUDA(fm::set_smem_once(fm::k_cache_attn_simt<DH>, C::SMEM));
  FM_LAUNCH_OK("cache attention plan",
               fm::launch_pdl(fm::k_cache_plan<fm::CS_KB>, dim3(1), dim3(fm::CP_THREADS), 0, st, k));
  FM_LAUNCH_OK("cache attention", fm::launch_pdl(fm::k_cache_attn_simt<DH>, dim3(p.grid),
                                                 dim3(fm::CS_THREADS), C::SMEM, st, k));
  // a warp per row
  const unsigned rows = (unsigned)std::min<int64_t>(fm::CS_QT, (int64_t)k.max_rows * k.G);
  FM_LAUNCH_OK("cache attention join",
               fm::launch_pdl(fm::k_cache_join_rows<float, DH, fm::CS_QT>, dim3(p.grid - 1, (rows + 3) / 4),
                              dim3(fm::CJ_THREADS), 0, st, k));
  return FM_OK;
}

template <typename T, int DH>
fm_status launch_decode(const fm::CacheAttnArgs& k, const AttnPlan& p, cudaStream_t st) {
  using C = fm::CdCfg<T, DH>;
  FM_CUDA(fm::set_smem_once(fm::k_cache_decode<T, DH>, C::SMEM));
  // no more CTAs than units
  const int64_t units = (int64_t)k.B * k.c.n_kv * ((k.max_kv + fm::CD_KB - 1) / fm::CD_KB + 1);
  const int grid = (int)std::min<int64_t>(p.grid, units);
  FM_LAUNCH_OK("cache attention", fm::launch_pdl(fm::k_cache_decode<T, DH>, dim3(grid),
                                                 dim3(fm::CD_THREADS), C::SMEM, st, k));
  if (grid > 1)
    FM_LAUNCH_OK("cache attention join",
                 fm::launch_pdl(fm::k_cache_join_rows<T, DH, fm::CD_QT>,
                                dim3(grid - 1, (unsigned)(k.max_rows * k.G)), dim3(fm::CJ_THREADS), 0,
                                st, k));
  return FM_OK;
}

template <int DH, bool PAIR>
fm_status launch_tc(const fm::CacheAttnArgs& k, const AttnPlan& p, cudaStream_t st) {
  using C = fm::CtCfg<DH>;
  constexpr int QT = PAIR ? 256 : 128;
  auto kernel = fm::k_cache_attn_tc<DH, PAIR>;
  char err[256] = "";
  auto enc = fm::tma_encoder(err, sizeof(err));
  if (!enc) return set_err(FM_ERR_CUDA, "%s", err);
  // one row of the map is one cached row of one head; a box is 64 columns of
  // the part of a page that one block of 128 rows takes
  CUtensorMap mk, mv;
  const cuuint64_t dims[2] = {(cuuint64_t)DH, ((cuuint64_t)k.c.n_pages * k.c.n_kv) << k.c.ps_log2};
  const cuuint64_t strides[1] = {(cuuint64_t)DH * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)(1 << k.c.ps_log2)};
  const cuuint32_t es[2] = {1, 1};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = enc(i ? &mv : &mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, i ? k.c.v : k.c.k, dims,
                           strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_err(FM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  // the queries as [T][key/value heads][G][DH]; a box is 64 columns of the G
  // heads of rt / G rows
  CUtensorMap mq;
  {
    const cuuint64_t d[4] = {(cuuint64_t)DH, (cuuint64_t)k.G, (cuuint64_t)k.c.n_kv, (cuuint64_t)k.T};
    const cuuint64_t st4[3] = {(cuuint64_t)DH * 2, (cuuint64_t)DH * 2 * k.G, (cuuint64_t)std::max<int64_t>(k.qs, (int64_t)k.n_heads * DH) * 2};
    const cuuint32_t b4[4] = {64, (cuuint32_t)k.G, 1, (cuuint32_t)(k.rt / k.G)};
    const cuuint32_t e4[4] = {1, 1, 1, 1};
    const CUresult r = enc(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(k.q), d, st4, b4,
                           e4, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_err(FM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  FM_CUDA(fm::set_smem_once(kernel, C::SMEM));
  FM_LAUNCH_OK("cache attention plan",
               fm::launch_pdl(fm::k_cache_plan<fm::CT_KB>, dim3(1), dim3(fm::CP_THREADS), 0, st, k));
  FM_LAUNCH_OK("cache attention", fm::launch_pdl(kernel, dim3(p.grid), dim3(fm::CT_THREADS), C::SMEM,
                                                 st, mk, mv, mq, k));
  FM_LAUNCH_OK("cache attention join",
               fm::launch_pdl(fm::k_cache_join_cols<DH, QT>, dim3(p.grid - 1, QT / 32),
                              dim3(fm::CJ_THREADS), 0, st, k));
  return FM_OK;
}

template <typename T, int DH>
fm_status run_attention(const fm::CacheAttnArgs& k, const AttnPlan& p, int accumulate,
                        cudaStream_t st) {
  if (p.kind == AttnPlan::DECODE) FM_TRY((launch_decode<T, DH>(k, p, st)));
  else if constexpr (std::is_same<T, bf16>::value) {
    if (p.kind == AttnPlan::TC_ONE) FM_TRY((launch_tc<DH, false>(k, p, st)));
    else FM_TRY((launch_tc<DH, true>(k, p, st)));
  } else FM_TRY((launch_simt<DH>(k, p, st)));
  if (!accumulate) return FM_OK;
  // at least two waves of CTAs where the rows allow it
  auto grid = [&](int per) {
    return dim3((unsigned)std::max(1, std::min((k.max_kv + per - 1) / per, 256)), k.c.n_kv, k.B);
  };
  if (p.kind == AttnPlan::DECODE) {
    FM_LAUNCH_OK("cache weights", fm::launch_pdl(fm::k_cache_weights_scores<T, DH>, grid(fm::CW_THREADS),
                                                 dim3(fm::CW_THREADS), 0, st, k));
  } else if constexpr (std::is_same<T, bf16>::value) {
    auto kernel = fm::k_cache_weights_mma<DH>;
    FM_CUDA(fm::set_smem_once(kernel, fm::WmCfg<DH>::SMEM));
    FM_LAUNCH_OK("cache weights", fm::launch_pdl(kernel, grid(fm::WM_KEYS), dim3(fm::WM_THREADS),
                                                 fm::WmCfg<DH>::SMEM, st, k));
  } else {
    FM_LAUNCH_OK("cache weights", fm::launch_pdl(fm::k_cache_weights<T, DH>, grid(fm::CW_THREADS / 32),
                                                 dim3(fm::CW_THREADS), 0, st, k));
  }
  return FM_OK;
}

}  // namespace

extern "C" fm_status fm_cache_attention_workspace(const fm_paged_cache* c,
                                                  const fm_attention_args* a, size_t* bytes) {
  if (!bytes) return set_err(FM_ERR_ARG, "NULL argument");
  FM_TRY(check_attention(c, a));
  AttnPlan p;
  FM_TRY(plan_attention(c, a, &p));
  *bytes = p.total;
  return FM_OK;
}

extern "C" fm_status fm_cache_attention(const fm_paged_cache* c, const fm_attention_args* a,
                                        void* ws, size_t ws_bytes, fm_stream stream) {
  FM_TRY(check_attention(c, a));
  if (!a->cu_rows || !a->kv_len) return set_err(FM_ERR_ARG, "NULL argument");
  FM_TRY(check_aligned4("cu_rows, kv_len, q_pos and lse", a->cu_rows, a->kv_len, a->q_pos, a->lse));
  if (!(a->scale > 0.f) || a->scale > 1e30f)
    return set_err(FM_ERR_ARG, "scale must be finite and > 0");
  if (c->pos && !a->q_pos) return set_err(FM_ERR_ARG, "a cache with positions needs q_pos");
  if (a->T == 0) return FM_OK;
  FM_TRY(check_stride(c, "q", a->q, a->q_stride, a->n_heads, a->T));
  FM_TRY(check_stride(c, "out", a->out, a->out_stride, a->n_heads, a->T));
  const RowSet out = row_set(c, a->out, a->out_stride, a->n_heads, a->T);
  const RowSet lse = {(uintptr_t)a->lse, a->n_heads * 4, a->n_heads * 4, a->T};
  const RowSet q = row_set(c, a->q, a->q_stride, a->n_heads, a->T);
  if (overlap(out, q) || (a->lse && (overlap(lse, out) || overlap(lse, q))))
    return set_err(FM_ERR_ARG, "q, out and lse must not overlap");
  if (!ws || ((uintptr_t)ws & 255)) return set_err(FM_ERR_ARG, "workspace must be 256-byte aligned");
  AttnPlan p;
  FM_TRY(plan_attention(c, a, &p));
  if (ws_bytes < p.total)
    return set_err(FM_ERR_ARG, "workspace of %zu bytes, %zu needed", ws_bytes, p.total);
  fm::CacheAttnArgs k;
  k.c = view(c);
  k.T = a->T;
  k.B = a->B;
  k.n_heads = a->n_heads;
  k.G = a->n_heads / c->n_kv_heads;
  k.max_rows = a->max_rows;
  k.max_kv = a->max_kv;
  k.rt = p.rt;
  k.tile_rows = p.tile_rows;
  k.ov = p.ov;
  k.max_tiles = (int)p.tiles;
  k.q = a->q;
  k.qs = a->q_stride;
  k.os = a->out_stride;
  k.cu = a->cu_rows;
  k.kv_len = a->kv_len;
  k.q_pos = c->pos ? a->q_pos : nullptr;
  k.scale_log2 = a->scale * 1.4426950408889634f;
  k.window = a->window;
  k.sinks = a->sinks;
  k.out = a->out;
  char* w = (char*)ws;
  k.lse = a->lse ? a->lse : a->accumulate ? (float*)(w + p.o_lse) : nullptr;
  k.plan_n = (int*)w;
  k.plan_first = (int*)(w + p.o_first);
  k.plan_tile = (int4*)(w + p.o_tile);
  k.plan_join = (int4*)(w + p.o_join);
  k.part_ml = (float2*)(w + p.o_ml);
  k.part = (float*)(w + p.o_part);
  k.scores = (float*)(w + p.o_scores);
  k.score_units = p.score_units;
  cudaStream_t st = (cudaStream_t)stream;
  if (c->dtype == FM_BF16)
    return c->head_dim == 128 ? run_attention<bf16, 128>(k, p, a->accumulate, st)
                              : run_attention<bf16, 64>(k, p, a->accumulate, st);
  if (c->head_dim == 128) return run_attention<float, 128>(k, p, a->accumulate, st);
  return c->head_dim == 64 ? run_attention<float, 64>(k, p, a->accumulate, st)
                           : run_attention<float, 32>(k, p, a->accumulate, st);
}

// ------------------------------------------------------------------ evict
extern "C" fm_status fm_cache_evict(const fm_paged_cache* c, const int32_t* kv_len,
                                    const int32_t* next_pos, int B, int max_kv, int budget, int sinks,
                                    int recent, int32_t* new_len, fm_stream stream) {
  FM_TRY(check_cache(c));
  if (!kv_len || !next_pos || !new_len) return set_err(FM_ERR_ARG, "NULL argument");
  FM_TRY(check_aligned4("kv_len, next_pos and new_len", kv_len, next_pos, new_len));
  if (!c->pos || !c->weight) return set_err(FM_ERR_ARG, "eviction needs cache->pos and cache->weight");
  if (B < 1 || max_kv < 1 || budget < 1) return set_err(FM_ERR_ARG, "sizes must be positive");
  if (B > FM_MAX_CALL_SEQS)
    return set_err(FM_ERR_UNSUPPORTED, "B=%d exceeds %d sequences", B, FM_MAX_CALL_SEQS);
  if (max_kv > FM_MAX_EVICT_ROWS)
    return set_err(FM_ERR_UNSUPPORTED, "max_kv %d exceeds %d", max_kv, FM_MAX_EVICT_ROWS);
  if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return set_err(FM_ERR_ARG, "sinks %d and recent %d must not be negative nor exceed the budget %d",
                   sinks, recent, budget);
  // a sequence's CTAs read its length and position while the first of them writes
  for (const int32_t* in : {kv_len, next_pos})
    if ((uintptr_t)new_len < (uintptr_t)(in + B) && (uintptr_t)in < (uintptr_t)(new_len + B))
      return set_err(FM_ERR_ARG, "new_len must not overlap kv_len or next_pos");
  fm::EvictArgs k;
  k.c = view(c);
  k.kv_len = kv_len;
  k.next_pos = next_pos;
  k.new_len = new_len;
  k.max_kv = max_kv;
  k.budget = budget;
  k.sinks = sinks;
  k.recent = recent;
  k.row_bytes = c->head_dim * esize(c);
  // CTAs per (sequence, head): a second wave of them never pays for the
  // barriers (64 pairs of 16,384 rows: 4 CTAs each 66 us, 8 94 us, 2 82 us),
  // nor do slices under 2,048 rows (64 pairs of 4,096: 2 CTAs 46 us, 1 60, 4
  // 60); below that, more CTAs share the rows (8 pairs of 16,384: 8 CTAs 38 us,
  // 4 44, 2 62)
  int sms = 0;
  FM_TRY(device_sms(&sms));
  int C = 1;
  while (C < fm::EV_MAX_CLUSTER &&
         ((max_kv + C - 1) / C > fm::EV_SLICE ||
          ((max_kv + C - 1) / C > 2048 && (int64_t)B * c->n_kv_heads * C <= sms)))
    C *= 2;
  k.slice_cap = ((max_kv + C - 1) / C + 127) & ~63;
  static_assert(FM_MAX_EVICT_ROWS <= fm::EV_SLICE * fm::EV_MAX_CLUSTER, "slice");
  FM_CUDA(fm::set_smem_once(fm::k_cache_evict, fm::evict_smem(fm::EV_SLICE + 128)));
  FM_LAUNCH_OK("cache evict",
               fm::launch_pdl_cluster(fm::k_cache_evict, dim3((unsigned)(B * c->n_kv_heads * C)),
                                      dim3(fm::EV_THREADS), (size_t)fm::evict_smem(k.slice_cap),
                                      (cudaStream_t)stream, (unsigned)C, k));
  return FM_OK;
}
