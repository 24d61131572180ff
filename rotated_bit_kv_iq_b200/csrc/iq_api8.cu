// extern "C" entry points of the 8-bit cache, rotary positions and pages: argument checks and dispatch.
#include <cuda_runtime.h>

#include <cmath>

#include "iq_internal8.h"

namespace iq {

static bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static bool dtype_ok(int d) { return d == IQ_F16 || d == IQ_F32 || d == IQ_BF16; }

static iq_status check_cache8(const iq_cache8* c, int32_t layer) {
  if (!c) return IQ_ERR_INVALID_ARG;
  if (c->head_dim != D) return IQ_ERR_UNSUPPORTED;
  if (c->n_layers < 1 || c->n_kv_heads < 1 || c->page_size < TILE_TOKENS || c->page_size % TILE_TOKENS != 0 ||
      c->n_pages < 1)
    return IQ_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->n_layers || !c->pool) return IQ_ERR_INVALID_ARG;
  if (c->block_table_dev && c->max_pages_per_seq < 1) return IQ_ERR_INVALID_ARG;
  if (c->code != IQ_E4M3 && c->code != IQ_S8) return IQ_ERR_UNSUPPORTED;
  if (!aligned_to(c->pool, 16) || !aligned_to(c->block_table_dev, 4) || !aligned_to(c->status_dev, 4))
    return IQ_ERR_ALIGNMENT;
  return IQ_OK;
}

static View8 view8(const iq_cache8* c, int32_t layer) {
  View8 v;
  v.pool = (uint8_t*)c->pool +
           (size_t)layer * c->n_pages * c->n_kv_heads * (c->page_size / TILE_TOKENS) * (size_t)TILE8_BYTES;
  v.block_table = c->block_table_dev;
  v.max_pages = c->block_table_dev ? c->max_pages_per_seq : 1;
  v.page_size = c->page_size;
  v.n_pages = c->n_pages;
  v.n_kv_heads = c->n_kv_heads;
  v.status = c->status_dev;
  v.code = c->code;
  return v;
}

static int64_t capacity8(const iq_cache8* c) {
  return (int64_t)c->page_size * (c->block_table_dev ? c->max_pages_per_seq : 1);
}

// The kernels count tiles of a sequence's heads, and steps of a prefill call, in 32 bits.
static bool context_ok(const iq_cache8* c, int32_t max_ctx) {
  return max_ctx <= 1 << 30 && (int64_t)max_ctx * c->n_kv_heads <= (int64_t)1 << 35;
}
static bool prefill_ok(const iq_cache8* c, int32_t batch, int32_t n_tokens, int32_t n_q_heads, int32_t max_ctx) {
  const int64_t rows = (int64_t)batch * c->n_kv_heads * n_tokens;
  if (rows > (int64_t)1 << 27 || !context_ok(c, max_ctx)) return false;
  const int32_t tq = 256 / (n_q_heads / c->n_kv_heads);
  return (int64_t)batch * c->n_kv_heads * ((n_tokens + tq - 1) / tq) * ((int64_t)max_ctx / 128 + 1) < (int64_t)1 << 31;
}

static iq_status check_heads(const iq_cache8* c, int32_t n_q_heads) {
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads != 0) return IQ_ERR_INVALID_ARG;
  return n_q_heads / c->n_kv_heads > 8 ? IQ_ERR_UNSUPPORTED : IQ_OK;
}

static iq_status check_pages(const iq_pages* p) {
  if (!p || !p->block_table_dev || !p->seq_len_dev || !p->ref_dev) return IQ_ERR_INVALID_ARG;
  if (p->max_seqs < 1 || p->max_pages_per_seq < 1 || p->n_pages < 1 || p->page_size < TILE_TOKENS ||
      p->page_size % TILE_TOKENS != 0)
    return IQ_ERR_INVALID_ARG;
  if (!aligned_to(p->block_table_dev, 4) || !aligned_to(p->seq_len_dev, 4) || !aligned_to(p->ref_dev, 4) ||
      !aligned_to(p->status_dev, 4))
    return IQ_ERR_ALIGNMENT;
  return IQ_OK;
}

static iq_status check_list(const void* a, const void* b, int32_t n) {
  if (n < 0 || (n > 0 && (!a || !b))) return IQ_ERR_INVALID_ARG;
  if (n > IQ_PAGES_MAX_LIST) return IQ_ERR_UNSUPPORTED;
  return aligned_to(a, 4) && aligned_to(b, 4) ? IQ_OK : IQ_ERR_ALIGNMENT;
}

static iq_status check_pools(const iq_page_pool* pools, int32_t n, PagePools* out) {
  if (n < 0 || n > PAGES_MAX_POOLS || (n > 0 && !pools)) return IQ_ERR_INVALID_ARG;
  out->n = n;
  for (int i = 0; i < n; ++i) {
    if (!pools[i].pool || pools[i].n_layers < 1 || pools[i].n_kv_heads < 1 || pools[i].tile_bytes < 16 ||
        pools[i].tile_bytes % 16 != 0)
      return IQ_ERR_INVALID_ARG;
    if (!aligned_to(pools[i].pool, 16)) return IQ_ERR_ALIGNMENT;
    out->base[i] = (uint8_t*)pools[i].pool;
    out->n_layers[i] = pools[i].n_layers;
    out->n_kv_heads[i] = pools[i].n_kv_heads;
    out->tile_bytes[i] = pools[i].tile_bytes;
  }
  return IQ_OK;
}

static iq_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need) return IQ_ERR_WORKSPACE;
  return aligned_to(ws, 256) ? IQ_OK : IQ_ERR_ALIGNMENT;
}

static iq_status result(int e) { return e ? IQ_ERR_CUDA : IQ_OK; }

}  // namespace iq

using namespace iq;

#define IQ_TRY(expr)                        \
  do {                                      \
    const iq_status st_ = (expr);           \
    if (st_ != IQ_OK) return st_;           \
  } while (0)

extern "C" {

iq_status iq_cache8_bytes(int32_t n_layers, int32_t n_kv_heads, int32_t page_size, int32_t n_pages,
                          size_t* pool_bytes_host) {
  if (n_layers < 1 || n_kv_heads < 1 || page_size < TILE_TOKENS || page_size % TILE_TOKENS != 0 || n_pages < 1)
    return IQ_ERR_INVALID_ARG;
  if (pool_bytes_host)
    *pool_bytes_host = (size_t)n_layers * n_pages * n_kv_heads * (page_size / TILE_TOKENS) * (size_t)TILE8_BYTES;
  return IQ_OK;
}

iq_status iq_append8(const iq_cache8* cache, int32_t layer, const void* k_dev, const void* v_dev, iq_dtype dtype,
                     int64_t k_stride, int64_t v_stride, int32_t batch, int32_t n_new, const int32_t* start_pos_dev,
                     const int32_t* n_valid_dev, iq_stream_t stream) {
  IQ_TRY(check_cache8(cache, layer));
  if (batch < 0 || n_new < 0 || !start_pos_dev || (!k_dev && !v_dev)) return IQ_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return IQ_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)cache->n_kv_heads * D;
  if (k_stride == 0) k_stride = row;
  if (v_stride == 0) v_stride = row;
  if (k_stride < row || k_stride % 8 != 0 || v_stride < row || v_stride % 8 != 0) return IQ_ERR_INVALID_ARG;
  if (!cache->block_table_dev && batch > cache->n_pages) return IQ_ERR_CAPACITY;
  if ((int64_t)n_new > capacity8(cache)) return IQ_ERR_CAPACITY;
  if (!aligned_to(k_dev, 16) || !aligned_to(v_dev, 16) || !aligned_to(start_pos_dev, 4) || !aligned_to(n_valid_dev, 4))
    return IQ_ERR_ALIGNMENT;
  return result(launch_append8(view8(cache, layer), k_dev, v_dev, dtype, k_stride, v_stride, batch, n_new,
                               start_pos_dev, n_valid_dev, stream));
}

size_t iq_decode8_workspace_size(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t max_ctx) {
  if (batch < 0 || n_q_heads < 0 || n_kv_heads < 1 || max_ctx < 0) return 0;
  return decode8_workspace_bytes(batch, n_kv_heads);
}

iq_status iq_decode8_attention(const iq_cache8* cache, int32_t layer, const void* q_dev, iq_dtype dtype, int32_t batch,
                               int32_t n_q_heads, const int32_t* ctx_len_dev, int32_t max_ctx, float scale,
                               void* out_dev, void* workspace_dev, size_t workspace_bytes, iq_stream_t stream) {
  IQ_TRY(check_cache8(cache, layer));
  if (batch < 0 || max_ctx < 0 || !q_dev || !ctx_len_dev || !out_dev) return IQ_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.f) return IQ_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || batch > DECODE_MAX_BATCH) return IQ_ERR_UNSUPPORTED;
  IQ_TRY(check_heads(cache, n_q_heads));
  if (!cache->block_table_dev && batch > cache->n_pages) return IQ_ERR_CAPACITY;
  if ((int64_t)max_ctx > capacity8(cache)) return IQ_ERR_CAPACITY;
  if (!context_ok(cache, max_ctx)) return IQ_ERR_UNSUPPORTED;
  if (!aligned_to(q_dev, 16) || !aligned_to(out_dev, 16) || !aligned_to(ctx_len_dev, 4)) return IQ_ERR_ALIGNMENT;
  IQ_TRY(check_ws(workspace_dev, workspace_bytes, decode8_workspace_bytes(batch, cache->n_kv_heads)));
  return result(launch_decode8(view8(cache, layer), q_dev, dtype, batch, n_q_heads, ctx_len_dev, max_ctx, scale, out_dev,
                               workspace_dev, stream));
}

size_t iq_prefill8_workspace_size(int32_t batch, int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads,
                                  int32_t max_ctx) {
  if (batch < 0 || n_tokens < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads || max_ctx < 0) return 0;
  return prefill8_workspace_bytes(batch, n_tokens, n_q_heads, n_kv_heads, max_ctx);
}

iq_status iq_prefill8_attention(const iq_cache8* cache, int32_t layer, const void* q_dev, iq_dtype dtype, int32_t batch,
                                int32_t n_tokens, int32_t n_q_heads, const int32_t* start_pos_dev,
                                const int32_t* n_valid_dev, int32_t max_ctx, float scale, void* out_dev,
                                void* workspace_dev, size_t workspace_bytes, iq_stream_t stream) {
  IQ_TRY(check_cache8(cache, layer));
  if (batch < 0 || n_tokens < 0 || max_ctx < n_tokens || !q_dev || !start_pos_dev || !out_dev) return IQ_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.f) return IQ_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return IQ_ERR_UNSUPPORTED;
  IQ_TRY(check_heads(cache, n_q_heads));
  if (!cache->block_table_dev && batch > cache->n_pages) return IQ_ERR_CAPACITY;
  if ((int64_t)max_ctx > capacity8(cache)) return IQ_ERR_CAPACITY;
  if (!prefill_ok(cache, batch, n_tokens, n_q_heads, max_ctx)) return IQ_ERR_UNSUPPORTED;
  if (!aligned_to(q_dev, 16) || !aligned_to(out_dev, 16) || !aligned_to(start_pos_dev, 4) || !aligned_to(n_valid_dev, 4))
    return IQ_ERR_ALIGNMENT;
  IQ_TRY(check_ws(workspace_dev, workspace_bytes,
                  prefill8_workspace_bytes(batch, n_tokens, n_q_heads, cache->n_kv_heads, max_ctx)));
  return result(launch_prefill8(view8(cache, layer), q_dev, dtype, batch, n_tokens, n_q_heads, start_pos_dev, n_valid_dev,
                                max_ctx, scale, out_dev, workspace_dev, stream));
}

iq_status iq_export8(const iq_cache8* cache, int32_t layer, int32_t kv, int32_t seq, int32_t t0, int32_t n,
                     float* values_dev, iq_stream_t stream) {
  IQ_TRY(check_cache8(cache, layer));
  if ((kv != 0 && kv != 1) || seq < 0 || t0 < 0 || n < 0 || !values_dev) return IQ_ERR_INVALID_ARG;
  if (!cache->block_table_dev && seq >= cache->n_pages) return IQ_ERR_CAPACITY;
  if ((int64_t)t0 + n > capacity8(cache)) return IQ_ERR_CAPACITY;
  if (!aligned_to(values_dev, 16)) return IQ_ERR_ALIGNMENT;
  return result(launch_export8(view8(cache, layer), kv, seq, t0, n, values_dev, stream));
}

iq_status iq_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor, double original_len,
                              double low, double high, double* freq_host, double* mscale_host) {
  if (!freq_host || !mscale_host) return IQ_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0) return IQ_ERR_UNSUPPORTED;
  if (scaling < IQ_ROPE_PLAIN || scaling > IQ_ROPE_YARN) return IQ_ERR_UNSUPPORTED;
  if (!(std::isfinite(base) && base > 1.0)) return IQ_ERR_INVALID_ARG;
  if (scaling != IQ_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return IQ_ERR_INVALID_ARG;
  const bool bands = scaling == IQ_ROPE_BANDS || scaling == IQ_ROPE_YARN;
  if (bands && !(std::isfinite(original_len) && original_len > 0.0 && std::isfinite(high) && low > 0.0 && low < high))
    return IQ_ERR_INVALID_ARG;
  if (scaling == IQ_ROPE_NTK) {
    if (rotary_dim <= 2) return IQ_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
  }
  const double two_pi = 6.283185307179586476925;
  // index of the pair that makes n turns within the original length (not whole)
  auto index_of = [&](double n) { return rotary_dim * std::log(original_len / (n * two_pi)) / (2.0 * std::log(base)); };
  double i0 = 0.0, i1 = 1.0;
  if (scaling == IQ_ROPE_YARN) {
    i0 = std::fmax(std::floor(index_of(high)), 0.0);
    i1 = std::fmin(std::ceil(index_of(low)), rotary_dim - 1.0);
    if (i1 <= i0) i1 = i0 + 0.001;  // a step
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1.0;  // share of f, the rest being f / factor
    if (scaling == IQ_ROPE_LINEAR) keep = 0.0;
    if (scaling == IQ_ROPE_BANDS) keep = (original_len * f / two_pi - low) / (high - low);
    if (scaling == IQ_ROPE_YARN) keep = 1.0 - (i - i0) / (i1 - i0);
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    freq_host[i] = scaling == IQ_ROPE_PLAIN || scaling == IQ_ROPE_NTK ? f : f * keep + f / factor * (1.0 - keep);
  }
  *mscale_host = scaling == IQ_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return IQ_OK;
}

iq_status iq_rope(const void* q_dev, int64_t q_stride, void* q_out_dev, int64_t q_out_stride, const void* k_dev,
                  int64_t k_stride, void* k_out_dev, int64_t k_out_stride, iq_dtype dtype, int32_t n_tokens,
                  int32_t n_q_heads, int32_t n_kv_heads, int32_t rotary_dim, int32_t layout,
                  const int32_t* positions_dev, const double* freq_dev, float mscale, int32_t inverse,
                  iq_stream_t stream) {
  if ((!q_dev && !k_dev) || (!q_dev != !q_out_dev) || (!k_dev != !k_out_dev)) return IQ_ERR_INVALID_ARG;
  if (n_tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 || !positions_dev || !freq_dev) return IQ_ERR_INVALID_ARG;
  if ((q_dev && n_q_heads < 1) || (k_dev && n_kv_heads < 1) || !std::isfinite(mscale)) return IQ_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (layout != IQ_ROPE_HALF && layout != IQ_ROPE_INTERLEAVED)) return IQ_ERR_UNSUPPORTED;
  if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0) return IQ_ERR_UNSUPPORTED;
  if ((int64_t)n_q_heads + n_kv_heads > 1 << 20) return IQ_ERR_UNSUPPORTED;
  RopeArgs a;
  const void* x[2] = {q_dev, k_dev};
  void* y[2] = {q_out_dev, k_out_dev};
  const int64_t xs[2] = {q_stride, k_stride}, ys[2] = {q_out_stride, k_out_stride};
  const int heads[2] = {n_q_heads, n_kv_heads};
  for (int i = 0; i < 2; ++i) {
    const int64_t row = (int64_t)heads[i] * D;
    a.x[i] = x[i];
    a.y[i] = y[i];
    a.heads[i] = x[i] ? heads[i] : 0;
    a.xs[i] = xs[i] ? xs[i] : row;
    a.ys[i] = ys[i] ? ys[i] : row;
    if (!x[i]) continue;
    if (a.xs[i] < row || a.ys[i] < row || a.xs[i] % 8 != 0 || a.ys[i] % 8 != 0) return IQ_ERR_INVALID_ARG;
    if (x[i] == y[i] && a.xs[i] != a.ys[i] && n_tokens > 1) return IQ_ERR_INVALID_ARG;
    if (!aligned_to(x[i], 16) || !aligned_to(y[i], 16)) return IQ_ERR_ALIGNMENT;
  }
  if (!aligned_to(positions_dev, 4) || !aligned_to(freq_dev, 8)) return IQ_ERR_ALIGNMENT;
  a.n_tokens = n_tokens;
  a.rd = rotary_dim;
  a.layout = layout;
  a.inverse = inverse;
  a.pos = positions_dev;
  a.freq = freq_dev;
  a.mscale = mscale;
  return result(launch_rope(a, dtype, stream));
}

size_t iq_pages_workspace_size(const iq_pages* pages) {
  return check_pages(pages) == IQ_OK ? pages_workspace_bytes(*pages) : 0;
}

iq_status iq_pages_extend(const iq_pages* pages, const int32_t* ids_dev, const int32_t* new_len_dev, int32_t n,
                          void* workspace_dev, size_t workspace_bytes, iq_stream_t stream) {
  IQ_TRY(check_pages(pages));
  IQ_TRY(check_list(ids_dev, new_len_dev, n));
  IQ_TRY(check_ws(workspace_dev, workspace_bytes, pages_workspace_bytes(*pages)));
  return result(launch_pages_extend(*pages, ids_dev, new_len_dev, n, workspace_dev, stream));
}

iq_status iq_pages_free(const iq_pages* pages, const int32_t* ids_dev, int32_t n, iq_stream_t stream) {
  IQ_TRY(check_pages(pages));
  IQ_TRY(check_list(ids_dev, ids_dev, n));
  return result(launch_pages_free(*pages, ids_dev, n, stream));
}

iq_status iq_pages_fork(const iq_pages* pages, const iq_page_pool* pools_host, int32_t n_pools,
                        const int32_t* parent_dev, const int32_t* child_dev, int32_t n, void* workspace_dev,
                        size_t workspace_bytes, iq_stream_t stream) {
  PagePools pools;
  IQ_TRY(check_pages(pages));
  IQ_TRY(check_pools(pools_host, n_pools, &pools));
  IQ_TRY(check_list(parent_dev, child_dev, n));
  IQ_TRY(check_ws(workspace_dev, workspace_bytes, pages_workspace_bytes(*pages)));
  return result(launch_pages_fork(*pages, pools, parent_dev, child_dev, n, workspace_dev, stream));
}

iq_status iq_pages_compact(const iq_pages* pages, const iq_page_pool* pools_host, int32_t n_pools,
                           int32_t* n_held_dev, void* workspace_dev, size_t workspace_bytes, iq_stream_t stream) {
  PagePools pools;
  IQ_TRY(check_pages(pages));
  IQ_TRY(check_pools(pools_host, n_pools, &pools));
  if (!aligned_to(n_held_dev, 4)) return IQ_ERR_ALIGNMENT;
  IQ_TRY(check_ws(workspace_dev, workspace_bytes, pages_workspace_bytes(*pages)));
  return result(launch_pages_compact(*pages, pools, n_held_dev, workspace_dev, stream));
}

iq_status iq_pages_copy(const iq_pages* pages, const iq_page_pool* pools_host, int32_t n_pools,
                        const int32_t* src_dev, const int32_t* dst_dev, int32_t n, void* workspace_dev,
                        size_t workspace_bytes, iq_stream_t stream) {
  PagePools pools;
  IQ_TRY(check_pages(pages));
  IQ_TRY(check_pools(pools_host, n_pools, &pools));
  IQ_TRY(check_list(src_dev, dst_dev, n));
  IQ_TRY(check_ws(workspace_dev, workspace_bytes, pages_workspace_bytes(*pages)));
  return result(launch_pages_copy(*pages, pools, src_dev, dst_dev, n, workspace_dev, stream));
}

}  // extern "C"
