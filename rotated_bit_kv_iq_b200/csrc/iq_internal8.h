// Internal declarations of the 8-bit cache, rotary positions and pages.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/iq8.h"
#include "iq_internal.h"

namespace iq {

constexpr int TILE8_BYTES = IQ_TILE8_BYTES;
constexpr int TILE8_V = TILE_TOKENS * D;           // byte offset of the V rows
constexpr int TILE8_SCALES = 2 * TILE_TOKENS * D;  // byte offset of the K and V scales
static_assert(TILE8_SCALES + 32 == TILE8_BYTES, "8-bit tile record");

// Device geometry of one layer of an 8-bit cache, resolved on the host.
struct View8 {
  uint8_t* pool;               // layer base
  const int32_t* block_table;  // NULL -> sequence b uses page b
  int32_t max_pages;           // pages per sequence (1 when the table is NULL)
  int32_t page_size, n_pages, n_kv_heads;
  uint32_t* status;
  int32_t code;
};

int launch_append8(const View8& v, const void* k, const void* vsrc, int dtype, long long ks, long long vs, int batch, int n_new,
                   const int32_t* start, const int32_t* n_valid, void* stream);
size_t decode8_workspace_bytes(int batch, int n_kv_heads);
int launch_decode8(const View8& v, const void* q, int dtype, int batch, int n_q_heads, const int32_t* ctx_len,
                   int max_ctx, float scale, void* out, void* workspace, void* stream);
size_t chunk8_workspace_bytes(int batch, int n_tok, int g, int n_kv_heads);
int launch_chunk8(const View8& v, const void* q, int dtype, int batch, int n_tok, int n_q_heads, const int32_t* start,
                  const int32_t* n_valid, int max_ctx, float scale, void* out, void* workspace, void* stream);
size_t prefill8_workspace_bytes(int batch, int n_tok, int n_q_heads, int n_kv_heads, int max_ctx);
int launch_prefill8(const View8& v, const void* q, int dtype, int batch, int n_tok, int n_q_heads, const int32_t* start,
                    const int32_t* n_valid, int max_ctx, float scale, void* out, void* workspace, void* stream);
int launch_export8(const View8& v, int kv, int seq, int t0, int n, float* values, void* stream);

struct RopeArgs {
  const void* x[2];  // q, k
  void* y[2];
  long long xs[2], ys[2];  // row strides, elements
  int heads[2];            // 0: absent
  int n_tokens, rd, layout, inverse;
  const int32_t* pos;
  const double* freq;
  float mscale;
};
int launch_rope(const RopeArgs& a, int dtype, void* stream);

constexpr int PAGES_MAX_POOLS = 8;
struct PagePools {
  uint8_t* base[PAGES_MAX_POOLS];
  int n_layers[PAGES_MAX_POOLS];
  int n_kv_heads[PAGES_MAX_POOLS];
  int tile_bytes[PAGES_MAX_POOLS];
  int n;
};
int launch_pages_extend(const iq_pages& p, const int32_t* ids, const int32_t* len, int n, void* ws, void* stream);
int launch_pages_free(const iq_pages& p, const int32_t* ids, int n, void* stream);
int launch_pages_fork(const iq_pages& p, const PagePools& pools, const int32_t* parent, const int32_t* child, int n,
                      void* ws, void* stream);
int launch_pages_compact(const iq_pages& p, const PagePools& pools, int32_t* n_held, void* ws, void* stream);
int launch_pages_copy(const iq_pages& p, const PagePools& pools, const int32_t* src, const int32_t* dst, int n,
                      void* ws, void* stream);
size_t pages_workspace_bytes(const iq_pages& p);

}  // namespace iq
