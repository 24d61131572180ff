/*
 * iq8.h -- C ABI of libiq beside the packed cache of iq.h: a cache in 8 bits and attention over it,
 * rotary positions of q and k, and the operations on the pages of either cache.  The conventions of
 * iq.h hold: device memory is the caller's, calls are asynchronous on the stream, nothing is allocated,
 * argument errors are returned before any launch, bad data on the device is skipped and flagged.
 */
#ifndef IQ8_H
#define IQ8_H

#include "iq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third number type, for the calls declared here only (IQ_ERR_UNSUPPORTED elsewhere). */
#define IQ_BF16 ((iq_dtype)2)

/* More bits of *status_dev. */
#define IQ_DEVERR_SEQ 32u /* page operation: sequence id outside the table, listed twice, or not empty */
#define IQ_DEVERR_NOPAGE 64u /* page operation: no free page left, or a sequence longer than its table row */

#define IQ_DEVERR_RANGE 128u /* prefill: V scales of a sequence too far apart (those rows may be wrong) */

/* ------------------------------------------------------------------ the 8-bit cache
 * A cache whose K and V are held in 8 bits, unrotated (no block rotation), with one scale for each block of 32 tokens
 * and kv head (K and V apart).  The calls beside it have the conventions above (asynchronous on the
 * stream, nothing allocated, argument errors before any launch, bad data skipped and flagged).
 *
 * Layout: one pool, [L][n_pages][Hkv][page_size/32] tile records of IQ_TILE8_BYTES = 8224 bytes; the
 * record of slots s0..s0+31 (s0 a multiple of 32) holds
 *     bytes [0, 4096)      K: row s (slot s0 + s) of 128 codes, in 16-byte chunks: chunk c (coordinates
 *                          16c..16c+15) at byte 128 s + 16 (c ^ (s mod 8))
 *     bytes [4096, 8192)   V, likewise
 *     bytes [8192, 8200)   float32 K scale, float32 V scale; the other 24 bytes are not used
 * The value of a code is code * scale:
 *     IQ_E4M3: code = e4m3 number; scale = 2^e, the smallest e >= -100 with amax <= 448 2^e;
 *     IQ_S8:   code = -127..127;   scale = amax / 127 rounded up to 8 significant bits, at least 2^-100;
 * amax the largest finite magnitude that the block was given.  Codes are the nearest (ties to even)
 * numbers of their type to x / scale; a NaN becomes 0, an infinity the largest code of its sign.
 * Pages and block tables are those of iq_cache. */
typedef enum { IQ_E4M3 = 0, IQ_S8 = 1 } iq_code8;
#define IQ_TILE8_BYTES 8224

typedef struct {
  void* pool;                      /* device, tile records, 16-byte aligned */
  int32_t n_layers;                /* L >= 1 */
  int32_t n_kv_heads;              /* Hkv >= 1 */
  int32_t head_dim;                /* must be 128 */
  int32_t page_size;               /* tokens per page, multiple of 32 */
  int32_t n_pages;                 /* pages in the pool */
  const int32_t* block_table_dev;  /* [batch][max_pages_per_seq] or NULL (sequence b owns page b) */
  int32_t max_pages_per_seq;       /* ignored when block_table_dev is NULL */
  uint32_t* status_dev;            /* device word for IQ_DEVERR_* bits, or NULL */
  int32_t code;                    /* iq_code8 */
} iq_cache8;

/* Bytes of an 8-bit cache's pool (host-only; errors as iq_cache_bytes). */
iq_status iq_cache8_bytes(int32_t n_layers, int32_t n_kv_heads, int32_t page_size, int32_t n_pages,
                          size_t* pool_bytes_host);

/* Quantise-and-append: up to n_new new tokens of every sequence into layer `layer`.
 *   k_dev, v_dev : [batch][n_new][Hkv][128] of `dtype` (IQ_F16, IQ_BF16 or IQ_F32); either may be
 *                  NULL (that side skipped).  Token i of sequence b is row b n_new + i, at that times
 *                  k_stride, v_stride elements (0: Hkv * 128; at least that and a multiple of 8), so
 *                  that they may be slices of a fused projection's rows.
 *   start_pos_dev: int32 [batch], position of each sequence's first new token.
 *   n_valid_dev  : int32 [batch] or NULL: only the first n_valid[b] (clamped to 0..n_new, flagged
 *                  with IQ_DEVERR_CTX) of the n_new tokens of sequence b are there.
 * A block that already holds tokens before start_pos keeps its scale unless the new tokens need a
 * larger one; then those tokens' codes are rounded again, from the values that they stood for, to
 * the larger scale.  Tokens at and behind start_pos are taken as not there: after the call the
 * positions behind the last appended one hold nothing.
 * (A scale there that is no positive number is taken as nothing: those tokens become 0.)
 * Tokens at positions outside the sequence's pages are skipped (IQ_DEVERR_POSITION,
 * IQ_DEVERR_PAGE).  Two sequences of one call must not append to the same page. */
iq_status iq_append8(const iq_cache8* cache, int32_t layer, const void* k_dev, const void* v_dev, iq_dtype dtype,
                     int64_t k_stride, int64_t v_stride, int32_t batch, int32_t n_new, const int32_t* start_pos_dev,
                     const int32_t* n_valid_dev, iq_stream_t stream);

/* Workspace bytes of iq_decode8_attention on the current device (split partials and counters);
 * zero-filled before its first use, left ready for the next call, as iq_decode_workspace_size's.  One that
 * is large enough for calls of several sizes serves them all in turn; other calls' scratch must not share it. */
size_t iq_decode8_workspace_size(int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t max_ctx);

/* Decode attention over the 8-bit cache of layer `layer`: out[b][h] = sum_t softmax_t(scale <q, K_t>) V_t
 * over tokens 0..ctx_len[b]-1.
 *   q_dev, out_dev : [batch][n_q_heads][128] of `dtype` (IQ_F16, IQ_BF16, IQ_F32); sums in float32.
 *   scale          : finite and > 0 (1/sqrt(128) for plain attention).
 * ctx_len, max_ctx, workspace, batch <= 2048 and the group size of 1..8 as for iq_decode_attention:
 * max_ctx at most 2^30, and 2^35 / Hkv (IQ_ERR_UNSUPPORTED above);
 * ctx_len 0 gives a zero row, values outside [0, max_ctx] are clamped and flagged (IQ_DEVERR_CTX).
 * Tokens of a page outside the pool, and of a record in which nothing was written (a K or V scale that is no positive
 * finite number), are left out and flagged (IQ_DEVERR_PAGE). */
iq_status iq_decode8_attention(const iq_cache8* cache, int32_t layer, const void* q_dev, iq_dtype dtype, int32_t batch,
                               int32_t n_q_heads, const int32_t* ctx_len_dev, int32_t max_ctx, float scale,
                               void* out_dev, void* workspace_dev, size_t workspace_bytes, iq_stream_t stream);

/* Workspace bytes of iq_prefill8_attention on the current device; needs no zeroing. */
size_t iq_prefill8_workspace_size(int32_t batch, int32_t n_tokens, int32_t n_q_heads, int32_t n_kv_heads,
                                  int32_t max_ctx);

/* Causal attention of up to n_tokens query tokens per sequence over the 8-bit cache (their own K and V
 * appended first): query token i of sequence b attends to positions 0 .. start_pos[b] + i.
 *   q_dev, out_dev : [batch][n_tokens][n_q_heads][128] of `dtype`.
 *   n_valid_dev    : int32 [batch] or NULL: only the first n_valid[b] tokens (clamped to 0..n_tokens,
 *                    flagged) are there; the rows of `out` behind them are left as they were.
 *   start_pos      : values outside [0, max_ctx - n_valid[b]] are clamped and flagged.
 * With 16-bit queries the V scales of a sequence's blocks of a kv head are to lie within a factor of 2^104 of
 * each other (a block of zeros has 2^-100); what is farther apart is flagged (IQ_DEVERR_RANGE).  Their softmax weights are
 * rounded to binary16 before the product with V, 2^-11 of each; float32 queries keep 22 bits of theirs.
 * Other arguments as for iq_decode8_attention.  At most 2^27 kv heads' tokens (batch Hkv n_tokens), and 2^31
 * steps of 128 keys by the blocks of 256 / G tokens (IQ_ERR_UNSUPPORTED above). */
iq_status iq_prefill8_attention(const iq_cache8* cache, int32_t layer, const void* q_dev, iq_dtype dtype, int32_t batch,
                                int32_t n_tokens, int32_t n_q_heads, const int32_t* start_pos_dev,
                                const int32_t* n_valid_dev, int32_t max_ctx, float scale, void* out_dev,
                                void* workspace_dev, size_t workspace_bytes, iq_stream_t stream);

/* Read back the values of tokens [t0, t0+n) of sequence `seq` (code * scale) as float32 [Hkv][n][128]
 * (a test and inspection utility, as iq_export_codes); kv: 0 = K, 1 = V; NaN where the page is bad. */
iq_status iq_export8(const iq_cache8* cache, int32_t layer, int32_t kv, int32_t seq, int32_t t0, int32_t n,
                     float* values_dev, iq_stream_t stream);

/* ------------------------------------------------------------------ rotary positions
 * Turns pairs of coordinates of q and k by an angle that grows with the token's position, before they
 * are attended with or appended to either cache. */
typedef enum {
  IQ_ROPE_HALF = 0,        /* pair i: coordinates i and i + rotary_dim/2 */
  IQ_ROPE_INTERLEAVED = 1  /* pair i: coordinates 2i and 2i + 1 */
} iq_rope_layout;

typedef enum {
  IQ_ROPE_PLAIN = 0,  /* f_i = base^(-2i/rotary_dim) */
  IQ_ROPE_LINEAR = 1, /* f_i / factor */
  IQ_ROPE_NTK = 2,    /* base times factor^(rotary_dim / (rotary_dim - 2)) (rotary_dim > 2) */
  IQ_ROPE_BANDS = 3,  /* by turns n_i = original_len f_i / (2 pi) within the trained length: f_i / factor
                         below `low` turns, f_i above `high`, linear in n_i between */
  IQ_ROPE_YARN = 4    /* by the pair's index: f_i above `high` turns, f_i / factor below `low`, linear in i
                         between floor and ceil of the indexes at which these turns are reached;
                         q and k times 0.1 ln(factor) + 1 */
} iq_rope_scaling;

/* Frequencies (radians per position) of the rotary_dim/2 pairs, in double, and the factor on q and k.
 * Host-only.  base > 1, factor >= 1, original_len > 0, 0 < low < high; factor, original_len, low and high
 * are read by the scalings that name them.  IQ_ERR_INVALID_ARG, IQ_ERR_UNSUPPORTED (rotary_dim not even or
 * outside 2..128, unknown scaling). */
iq_status iq_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor, double original_len,
                              double low, double high, double* freq_host, double* mscale_host);

/* (x0, x1) -> mscale (x0 cos a - x1 sin a, x0 sin a + x1 cos a), a = positions[n] freq[i], of the first
 * rotary_dim coordinates of every head; the others are copied.  inverse != 0 turns by -a (the gradient of
 * the call, and, with 1/mscale, its undoing).
 *   q_dev, k_dev       : n_tokens rows of n_q_heads, n_kv_heads heads of 128 of `dtype` (IQ_F16, IQ_BF16,
 *                        IQ_F32); row n at n * q_stride, n * k_stride elements (0: heads * 128; at least
 *                        that and a multiple of 8).  Either may be NULL (with its out).
 *   q_out_dev, k_out_dev: [n_tokens][heads][128], rows of q_out_stride, k_out_stride elements; may be the
 *                        input itself (same pointer and stride), must not overlap it otherwise.
 *   positions_dev      : int32 [n_tokens], any value.
 *   freq_dev           : float64 [rotary_dim/2].  The angle is reduced to one turn in double, so that far
 *                        positions lose nothing; sines, cosines and products are float32. */
iq_status iq_rope(const void* q_dev, int64_t q_stride, void* q_out_dev, int64_t q_out_stride, const void* k_dev,
                  int64_t k_stride, void* k_out_dev, int64_t k_out_stride, iq_dtype dtype, int32_t n_tokens,
                  int32_t n_q_heads, int32_t n_kv_heads, int32_t rotary_dim, int32_t layout,
                  const int32_t* positions_dev, const double* freq_dev, float mscale, int32_t inverse,
                  iq_stream_t stream);

/* ------------------------------------------------------------------ pages
 * The block table of a paged cache and the operations that keep it, on the device: nothing comes back to
 * the host.  One table serves the caches (of either kind) that are given it as block_table_dev.  All calls
 * are deterministic: free pages are taken in ascending order, in the order of the list and of each
 * sequence's pages.  Every call ends with an empty kernel, so that a call that may start early
 * (iq_decode_step, iq_decode_step_deferred) may follow at once. */
typedef struct {
  int32_t* block_table_dev;  /* [max_seqs][max_pages_per_seq]; -1 where there is no page */
  int32_t* seq_len_dev;      /* [max_seqs] tokens */
  int32_t* ref_dev;          /* [n_pages] how many sequences hold the page; 0: free */
  int32_t max_seqs;
  int32_t max_pages_per_seq;
  int32_t page_size;         /* multiple of 32 */
  int32_t n_pages;
  uint32_t* status_dev;      /* device word for IQ_DEVERR_* bits, or NULL */
} iq_pages;

/* A pool whose pages the table names: page p of layer l is n_kv_heads * page_size/32 tile records of
 * tile_bytes (a multiple of 16) at pool + (l n_pages + p) * n_kv_heads * (page_size/32) * tile_bytes. */
typedef struct {
  void* pool;
  int32_t n_layers;
  int32_t n_kv_heads;
  int32_t tile_bytes;
} iq_page_pool;

/* Workspace bytes of the calls below (no zeroing needed; calls that overlap must not share one). */
size_t iq_pages_workspace_size(const iq_pages* pages);

/* Most entries of one list (IQ_ERR_UNSUPPORTED above). */
#define IQ_PAGES_MAX_LIST 4096

/* Sequence ids[i] grows to new_len[i] tokens and gets the pages for them.  new_len at or below its length
 * changes nothing.  When the free pages run out, that entry and every later one is refused; a length past
 * the row's capacity is refused (both IQ_DEVERR_NOPAGE).  Refused entries leave no trace.  An id outside
 * the table, or listed before, is refused (IQ_DEVERR_SEQ). */
iq_status iq_pages_extend(const iq_pages* pages, const int32_t* ids_dev, const int32_t* new_len_dev, int32_t n,
                          void* workspace_dev, size_t workspace_bytes, iq_stream_t stream);

/* Sequences ids[0..n) end: their pages lose a holder, their rows become -1, their lengths 0. */
iq_status iq_pages_free(const iq_pages* pages, const int32_t* ids_dev, int32_t n, iq_stream_t stream);

/* Sequence child[i] (empty) becomes a copy of sequence parent[i]: it shares the parent's full pages and gets
 * a copy, in every layer of every pool, of the tile records in use of the last, part-filled one.  Entries
 * read the table as it was before the call.  A child that is not empty, is listed before, or is its own
 * parent is refused (IQ_DEVERR_SEQ); a fresh page is taken as by iq_pages_extend.
 * pools: n_pools (0..8) host structs. */
iq_status iq_pages_fork(const iq_pages* pages, const iq_page_pool* pools_host, int32_t n_pools,
                        const int32_t* parent_dev, const int32_t* child_dev, int32_t n, void* workspace_dev,
                        size_t workspace_bytes, iq_stream_t stream);

/* Moves the held pages to the front of the pools: with N pages held, the k-th held page at or above N moves
 * to the k-th free one below N; tables and counts follow.  n_held_dev (or NULL) gets N.  An entry that names a page
 * that nobody holds, or none of the pool's, stays as it is (IQ_DEVERR_PAGE). */
iq_status iq_pages_compact(const iq_pages* pages, const iq_page_pool* pools_host, int32_t n_pools,
                           int32_t* n_held_dev, void* workspace_dev, size_t workspace_bytes, iq_stream_t stream);

/* Copies page src[i] to page dst[i], in every layer of every pool; tables and counts stay.  An entry whose
 * dst is the src of another entry or the dst of an earlier one, or whose pages lie outside the pool, is left
 * out (IQ_DEVERR_PAGE). */
iq_status iq_pages_copy(const iq_pages* pages, const iq_page_pool* pools_host, int32_t n_pools,
                        const int32_t* src_dev, const int32_t* dst_dev, int32_t n, void* workspace_dev,
                        size_t workspace_bytes, iq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IQ8_H */
