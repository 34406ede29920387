/*
 * starkv_full.h -- full-width layers: prompt attention, a 4-bit paged cache with
 * the decode attention that reads it, the attention weights of a prompt, and
 * eviction by accumulated weight.
 *
 * Some layers of a model with latent caches keep their full width (the
 * protected layers of the technical review of arXiv 2606.08382, section 6.2 and
 * eq. 16; its section 7.3 combines the method with token eviction by
 * accumulated attention weight).  These entries serve such layers.  They take a
 * context (starkv.h) for the head shape (num_q_heads, num_kv_heads, head_dim),
 * the device and the device status word; the context's factors are not used.
 *
 * Conventions are those of starkv.h.  In addition:
 *   - q and k are taken as they enter the score: a rotary position is applied by
 *     the caller, so any position scheme works and a token keeps its position
 *     when eviction moves it.  Scores are q.k / sqrt(head_dim).
 *   - The context's device must be current (else STARKV_ERR_INVALID_ARG).
 *   - A row stride counts elements between one token's row and the next, so that
 *     q, k and v may be parts of one projection's output; a row's heads are dense:
 *     head h at h * head_dim.  Strides are multiples of 8, pointers 16-byte aligned.
 *   - Scores are held in fp32, so a probability is good to about 2^-22 of its score's
 *     magnitude.  The prompt entries take scores of magnitudes below 2^30 (a row with
 *     larger ones may be NaN).
 *   - Entries here neither allocate device memory nor keep state between calls;
 *     calls on different streams may overlap when their outputs and workspaces
 *     are different, and every call can be captured into a CUDA graph.
 */
#ifndef STARKV_FULL_H
#define STARKV_FULL_H

#include "starkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define STARKV_KV4_GROUP 32 /* channels that share a scale and a zero */

/* starkv_workspace_bytes, a further op.  Errors: INVALID_ARG, UNSUPPORTED_SHAPE (of the call). */
enum {
  STARKV_OP_KV4_DECODE = 16 /* starkv_kv4_decode_attn; total_q: its `accumulate` */
};

/* ---------------------------------------------------------------------------
 * The 4-bit cache.  Keys and values are quantised per (token, KV head, group of
 * 32 channels): scale s = fl16(fl32((max - min) / 15)), zero z = fl16(min), code
 * = clamp(rint_even(fl32(fl32(x - z) / s)), 0, 15) (s = 0: code 0); the stored
 * value is code * s + z.  A group whose s, z or 15 s + z is not finite in fp16,
 * or that holds a non-finite value, is stored as zeros and sets
 * STARKV_DEV_QUANT_OVERFLOW.
 *
 * pages: [n_pages][num_kv_heads][head_page_bytes], 16-byte aligned.  The 16 tokens of
 *   one KV head in a page, d = head_dim, NG = d / 32, in 32-bit words (8 codes each,
 *   low nibble first):
 *     K codes  [16][d/8]  channels 32 g + 8 c .. + 7 at word c * NG + g (c < 4)
 *     V codes  [16][d/8]  channels 8 w .. + 7 at word w
 *     K meta   [16][NG]   scale in the low 16 bits, zero in the high 16 bits
 *     V meta   [16][NG]
 * weights: [n_pages][num_kv_heads][16] fp32, 16-byte aligned, the attention weight that each token has
 *   drawn so far, summed over the query heads that share the KV head; NULL where the
 *   caller keeps none. */
typedef struct starkv_kv4_cache {
  void* pages;
  float* weights;
  int64_t n_pages;
} starkv_kv4_cache;

typedef struct starkv_kv4_sizes {
  int64_t pages_bytes;     /* for the requested n_pages                  */
  int64_t weights_bytes;
  int32_t head_page_bytes; /* 16 d + 128 (d / 32)                        */
  int32_t groups;          /* d / 32                                     */
} starkv_kv4_sizes;

/* Host-only: sizes of a 4-bit cache of n_pages pages.  Errors: as starkv_cache_layout, and
 * UNSUPPORTED_SHAPE for 2^63 bytes or more. */
STARKV_API starkv_status starkv_kv4_layout(const starkv_config* cfg, int64_t n_pages, starkv_kv4_sizes* out);

/* Quantise n tokens' keys and values into the cache.  k, v: device bf16
 * [n][num_kv_heads][head_dim], rows k_stride and v_stride apart.  slot_mapping: device
 * int64 [n], slot = page*16 + offset; a negative slot skips that token; slots must be
 * distinct within one call.  weights: device fp32 [n][num_kv_heads], the tokens' first
 * accumulated weights (starkv_prompt_weights), or NULL for zero; written where the
 * cache keeps weights.  Only the written tokens' bytes change.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE (2^35 channels of k or more); device bits BAD_SLOT,
 * QUANT_OVERFLOW. */
STARKV_API starkv_status starkv_kv4_append(starkv_ctx* ctx, const starkv_kv4_cache* cache, const void* k,
                                           const void* v, int64_t k_stride, int64_t v_stride,
                                           const int64_t* slot_mapping, const float* weights, int64_t n,
                                           starkv_stream_t stream);

/* Read tokens of the cache back, rounded to bf16 (the keys and values of a prompt's
 * earlier chunks, for starkv_prompt_attn).  Row r of k_out and v_out, device bf16
 * [total][num_kv_heads][head_dim] (dense), with cu[b] <= r < cu[b+1], is token
 * starts[b] + r - cu[b] of sequence b.  cu: device int32 [batch+1], cu[0] = 0, cu[batch]
 * = total; starts: device int32 [batch], or NULL for zeros; block_table: device int32
 * [batch][max_pages].  A token that is out of its block table, or whose page is out of
 * the pool, reads as zeros.
 * Errors: INVALID_ARG; device bits BAD_PAGE, BAD_SEQ_LEN, BAD_QUERY_SPAN (cu). */
STARKV_API starkv_status starkv_kv4_read(starkv_ctx* ctx, const starkv_kv4_cache* cache, const int32_t* block_table,
                                         const int32_t* starts, const int32_t* cu, int32_t batch, int32_t max_pages,
                                         int64_t total, void* k_out, void* v_out, starkv_stream_t stream);

/* Single-query attention over the 4-bit cache.  q: device bf16
 * [batch][num_q_heads][head_dim] (dense), of magnitudes below 2^115 (beyond, and for NaN,
 * the head's row may be NaN); sequence b's query attends to tokens [0, seq_lens[b]).
 * out: device bf16 [batch][num_q_heads][head_dim]; seq_len 0 gives a
 * zero row.  accumulate != 0: cache.weights of each attended token gains the
 * probabilities that the query heads of its KV head gave it.  A page that stands in two
 * tables gains both sequences' share; the order of those additions is not fixed, all else
 * is.  A bad length sets its bit and gives a zero row and no weight; a bad page sets its
 * bit, and its tokens are left out.
 * workspace: >= starkv_workspace_bytes(STARKV_OP_KV4_DECODE, batch, max_pages, total_q =
 * accumulate), 256-byte aligned; it must not be used by another call at the same time.
 * It grows with max_pages where weights are accumulated (4 bytes a token and query head).
 * Errors: INVALID_ARG, WORKSPACE_TOO_SMALL; device bits BAD_PAGE, BAD_SEQ_LEN. */
STARKV_API starkv_status starkv_kv4_decode_attn(starkv_ctx* ctx, const starkv_kv4_cache* cache, const void* q,
                                                const int32_t* block_table, const int32_t* seq_lens, int32_t batch,
                                                int32_t max_pages, int32_t accumulate, void* out, void* workspace,
                                                size_t workspace_bytes, starkv_stream_t stream);

/* Keep keep_lens[b] of each sequence's seq_lens[b] tokens (all, where it has no more):
 * per KV head, the `recent` last ones and, of the others, those with the largest
 * weights; equal weights go to the lowest index, NaN counts as the lowest weight.  Their
 * bytes and weights are gathered, in order, into the pages of dst_block_table (device
 * int32 [batch][dst_max_pages]) of the same pool; the sequence's own pages stay as they are
 * and may be freed behind the call.  The destination pages must be distinct and not
 * among the pages that are read.  Slots behind the last kept token stay as they were.
 * keep_lens: device int32 [batch], 0 <= keep_lens[b] <= dst_max_pages*16 (only
 * min(keep_lens[b], seq_lens[b]) slots are used).  recent >= 0 (at most the kept count
 * is used).  new_lens: device int32 [batch], min(keep_lens, seq_lens); it may be seq_lens
 * or keep_lens itself.  kept: device int32 [batch][num_kv_heads][dst_max_pages*16], the kept
 * tokens' indices in rising order, -1 behind them.  A sequence with a bad length or page
 * sets its bit, gets new_lens 0 and kept -1, and moves nothing.
 * Errors: INVALID_ARG; device bits BAD_PAGE, BAD_SEQ_LEN. */
STARKV_API starkv_status starkv_kv4_evict(starkv_ctx* ctx, const starkv_kv4_cache* cache, const int32_t* block_table,
                                          const int32_t* seq_lens, const int32_t* keep_lens, int32_t recent,
                                          int32_t batch, int32_t max_pages, const int32_t* dst_block_table,
                                          int32_t dst_max_pages, int32_t* new_lens, int32_t* kept,
                                          starkv_stream_t stream);

/* ---------------------------------------------------------------------------
 * Causal attention of packed sequences over their own keys and values.
 * q: device bf16 [total_q][num_q_heads][head_dim], k and v: device bf16
 * [total_k][num_kv_heads][head_dim], rows q_stride, k_stride, v_stride apart; sequence b
 * has rows cu_q[b] .. cu_q[b+1]-1 of q and cu_k[b] .. cu_k[b+1]-1 of k and v (cu_q, cu_k:
 * device int32 [batch+1], from 0 to total_q and total_k).  With n_q and n_k rows, query
 * i sees keys j <= n_k - n_q + i: the last query sees every key.  Only the keys that a
 * query sees reach its row.  max_q_len: upper bound of n_q.
 * out: device bf16 [total_q][num_q_heads][head_dim] (dense); lse: device fp32
 * [total_q][num_q_heads], ln sum_j exp(score), or NULL.  A query that sees no key has a
 * zero row and lse -inf.
 * workspace: >= starkv_prompt_workspace_bytes, 256-byte aligned (may be NULL where that is
 * 0); it must not be used by another call at the same time.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE (more than 65535 sequences, or 2^31 blocks),
 * WORKSPACE_TOO_SMALL; device
 * bit BAD_QUERY_SPAN (cu_q, cu_k or max_q_len; the sequence's rows are left as they were). */
STARKV_API starkv_status starkv_prompt_attn(starkv_ctx* ctx, const void* q, const void* k, const void* v,
                                            int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                            const int32_t* cu_q, const int32_t* cu_k, int32_t batch, int64_t total_q,
                                            int64_t total_k, int32_t max_q_len, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes, starkv_stream_t stream);

/* Workspace bytes of starkv_prompt_attn for packed rows of these sizes (40 MB at most, where
 * units of its work are shared between SMs).  out: host.  Errors: INVALID_ARG, UNSUPPORTED_SHAPE
 * (more than 65535 sequences, 2^31 rows). */
STARKV_API starkv_status starkv_prompt_workspace_bytes(const starkv_ctx* ctx, int32_t batch, int64_t total_q,
                                                       int64_t total_k, size_t* out);

/* The attention weight that the last `window` queries of each packed sequence give to
 * its keys: weights[j][kv] = sum over the query heads of KV head kv and over those
 * queries that see key j of exp(score - lse).  q, k, strides, cu_q, cu_k: as
 * starkv_prompt_attn, lse: its result; max_k_len: upper bound of n_k.  weights: device
 * fp32 [total_k][num_kv_heads], overwritten.  Sums are fp32, in a fixed order.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE (more than 65535 sequences); device bit
 * BAD_QUERY_SPAN (cu_q, cu_k or max_k_len; the sequence's rows are left as they were). */
STARKV_API starkv_status starkv_prompt_weights(starkv_ctx* ctx, const void* q, const void* k, int64_t q_stride,
                                               int64_t k_stride, const float* lse, const int32_t* cu_q,
                                               const int32_t* cu_k, int32_t batch, int64_t total_q, int64_t total_k,
                                               int32_t max_k_len, int32_t window, float* weights,
                                               starkv_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* STARKV_FULL_H */
