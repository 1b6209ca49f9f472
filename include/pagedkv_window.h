/*
 * pagedkv_window.h -- attention over the pages with a sliding window and a few
 * first tokens that stay visible (sinks), for single tokens and for chunks, and
 * one layer's step of it with the rotary positions and the page write.
 *
 * Conventions (pointers, streams, status codes, dev_status, pool and table
 * layout) are those of pagedkv.h.
 *
 * The mask.  A query at position p sees token t when
 *   t <= p  and  (t < sinks  or  t > p - window):
 * the first `sinks` tokens and the last `window` ones, itself among them.
 * window >= 1, sinks >= 0; a window of at least the context is plain causal
 * attention.  Table entries of blocks none of whose tokens a query of the call
 * sees are never read, so such blocks may have been freed and their entries may
 * hold anything; rows of the blocks that are read, but that no query sees, may
 * hold anything too (NaN among it).  In a chunk, every row that some query sees
 * has to be finite, as one masked for another query of the same tile.
 */
#ifndef PAGEDKV_WINDOW_H
#define PAGEDKV_WINDOW_H

#include "pagedkv.h"
#include "pagedkv_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The most tokens a table row may span in the calls below (max_blocks *
 * block_size; PKV_ERR_OUT_OF_RANGE above): positions are int32, with room for a
 * tile behind the last one. */
#define PKV_WINDOW_MAX_TOKENS 0x7fffff00

/*
 * paged_decode_attention_window -- one query per sequence, at position
 * ctx_lens[s] - 1, over bf16 or int8 pages.  Arguments as in
 * paged_decode_attention; no workspace: the pieces of a long window are joined
 * through the shared memory of a thread-block cluster.  n_q_heads / n_kv_heads
 * in 1 .. 8 (any of them), any number of kv heads for int8 pages too.
 * ctx_lens[s] == 0 gives o = 0 and lse = -inf.
 */
int paged_decode_attention_window(const pkv_bf16 *q, int32_t n_q_heads, const void *k_pool, const void *v_pool,
                                  const float *k_scales, const float *v_scales, int32_t kv_dtype, pkv_dims dims,
                                  const int32_t *block_tables, int32_t max_blocks, const int32_t *ctx_lens,
                                  int32_t n_seqs, float softmax_scale, int32_t window, int32_t sinks, pkv_bf16 *out,
                                  float *lse_out, int32_t *dev_status, pkv_stream_t stream);

/*
 * paged_decode_step_window -- one layer's step of one token per sequence in one
 * launch: the new token's query and key heads turned (rope nullable: as they
 * are), its key and value rows written at position start_pos[s], then
 * paged_decode_attention_window over ctx_lens tokens, which must count the new
 * one.  Results are those of paged_kv_write_rope (or the page write) followed
 * by the attention, except that the turned queries are not rounded to bf16 in
 * between.  q, k_new, v_new: one token per sequence, q_stride, k_stride,
 * v_stride elements apart (as in paged_kv_write_rope).  A block that is
 * written may belong to one sequence of the call only, inactive sequences with
 * an all-scratch table row excepted (their output is undefined).
 */
int paged_decode_step_window(const pkv_bf16 *k_new, int64_t k_stride, const pkv_bf16 *v_new, int64_t v_stride,
                             const int32_t *start_pos, const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads,
                             const pkv_rope *rope, void *k_pool, void *v_pool, float *k_scales, float *v_scales,
                             int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables, int32_t max_blocks,
                             const int32_t *ctx_lens, int32_t n_seqs, float softmax_scale, int32_t window,
                             int32_t sinks, pkv_bf16 *out, float *lse_out, int32_t *dev_status, pkv_stream_t stream);

/*
 * paged_prefill_attention_window -- paged_prefill_attention (bf16 pages) under the mask
 * above: query i of sequence s sits at position prefix_lens[s] + i.  Key tiles
 * that no query of a CTA's rows sees are not loaded, so the work grows with
 * the window and not with the prefix.  A sequence whose length is bad (prefix_lens[s]
 * negative, or prefix_lens[s] + chunk more than its table row spans:
 * PKV_DEV_BAD_LENGTH) leaves all of its output rows as they were.
 */
int paged_prefill_attention_window(const pkv_bf16 *q, int32_t n_q_heads, const pkv_bf16 *k_pool,
                                   const pkv_bf16 *v_pool, pkv_dims dims, const int32_t *block_tables,
                                   int32_t max_blocks, const int32_t *prefix_lens, int32_t n_seqs, int32_t chunk,
                                   float softmax_scale, int32_t window, int32_t sinks, pkv_bf16 *out, float *lse_out,
                                   int32_t *dev_status, pkv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_WINDOW_H */
