/*
 * pagedkv_batch.h -- calls for a batch of requests of any lengths: the block
 * tables and slot maps of a step built on the device, the page write of packed
 * rows by slot, the attention of packed queries to keys of another length, and
 * the decode of groups of sequences that share their first tokens.
 *
 * Conventions (pointers, streams, status codes, dev_status, pool and table
 * layout) are those of pagedkv.h.
 *
 * A packed batch is n_rows rows without padding between the sequences: those
 * of sequence s are starts[s] .. starts[s + 1] - 1 (int32 [n_seqs + 1], on the
 * device, not decreasing, 0 <= starts[s] <= n_rows).  Rows before the first
 * sequence and behind the last belong to none: they are left as they were.
 */
#ifndef PAGEDKV_BATCH_H
#define PAGEDKV_BATCH_H

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * paged_step_maps -- the tables and maps of one step, from what each sequence
 * holds and what it adds (the device half of pkv_bm_admit / pkv_bm_begin_step,
 * AstrAI cache.py, PagedCache.alloc_n and write).
 *   lens, n_new  int32 [n_seqs]: tokens held before the step, tokens it adds
 *            (0: the sequence sits the step out)
 *   free_blocks  int32 [n_free]: free block ids in the order in which they are
 *            handed out; cursor int32 [1] (nullable: 0): how many of them
 *            earlier steps have taken
 *   block_tables int32 [n_seqs][max_blocks]  (read and written)
 *   ctx_lens     int32 [n_seqs]  lens + n_new                        (written)
 *   token_starts int32 [n_seqs + 1]  the packed batch's starts: exclusive sums
 *            of n_new                                                (written)
 *   token_seqs, positions int32 [n_tokens], slots int64 [n_tokens]: sequence,
 *            position and pool row (table[t / bs] * bs + t % bs) of each row of
 *            the packed batch; -1, 0, -1 behind its last row         (written)
 *   cursor_out   int32 [1]  cursor plus the blocks the step wants    (written)
 * Sequence s holds ceil(lens[s] / bs) blocks and wants ceil((lens[s] + n_new[s])
 * / bs): the new ones are the next of the free list, in the order of the
 * sequences.  Its table entries before them are kept.  Those behind them are
 * kept too where lens[s] > 0, and are set to the scratch id (n_blocks) where
 * lens[s] == 0, so that a row taken over from an earlier sequence holds nothing
 * of it.
 * A sequence whose length is bad (lens[s] or n_new[s] negative, or their sum
 * more than its table row spans: PKV_DEV_BAD_LENGTH) adds no token, takes no
 * block and gets ctx_lens[s] = 0; its table row stays as it was.  Where the
 * free list has run out (PKV_DEV_OUT_OF_BLOCKS; a negative cursor counts as
 * that) or names an id outside [0, n_blocks) (PKV_DEV_BAD_BLOCK_ID), the entry
 * is the scratch id and the block's tokens have slot -1; so have the tokens
 * that fall into a held block whose id is outside [0, n_blocks]
 * (PKV_DEV_BAD_BLOCK_ID), or that is the scratch block in a row which begins with
 * another one (PKV_DEV_OUT_OF_BLOCKS: an earlier step found no block for it, and
 * the caller has not put one in its place).  A row that begins with the scratch
 * block is an inactive sequence's: its tokens have slots in the scratch block,
 * and a sequence that found no block for its first tokens is one until the
 * caller has given it some.  When the batch has more than n_tokens tokens, those
 * behind them are in no map (PKV_DEV_BAD_POSITION).  Sums that pass 2^31 - 1
 * are written as that.  block_size is a multiple of 16, at most 256.  Outputs
 * must not overlap inputs (lens is not ctx_lens, cursor not cursor_out).
 */
int paged_step_maps(const int32_t *lens, const int32_t *n_new, int32_t n_seqs, const int32_t *free_blocks,
                    int32_t n_free, const int32_t *cursor, int32_t n_blocks, int32_t block_size,
                    int32_t *block_tables, int32_t max_blocks, int32_t n_tokens, int32_t *ctx_lens,
                    int32_t *token_starts, int32_t *token_seqs, int32_t *positions, int64_t *slots,
                    int32_t *cursor_out, int32_t *dev_status, pkv_stream_t stream);

/*
 * paged_kv_write_slots -- packed rows to their pool rows: row i of k_new and
 * v_new goes to pool row slots[i] (as paged_step_maps gives them), stored as
 * paged_kv_write or paged_kv_write_int8 (kv_dtype) store a row, bit for bit.
 *   k_new, v_new  bf16, n_kv_heads rows of head_dim behind one another per
 *            row, k_stride / v_stride elements apart (a multiple of 8, at least
 *            a row's length: they may be parts of a fused projection's rows)
 *   slots    int64 [n_rows]; distinct where they are not negative and not of the
 *            scratch block (what rows with the same slot leave there is any of theirs)
 * A row of a negative slot is skipped; one of a slot outside the pool
 * (>= (n_blocks + 1) * block_size) too, with PKV_DEV_BAD_POSITION.
 * n_rows == 0 is a no-op.
 */
int paged_kv_write_slots(const pkv_bf16 *k_new, int64_t k_stride, const pkv_bf16 *v_new, int64_t v_stride,
                         void *k_pool, void *v_pool, float *k_scales, float *v_scales, int32_t kv_dtype,
                         pkv_dims dims, const int64_t *slots, int32_t n_rows, int32_t *dev_status,
                         pkv_stream_t stream);

/* The most tokens a table row may span in the two calls below (PKV_ERR_OUT_OF_RANGE
 * above): positions are int32, with room for a tile behind the last one. */
#define PKV_ROWS_MAX_TOKENS 0x7fffff00

/*
 * pkv_rows_workspace_bytes -- the workspace of the two calls below, for n_rows
 * packed rows (paged_decode_attention_shared: n_seqs) of n_q_heads query heads.
 * 0 on invalid arguments.
 */
size_t pkv_rows_workspace_bytes(int32_t n_rows, int32_t n_q_heads, int32_t head_dim);

/*
 * paged_cross_attention -- every query row of sequence s sees all key_lens[s]
 * tokens of its pages (an encoder's states, say, of another length than the
 * queries): no causal mask.
 *   q        bf16, row i at q + i q_stride, its n_q_heads rows of head_dim
 *            behind one another (q_stride in elements, a multiple of 8)
 *   q_starts int32 [n_seqs + 1]: the packed batch's starts
 *   pools, scales, kv_dtype, block_tables, softmax_scale  as in
 *            paged_decode_attention; n_q_heads / n_kv_heads in 1 .. 16, any
 *            number of kv heads for int8 pages too
 *   out      bf16 [n_rows][n_q_heads][head_dim]; not q
 *   lse_out  fp32 [n_rows][n_q_heads] (nullable)
 *   workspace  as in paged_decode_attention: pkv_rows_workspace_bytes(n_rows,
 *            ...) bytes, 256-byte aligned, not shared by calls that run at once
 * key_lens[s] == 0 gives o = 0 and lse = -inf; so does a bad one (negative, or
 * more than the table row spans: PKV_DEV_BAD_LENGTH).  A block id outside
 * [0, n_blocks] (PKV_DEV_BAD_BLOCK_ID): its tokens are seen as rows of zeros.
 * Starts that decrease or pass n_rows: PKV_DEV_BAD_LENGTH, outputs undefined.
 * Rows are contracted all at once, up to 256 of a sequence in one product, or,
 * where that is less work, one by one, with up to 8 query heads per kv head (the
 * same results within the bounds below).  A call of as many rows as sequences is
 * taken for a step, of a row each, and goes one by one; where most of the rows
 * are a few sequences', one row more (of no sequence) sends those at once.
 * PKV_ROWS_IMPL in the environment, read at every call here and in
 * paged_decode_attention_shared, takes a way: all, one, or both (sequences or
 * groups of few rows one by one, the others at once).
 * Rounding: scores, maxima, sums and unfinished outputs are binary32, outputs are
 * rounded once to bf16.  bf16 pages: probabilities are rounded to bf16 (2^-8 of
 * each) at once, as in the prefills, and held to 2^-16 one by one.  int8 pages:
 * at once, probabilities and values (code times scale) are rounded to fp16, 2^-11
 * of each, where probabilities below 2^-21 are held to 2^-32 and values of a
 * scale below 2^-13 of the largest V scale of their kv head in the sequence (or
 * the group's prefix) to 2^-24 of that scale; one by one, queries are rounded to fp16 multiples of a power of two of their own
 * (bf16 queries exactly but for elements below 2^-17 of the largest) and the
 * weights, each with its scale, held to 2^-22, whatever the other scales are.
 */
int paged_cross_attention(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, const int32_t *q_starts,
                          int32_t n_rows, const void *k_pool, const void *v_pool, const float *k_scales,
                          const float *v_scales, int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables,
                          int32_t max_blocks, const int32_t *key_lens, int32_t n_seqs, float softmax_scale,
                          pkv_bf16 *out, float *lse_out, void *workspace, size_t workspace_bytes,
                          int32_t *dev_status, pkv_stream_t stream);

/*
 * paged_decode_attention_shared -- paged_decode_attention for groups of
 * sequences that share their first tokens (a system prompt, a prompt that is
 * sampled many times): those are read and contracted once for a group's
 * queries together.
 *   group_starts   int32 [n_groups + 1]: sequences group_starts[g] ..
 *            group_starts[g + 1] - 1 are group g (not decreasing, within
 *            [0, n_seqs]); a sequence of no group shares nothing
 *   prefix_tables  int32 [n_groups][max_prefix_blocks], prefix_lens int32
 *            [n_groups]: the pages of the group's first tokens and their
 *            number (any, not only whole blocks)
 *   block_tables, ctx_lens  as in paged_decode_attention: a sequence's tokens
 *            from prefix_lens[g] on, at the places they would have without
 *            sharing.  Entries of blocks wholly within the prefix are not read.
 *   q (with q_stride), pools, scales, out, lse_out, workspace  as above
 * Sequence s of group g sees tokens 0 .. min(ctx_lens[s], prefix_lens[g]) - 1
 * of the group and prefix_lens[g] .. ctx_lens[s] - 1 of its own; the outputs
 * are paged_decode_attention's over the two one behind the other.  A sequence
 * that ends within the prefix is attended by itself; what the tokens behind its
 * end hold (pages that are not written yet, say) does not reach it.  n_q_heads /
 * n_kv_heads in 1 .. 8, any number of kv heads for int8 pages too.
 * ctx_lens[s] == 0 gives o = 0 and lse = -inf; so do a bad length of the
 * sequence or of its group (PKV_DEV_BAD_LENGTH).  Bad starts and block ids as
 * above.
 */
int paged_decode_attention_shared(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, const void *k_pool,
                                  const void *v_pool, const float *k_scales, const float *v_scales,
                                  int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables,
                                  int32_t max_blocks, const int32_t *ctx_lens, int32_t n_seqs,
                                  const int32_t *group_starts, int32_t n_groups, const int32_t *prefix_tables,
                                  int32_t max_prefix_blocks, const int32_t *prefix_lens, float softmax_scale,
                                  pkv_bf16 *out, float *lse_out, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, pkv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_BATCH_H */
