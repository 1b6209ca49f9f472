/*
 * pagedkv_rope.h -- rotary positions written into the pages: the queries and
 * keys of a call are turned by the angles of their positions, keys and values
 * go into the pool (bf16 or int8 pages), the turned queries are returned.  One
 * launch in place of a rotation of q, a rotation of k and a page write.
 *
 * Conventions (pointers, streams, status codes, dev_status, pool and table
 * layout) are those of pagedkv.h.
 *
 * The turn.  A row x of a query or key head at position t has its first rot_dim
 * elements turned in pairs, the others kept:
 *   half layout         pair i = (x[i], x[i + rot_dim / 2])
 *   interleaved layout  pair i = (x[2 i], x[2 i + 1])
 *   (a, b) -> magnitude * (a cos A_i - b sin A_i, b cos A_i + a sin A_i),
 *   A_i = t * f_i, with f_i the pair's frequency in radians per position.
 * Frequencies are given as phases: round(f_i / (2 pi) * 2^64), the turns per
 * position in units of 2^-64.  The kernels multiply them by the position modulo
 * 2^64, which is exact, so far positions lose nothing (a product in binary32 is
 * off by about t * f_i * 2^-24 radians: 0.06 at position 10^6).
 */
#ifndef PAGEDKV_ROPE_H
#define PAGEDKV_ROPE_H

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the frequencies base^(-2 i / rot_dim) are changed for contexts longer than
 * the original_context a model was trained on, by a factor >= 1. */
enum pkv_rope_scaling {
    PKV_ROPE_NONE = 0,
    PKV_ROPE_LINEAR = 1, /* f / factor (positions interpolated) */
    PKV_ROPE_NTK = 2,    /* base * factor^(rot_dim / (rot_dim - 2)): the fastest pair kept, the slowest / factor */
    PKV_ROPE_BANDS = 3,  /* by the turns n = original_context f / (2 pi) of a pair: f kept for n >= high_turns,
                            f / factor for n <= low_turns, blended linearly in n between */
    PKV_ROPE_YARN = 4    /* a linear ramp over the pair index i between the pairs of high_turns and of low_turns
                            (floor, ceil): f to f / factor; magnitude 0.1 ln(factor) + 1 */
};

/* The turn of a call.  phases: rot_dim / 2 values in device memory, 16-byte
 * aligned.  rot_dim: a multiple of 16, at most head_dim.  magnitude: finite (as a float). */
typedef struct pkv_rope {
    const uint64_t *phases;
    int32_t rot_dim;
    int32_t interleaved; /* 0: half layout */
    double magnitude;
} pkv_rope;

/*
 * pkv_rope_phases -- the phases and the magnitude of a base and a scaling
 * (host only; phases_out has rot_dim / 2 entries in host memory, to be copied
 * to the device).  low_turns and high_turns are used by BANDS and YARN
 * (0 < low_turns < high_turns), original_context by those two, factor by all
 * but NONE.  PKV_ERR_INVALID_ARG for a null pointer, a rot_dim that is not a
 * positive multiple of 16, a base that is not finite and above 1, a factor
 * that is not finite and >= 1, or bad turns or context; PKV_ERR_UNSUPPORTED for
 * another scaling.
 */
int pkv_rope_phases(int32_t rot_dim, double base, int32_t scaling, double factor, double original_context,
                    double low_turns, double high_turns, uint64_t *phases_out, double *magnitude_out);

/*
 * paged_kv_write_rope -- token j < n_new of sequence s sits at position
 * start_pos[s] + j: its query and key heads are turned, its key and value rows
 * written to the pages at that position, its turned queries to q_out.
 *   q, k_new, v_new  bf16; token (s, j) of q is at q + (s n_new + j) q_stride,
 *            its n_q_heads rows of head_dim behind one another (k_new, v_new:
 *            n_kv_heads rows, k_stride, v_stride).  Strides are in elements, a
 *            multiple of 8, at least the rows' length: the three may be parts
 *            of one fused projection's rows.
 *   q_out    bf16 [n_seqs][n_new][n_q_heads][head_dim]; may be q itself where
 *            q_stride is n_q_heads * head_dim (another overlap is undefined)
 *   pools, scales  as in paged_kv_write / paged_kv_write_int8 (kv_dtype)
 * The turned rows are computed in binary32 and rounded once: to bf16, or for
 * int8 pages to their codes (scale = absmax / 127 of the turned row) without a
 * bf16 rounding between.  Values are stored as paged_kv_write(_int8) stores them,
 * bit for bit.  A row whose position or block is bad is not written to the
 * pages (PKV_DEV_BAD_POSITION / PKV_DEV_BAD_BLOCK_ID); its query is turned all
 * the same.  n_seqs == 0 or n_new == 0 is a no-op.
 */
int paged_kv_write_rope(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, const pkv_bf16 *k_new,
                        int64_t k_stride, const pkv_bf16 *v_new, int64_t v_stride, const pkv_rope *rope,
                        pkv_bf16 *q_out, void *k_pool, void *v_pool, float *k_scales, float *v_scales,
                        int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables, int32_t max_blocks,
                        const int32_t *start_pos, int32_t n_seqs, int32_t n_new, int32_t *dev_status,
                        pkv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_ROPE_H */
