// rows.cu -- the calls over packed query rows (pagedkv_batch.h): host checks, and the
// launches of rows_tc.cu and decode_shared.cu one behind the other.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "rows.h"
#include "../../include/pagedkv_batch.h"

namespace pkv {
namespace {

// Whether rows are attended one by one, each reading its run's keys again (from the L2, where
// they are shared), in one launch: where what the rows can read, by the width of their table
// rows, is below what the two or three launches of the other way cost, and where a run has so
// few rows, on the average, that products of 256 rows are mostly empty.  Measured (8 kv heads
// of 128; all at once / one by one, us): decode behind a shared prefix, 32 sequences behind 256
// tokens (38 MB) 18.7 / 7.4, 4 behind 4096 (68 MB) 21.2 / 11.4, 16 behind 4096 (285 MB) 24.2 /
// 26.9.  Rows per run: cross attention of 64 sequences to 512 .. 4096 keys, 1 row 124.6 / 121.1
// (int8 pages 234 / 91), 2 rows 118.9 / 138.7 (247 / 145), 3 rows 119.5 / 189.6 (246 / 213), of
// 512 to 200 .. 256 int8 keys, 4 rows 284 / 261; decode of 64 sequences behind 2000 tokens, 1 a
// group 110.6 / 93.1 (218 / 73.4), 2 67.9 / 67.8 (120 / 69.5), 4 46.9 / 60.3 (69.7 / 68.7), of
// 256 behind 200 to 600, 2 a group 92.5 / 68.7 (138 / 66).
//
// The mean says little of single runs (idle ones beside one of many rows), so each run goes its
// own way: those of up to that many rows one by one, beside the others at once.  Measured (so /
// all at once / one by one): one of 64 sequences has 60 rows and 8192 keys 31.0 / 26.6 / 171, over
// int8 pages 36.5 / 33.7 / 216; one has 100 rows and 16384 int8 keys, 60 have one and 2048, 137 /
// 245 / 682; 64 sequences of one row, as above, 110 / 111 / 104 and 91 / 256 / 83.  A cross
// attention of as many rows as sequences is taken for a step, whose sequences have a row each, and
// spared those 6 us (where 60 of 64 rows are one sequence's: 41 / 27 / 171).  Not a decode: room
// for as many groups as sequences is the fixed shape of a captured step, whatever the groups hold.
// 64 sequences with room for 64 groups, all in one of 4096 tokens 38.6 / 32.4 / 103, over int8
// pages 44 / 32 / 128; a group of 2000 each 112 / 117 / 106 and 90 / 235 / 80.
constexpr int64_t kOneByOneBytes = 192 << 20;       // as bf16

// Runs of up to how many rows are attended row by row (-1: none).
int32_t rows_one_by_one(const RowsArgs &a)
{
    if (a.n_q_heads / a.dims.n_kv_heads > 8) return -1;
    const int32_t few = a.kv_dtype == PKV_KV_INT8 ? 3 : a.ctx_lens ? 2 : 1;
    if (const char *impl = getenv("PKV_ROWS_IMPL")) {
        if (strcmp(impl, "all") == 0) return -1;
        if (strcmp(impl, "one") == 0) return kAllRows;
        if (strcmp(impl, "both") == 0) return few;
    }
    const int64_t tokens = (int64_t)(a.ctx_lens ? a.max_blocks : a.max_run_blocks) * a.dims.block_size;
    if (tokens * a.dims.n_kv_heads * a.dims.head_dim * 4 <= kOneByOneBytes / a.n_rows) return kAllRows;
    if (!a.ctx_lens && a.n_rows == a.n_runs) return kAllRows;
    return a.n_rows <= (int64_t)few * a.n_runs ? few : -1;
}

cudaError_t launch_rows(RowsArgs &a, int num_sms, cudaStream_t stream)
{
    a.few = rows_one_by_one(a);
    if (a.few == kAllRows) return launch_rows_whole(a, num_sms, stream);
    cudaError_t e = cudaSuccess;
    if (a.n_runs > 0) e = launch_rows_tc(a, num_sms, stream);
    if (e == cudaSuccess && a.few >= 0) e = launch_rows_whole(a, num_sms, stream);
    if (e == cudaSuccess && a.ctx_lens) e = launch_rows_rest(a, num_sms, stream);
    return e == cudaSuccess ? launch_rows_join(a, num_sms, stream) : e;
}

// Checks that the two calls share; fills what they share of *a.
int prepare_rows(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, int32_t n_rows, const void *k_pool,
                 const void *v_pool, const float *k_scales, const float *v_scales, int32_t kv_dtype,
                 const pkv_dims &dims, float softmax_scale, int32_t most_heads, pkv_bf16 *out, float *lse_out,
                 void *workspace, size_t workspace_bytes, int32_t *dev_status, RowsArgs *a)
{
    const int st = check_dims(dims);
    if (st != PKV_OK) return st;
    if (n_rows < 0 || n_q_heads <= 0 || n_q_heads % dims.n_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (n_q_heads / dims.n_kv_heads > most_heads || n_q_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (kv_dtype != PKV_KV_BF16 && kv_dtype != PKV_KV_INT8) return PKV_ERR_UNSUPPORTED;
    if (!row_stride_ok(q_stride, n_q_heads, dims.head_dim)) return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return PKV_ERR_INVALID_ARG;
    if (n_rows == 0) return PKV_OK;
    if ((int64_t)n_rows * n_q_heads > 0x7fffffffLL) return PKV_ERR_OUT_OF_RANGE;
    const void *p[] = {q, k_pool, v_pool, out};
    for (const void *x : p)
        if (!x || !aligned16(x)) return PKV_ERR_INVALID_ARG;
    if (out == q || (reinterpret_cast<uintptr_t>(lse_out) & 3u)) return PKV_ERR_INVALID_ARG;
    if (kv_dtype == PKV_KV_INT8 &&
        (!k_scales || !v_scales ||
         ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3u)))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pkv_rows_workspace_bytes(n_rows, n_q_heads, dims.head_dim))
        return PKV_ERR_WORKSPACE;
    a->q = q;
    a->q_stride = q_stride;
    a->n_q_heads = n_q_heads;
    a->n_rows = n_rows;
    a->k_pool = k_pool;
    a->v_pool = v_pool;
    a->k_scales = k_scales;
    a->v_scales = v_scales;
    a->kv_dtype = kv_dtype;
    a->dims = dims;
    a->softmax_scale = softmax_scale;
    a->out = out;
    a->lse_out = lse_out;
    a->partials = carve_rows_workspace(workspace, n_rows, n_q_heads, dims.head_dim);
    a->dev_status = dev_status;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_rows_workspace_bytes(int32_t n_rows, int32_t n_q_heads, int32_t head_dim)
{
    if (n_rows < 0 || n_q_heads <= 0 || (head_dim != 64 && head_dim != 128)) return 0;
    return rows_workspace_bytes(n_rows, n_q_heads, head_dim);
}

int paged_cross_attention(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, const int32_t *q_starts,
                          int32_t n_rows, const void *k_pool, const void *v_pool, const float *k_scales,
                          const float *v_scales, int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables,
                          int32_t max_blocks, const int32_t *key_lens, int32_t n_seqs, float softmax_scale,
                          pkv_bf16 *out, float *lse_out, void *workspace, size_t workspace_bytes,
                          int32_t *dev_status, pkv_stream_t stream)
{
    RowsArgs a{};
    int st = prepare_rows(q, q_stride, n_q_heads, n_rows, k_pool, v_pool, k_scales, v_scales, kv_dtype, dims,
                          softmax_scale, 16, out, lse_out, workspace, workspace_bytes, dev_status, &a);
    if (st != PKV_OK) return st;
    if (n_seqs < 0 || max_blocks <= 0) return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks * dims.block_size > PKV_ROWS_MAX_TOKENS) return PKV_ERR_OUT_OF_RANGE;
    if (n_rows == 0 || n_seqs == 0) return PKV_OK;
    if (!q_starts || !block_tables || !key_lens) return PKV_ERR_INVALID_ARG;
    a.starts = q_starts;
    a.run_tables = block_tables;
    a.run_lens = key_lens;
    a.n_runs = n_seqs;
    a.max_run_blocks = max_blocks;
    int sms = 0;
    st = num_sms_of_current_device(&sms);
    if (st != PKV_OK) return st;
    return cuda_status(launch_rows(a, sms, (cudaStream_t)stream));
}

int paged_decode_attention_shared(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, const void *k_pool,
                                  const void *v_pool, const float *k_scales, const float *v_scales,
                                  int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables,
                                  int32_t max_blocks, const int32_t *ctx_lens, int32_t n_seqs,
                                  const int32_t *group_starts, int32_t n_groups, const int32_t *prefix_tables,
                                  int32_t max_prefix_blocks, const int32_t *prefix_lens, float softmax_scale,
                                  pkv_bf16 *out, float *lse_out, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, pkv_stream_t stream)
{
    RowsArgs a{};
    int st = prepare_rows(q, q_stride, n_q_heads, n_seqs, k_pool, v_pool, k_scales, v_scales, kv_dtype, dims,
                          softmax_scale, 8, out, lse_out, workspace, workspace_bytes, dev_status, &a);
    if (st != PKV_OK) return st;
    if (n_groups < 0 || max_blocks <= 0 || max_prefix_blocks < 0 || (n_groups > 0 && max_prefix_blocks == 0))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks * dims.block_size > PKV_ROWS_MAX_TOKENS ||
        (int64_t)max_prefix_blocks * dims.block_size > PKV_ROWS_MAX_TOKENS)
        return PKV_ERR_OUT_OF_RANGE;
    if (n_seqs == 0) return PKV_OK;
    if (!block_tables || !ctx_lens) return PKV_ERR_INVALID_ARG;
    if (n_groups > 0 && (!group_starts || !prefix_tables || !prefix_lens)) return PKV_ERR_INVALID_ARG;
    a.starts = group_starts;
    a.run_tables = prefix_tables;
    a.run_lens = prefix_lens;
    a.n_runs = n_groups;
    a.max_run_blocks = max_prefix_blocks;
    a.tables = block_tables;
    a.ctx_lens = ctx_lens;
    a.max_blocks = max_blocks;
    int sms = 0;
    st = num_sms_of_current_device(&sms);
    if (st != PKV_OK) return st;
    return cuda_status(launch_rows(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
