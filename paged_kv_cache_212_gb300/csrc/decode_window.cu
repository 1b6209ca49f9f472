// decode_window.cu -- the windowed decode and its step (pagedkv_window.h): host checks and
// the launch of decode_window.cuh's kernels.
#include "decode_window.cuh"

namespace pkv {
namespace {

cudaError_t launch_window(WindowArgs &a, int32_t head_dim, bool int8, int32_t n_seqs, int sms, cudaStream_t stream)
{
    const int64_t units = (int64_t)n_seqs * a.n_kv_heads;
    int64_t tokens = (int64_t)a.max_blocks * a.block_size;
    if ((int64_t)a.window + a.sinks < tokens) tokens = (int64_t)a.window + a.sinks;
    const int64_t tiles = (tokens + kTile - 1) / kTile;
    const bool wide = a.group > 4;
    if (head_dim == 128) {
        if (int8) return launch_sized<128, true, true>(a, units, tiles, sms, stream);
        return wide ? launch_sized<128, false, true>(a, units, tiles, sms, stream)
                    : launch_sized<128, false, false>(a, units, tiles, sms, stream);
    }
    if (int8) return launch_sized<64, true, true>(a, units, tiles, sms, stream);
    return wide ? launch_sized<64, false, true>(a, units, tiles, sms, stream)
                : launch_sized<64, false, false>(a, units, tiles, sms, stream);
}

// Host checks of both calls; fills *a.
int prepare_window(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, void *k_pool, void *v_pool, float *k_scales,
                   float *v_scales, int32_t kv_dtype, const pkv_dims &dims, const int32_t *block_tables,
                   int32_t max_blocks, const int32_t *ctx_lens, int32_t n_seqs, float softmax_scale, int32_t window,
                   int32_t sinks, pkv_bf16 *out, float *lse_out, int32_t *dev_status, WindowArgs *a)
{
    int st = check_dims(dims);
    if (st != PKV_OK) return st;
    if (n_seqs < 0 || n_q_heads <= 0 || max_blocks <= 0 || window < 1 || sinks < 0) return PKV_ERR_INVALID_ARG;
    if (n_q_heads % dims.n_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (n_q_heads / dims.n_kv_heads > kHeads) return PKV_ERR_UNSUPPORTED;
    if (kv_dtype != PKV_KV_BF16 && kv_dtype != PKV_KV_INT8) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks * dims.block_size > PKV_WINDOW_MAX_TOKENS) return PKV_ERR_OUT_OF_RANGE;
    if ((int64_t)n_seqs * dims.n_kv_heads * kMaxSplits > 0x7fffffffLL) return PKV_ERR_OUT_OF_RANGE;
    if (!row_stride_ok(q_stride, n_q_heads, dims.head_dim)) return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0) return PKV_OK;
    if (!q || !k_pool || !v_pool || !block_tables || !ctx_lens || !out) return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return PKV_ERR_INVALID_ARG;
    if (kv_dtype == PKV_KV_INT8 &&
        (!k_scales || !v_scales ||
         ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3u)))
        return PKV_ERR_INVALID_ARG;
    a->q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a->q_stride = q_stride;
    a->n_q_heads = n_q_heads;
    a->group = n_q_heads / dims.n_kv_heads;
    a->k_pool = k_pool;
    a->v_pool = v_pool;
    a->k_scales = k_scales;
    a->v_scales = v_scales;
    a->n_blocks = dims.n_blocks;
    a->block_size = dims.block_size;
    a->n_kv_heads = dims.n_kv_heads;
    set_block_lookup(*a, dims.block_size);
    a->tables = block_tables;
    a->max_blocks = max_blocks;
    a->ctx_lens = ctx_lens;
    a->scale_log2 = softmax_scale * 1.4426950408889634f;
    a->window = window;
    a->sinks = sinks;
    a->out = reinterpret_cast<__nv_bfloat16 *>(out);
    a->lse_out = lse_out;
    a->dev_status = dev_status;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int paged_decode_attention_window(const pkv_bf16 *q, int32_t n_q_heads, const void *k_pool, const void *v_pool,
                                  const float *k_scales, const float *v_scales, int32_t kv_dtype, pkv_dims dims,
                                  const int32_t *block_tables, int32_t max_blocks, const int32_t *ctx_lens,
                                  int32_t n_seqs, float softmax_scale, int32_t window, int32_t sinks, pkv_bf16 *out,
                                  float *lse_out, int32_t *dev_status, pkv_stream_t stream)
{
    WindowArgs a{};
    int st = prepare_window(q, (int64_t)n_q_heads * dims.head_dim, n_q_heads, const_cast<void *>(k_pool),
                            const_cast<void *>(v_pool), const_cast<float *>(k_scales), const_cast<float *>(v_scales),
                            kv_dtype, dims, block_tables, max_blocks, ctx_lens, n_seqs, softmax_scale, window, sinks,
                            out, lse_out, dev_status, &a);
    if (st != PKV_OK || n_seqs == 0) return st;
    int sms = 0;
    st = num_sms_of_current_device(&sms);
    if (st != PKV_OK) return st;
    return cuda_status(launch_window(a, dims.head_dim, kv_dtype == PKV_KV_INT8, n_seqs, sms, (cudaStream_t)stream));
}

int paged_decode_step_window(const pkv_bf16 *k_new, int64_t k_stride, const pkv_bf16 *v_new, int64_t v_stride,
                             const int32_t *start_pos, const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads,
                             const pkv_rope *rope, void *k_pool, void *v_pool, float *k_scales, float *v_scales,
                             int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables, int32_t max_blocks,
                             const int32_t *ctx_lens, int32_t n_seqs, float softmax_scale, int32_t window,
                             int32_t sinks, pkv_bf16 *out, float *lse_out, int32_t *dev_status, pkv_stream_t stream)
{
    WindowArgs a{};
    int st = prepare_window(q, q_stride, n_q_heads, k_pool, v_pool, k_scales, v_scales, kv_dtype, dims, block_tables,
                            max_blocks, ctx_lens, n_seqs, softmax_scale, window, sinks, out, lse_out, dev_status, &a);
    if (st != PKV_OK) return st;
    if (rope) {
        st = check_rope(rope, dims.head_dim);
        if (st != PKV_OK) return st;
    }
    if (!row_stride_ok(k_stride, dims.n_kv_heads, dims.head_dim) || !row_stride_ok(v_stride, dims.n_kv_heads, dims.head_dim))
        return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0) return PKV_OK;
    if (!k_new || !v_new || !start_pos || !aligned16(k_new) || !aligned16(v_new)) return PKV_ERR_INVALID_ARG;
    a.k_new = reinterpret_cast<const __nv_bfloat16 *>(k_new);
    a.v_new = reinterpret_cast<const __nv_bfloat16 *>(v_new);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.start_pos = start_pos;
    if (rope) a.rope = rope_args(rope->phases, rope->rot_dim, rope->interleaved, rope->magnitude);
    int sms = 0;
    st = num_sms_of_current_device(&sms);
    if (st != PKV_OK) return st;
    return cuda_status(launch_window(a, dims.head_dim, kv_dtype == PKV_KV_INT8, n_seqs, sms, (cudaStream_t)stream));
}

}  // extern "C"
