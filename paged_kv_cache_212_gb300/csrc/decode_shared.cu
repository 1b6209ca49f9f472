// decode_shared.cu -- decode_window.cuh's kernels over runs (rows.h).
//
// launch_rows_rest: the tokens of a decode's sequences behind those that their group shares,
// whose partials are joined with those of the group's tokens (rows_tc.cu).  The launch is a
// programmatic dependent of the rows kernel, which lets it start as soon as its own CTAs run:
// these units fill the SMs that the group's tiles leave to them.
//
// launch_rows_whole: a run's tokens and a row's own, each row by itself, in one launch, for all
// rows or for those of short runs.
#include "decode_window.cuh"
#include "../../include/pagedkv_batch.h"

namespace pkv {

namespace {

WindowArgs window_args(const RowsArgs &r)
{
    WindowArgs a{};
    const pkv_dims &dims = r.dims;
    a.q = static_cast<const __nv_bfloat16 *>(r.q);
    a.q_stride = r.q_stride;
    a.n_q_heads = r.n_q_heads;
    a.group = r.n_q_heads / dims.n_kv_heads;
    a.k_pool = const_cast<void *>(r.k_pool);
    a.v_pool = const_cast<void *>(r.v_pool);
    a.k_scales = const_cast<float *>(r.k_scales);
    a.v_scales = const_cast<float *>(r.v_scales);
    a.n_blocks = dims.n_blocks;
    a.block_size = dims.block_size;
    a.n_kv_heads = dims.n_kv_heads;
    set_block_lookup(a, dims.block_size);
    a.tables = r.tables;
    a.max_blocks = r.max_blocks;
    a.ctx_lens = r.ctx_lens;
    a.scale_log2 = r.softmax_scale * 1.4426950408889634f;
    a.window = 0x7fffffff;
    a.out = static_cast<__nv_bfloat16 *>(r.out);
    a.lse_out = r.lse_out;
    a.dev_status = r.dev_status;
    a.run_starts = r.starts;
    a.run_lens = r.run_lens;
    a.run_tables = r.run_tables;
    a.n_runs = r.n_runs;
    a.max_run_blocks = r.max_run_blocks;
    a.n_rows = r.n_rows;
    a.part = r.partials;
    a.after_rows = r.n_runs > 0 && r.few < kAllRows;
    a.few = r.few;
    return a;
}

template <int RUNS>
cudaError_t launch_over(const RowsArgs &r, int64_t tokens, int sms, cudaStream_t stream)
{
    WindowArgs a = window_args(r);
    const int64_t units = (int64_t)r.n_rows * r.dims.n_kv_heads, tiles = (tokens + kTile - 1) / kTile;
    const bool wide = a.group > 4;
    if (r.dims.head_dim == 128) {
        if (r.kv_dtype == PKV_KV_INT8) return launch_sized<128, true, true, RUNS>(a, units, tiles, sms, stream);
        return wide ? launch_sized<128, false, true, RUNS>(a, units, tiles, sms, stream)
                    : launch_sized<128, false, false, RUNS>(a, units, tiles, sms, stream);
    }
    if (r.kv_dtype == PKV_KV_INT8) return launch_sized<64, true, true, RUNS>(a, units, tiles, sms, stream);
    return wide ? launch_sized<64, false, true, RUNS>(a, units, tiles, sms, stream)
                : launch_sized<64, false, false, RUNS>(a, units, tiles, sms, stream);
}

}  // namespace

cudaError_t launch_rows_rest(const RowsArgs &r, int sms, cudaStream_t stream)
{
    return launch_over<kRest>(r, (int64_t)r.max_blocks * r.dims.block_size, sms, stream);
}

cudaError_t launch_rows_whole(const RowsArgs &r, int sms, cudaStream_t stream)
{
    // (a decode: a tile more where the run ends inside one)
    const int64_t tokens = r.ctx_lens ? (int64_t)r.max_blocks * r.dims.block_size + kTile : (int64_t)r.max_run_blocks * r.dims.block_size;
    return launch_over<kWhole>(r, tokens, sms, stream);
}

}  // namespace pkv
