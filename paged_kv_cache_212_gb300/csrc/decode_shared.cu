// decode_shared.cu -- the tokens of a decode's sequences behind those that their group
// shares: decode_window.cuh's kernels over tokens prefix_lens[g] .. ctx_lens[s] - 1, whose
// partials are joined with those of the group's tokens (rows_tc.cu).
//
// The launch is a programmatic dependent of the rows kernel, which lets it start as soon as
// its own CTAs run: these units fill the SMs that the group's tiles leave to them.
#include "decode_window.cuh"
#include "../../include/pagedkv_batch.h"

namespace pkv {

cudaError_t launch_shared_rest(const RowsArgs &r, int sms, cudaStream_t stream)
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
    a.group_starts = r.starts;
    a.prefix_lens = r.run_lens;
    a.n_groups = r.n_runs;
    a.max_prefix_blocks = r.max_run_blocks;
    a.n_seqs = r.n_rows;
    a.part = r.partials;
    a.after_rows = r.n_runs > 0;
    const int64_t units = (int64_t)r.n_rows * dims.n_kv_heads;
    const int64_t tiles = ((int64_t)r.max_blocks * dims.block_size + kTile - 1) / kTile;
    const bool wide = a.group > 4;
    if (dims.head_dim == 128) {
        if (r.kv_dtype == PKV_KV_INT8) return launch_sized<128, true, true, true>(a, units, tiles, sms, stream);
        return wide ? launch_sized<128, false, true, true>(a, units, tiles, sms, stream)
                    : launch_sized<128, false, false, true>(a, units, tiles, sms, stream);
    }
    if (r.kv_dtype == PKV_KV_INT8) return launch_sized<64, true, true, true>(a, units, tiles, sms, stream);
    return wide ? launch_sized<64, false, true, true>(a, units, tiles, sms, stream)
                : launch_sized<64, false, false, true>(a, units, tiles, sms, stream);
}

}  // namespace pkv
