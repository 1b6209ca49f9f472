// rows.h -- internal interface of the calls over packed query rows (pagedkv_batch.h):
// cross attention, and the decode of groups that share their first tokens.
#pragma once

#include "window.h"

namespace pkv {

// Packed query rows, each of which sees keys of two runs, one behind the other.  Rows
// starts[g] .. starts[g + 1] - 1 are run g's; all of them see its keys 0 .. run_lens[g] - 1
// at run_tables[g].  In a decode (ctx_lens not null) row s is a sequence, which sees of its
// run's keys those below ctx_lens[s], and goes on with keys run_lens[g] .. ctx_lens[s] - 1
// of its own at tables[s].
struct RowsArgs {
    const void *q;
    int64_t q_stride;
    int32_t n_q_heads, n_rows;
    const void *k_pool, *v_pool;
    const float *k_scales, *v_scales;
    int32_t kv_dtype;
    pkv_dims dims;
    const int32_t *starts, *run_tables, *run_lens;
    int32_t n_runs, max_run_blocks;
    const int32_t *tables, *ctx_lens;
    int32_t max_blocks;
    float softmax_scale;
    void *out;
    float *lse_out;
    int32_t *dev_status;
};

cudaError_t launch_rows(const RowsArgs &a, int num_sms, cudaStream_t stream);

}  // namespace pkv
