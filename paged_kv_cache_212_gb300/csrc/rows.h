// rows.h -- internal interface of the calls over packed query rows (pagedkv_batch.h):
// cross attention, and the decode of groups that share their first tokens.
#pragma once

#include "window.h"

namespace pkv {

constexpr int kMaxCtas = 192;      // CTAs that share out the keys of runs
constexpr int kUnitRows = 256;     // query head rows of a unit

// Where the rows kernel leaves what it has of a (row, query head), unnormalised in 32 bits.
// The keys of a run are cut at the borders of the CTAs' shares.  The first piece of every
// row, and how many there are, stand at the row's own place:
//   stat[row * Hq + head]  (maximum in log2 units, sum, first CTA, last CTA as int bits;
//                           first CTA -1: the row is finished, nothing is to be joined)
//   first[row * Hq + head][D]
// and what CTAs first + 1 .. last add to it at their own, a unit's row each:
//   cont_ml[cta][256]  (maximum, sum), cont[cta][256][D].
struct RowsPartials {
    float4 *stat;
    float *first;
    float2 *cont_ml;
    float *cont;
};

inline size_t rows_workspace_bytes(int64_t n_rows, int32_t n_q_heads, int32_t head_dim)
{
    const size_t rows = (size_t)n_rows * (size_t)n_q_heads, cont = (size_t)kMaxCtas * kUnitRows;
    return (rows + cont) * (size_t)head_dim * sizeof(float) + rows * sizeof(float4) + cont * sizeof(float2);
}

inline RowsPartials carve_rows_workspace(void *ws, int64_t n_rows, int32_t n_q_heads, int32_t head_dim)
{
    const size_t rows = (size_t)n_rows * (size_t)n_q_heads, cont = (size_t)kMaxCtas * kUnitRows;
    RowsPartials p;
    p.cont = static_cast<float *>(ws);
    p.first = p.cont + cont * head_dim;
    p.stat = reinterpret_cast<float4 *>(p.first + rows * head_dim);
    p.cont_ml = reinterpret_cast<float2 *>(p.stat + rows);
    return p;
}

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
    RowsPartials partials;
    int32_t *dev_status;
};

// Run g's rows and keys, none of either where they are bad.
struct Run {
    int32_t row0, rows, len;
    bool good;
};

#ifdef __CUDACC__
// (Read past the L1, which a kernel that starts before its predecessor ends may find as an
// earlier kernel left it.)
__device__ __forceinline__ Run run_at(const int32_t *starts, const int32_t *run_lens, int32_t n_rows, int32_t max_run_blocks,
                                      int32_t block_size, int32_t g)
{
    Run r;
    const int32_t a = __ldcg(starts + g), b = __ldcg(starts + g + 1);
    r.len = __ldcg(run_lens + g);
    r.row0 = a;
    r.rows = b - a;
    r.good = true;
    if (a < 0 || b < a || b > n_rows) {
        r.row0 = r.rows = 0;
        r.good = false;
    }
    if (r.len < 0 || (int64_t)r.len > (int64_t)max_run_blocks * block_size) {
        r.len = 0;
        r.good = false;
    }
    return r;
}

// The run of a row: the last g with starts[g] <= row, if row < starts[g + 1]; else -1.
__device__ __forceinline__ int32_t run_of(const int32_t *starts, int32_t n_runs, int32_t row)
{
    int32_t lo = -1, hi = n_runs;
    while (hi - lo > 1) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (__ldcg(starts + mid) <= row)
            lo = mid;
        else
            hi = mid;
    }
    return lo >= 0 && row < __ldcg(starts + lo + 1) ? lo : -1;
}
#endif

// The runs' keys: partials (decode), or outputs where a CTA has all of a row's keys.
cudaError_t launch_rows_tc(const RowsArgs &a, int num_sms, cudaStream_t stream);
// Behind it, a decode: the sequences' own keys, joined with those partials.
cudaError_t launch_shared_rest(const RowsArgs &a, int num_sms, cudaStream_t stream);
// Behind it: joins the partials of a cross attention's rows.
cudaError_t launch_rows_join(const RowsArgs &a, cudaStream_t stream);

}  // namespace pkv
