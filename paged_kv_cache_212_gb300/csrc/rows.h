// rows.h -- internal interface of the calls over packed query rows (pagedkv_batch.h):
// cross attention, and the decode of groups that share their first tokens.
#pragma once

#include "window.h"

namespace pkv {

constexpr int kMaxCtas = 192;      // CTAs that share out the keys of runs
constexpr int kUnitRows = 256;     // query head rows of a unit

// Where the rows kernel leaves what it has of a (row, query head), unnormalised in 32 bits.
// The keys of a run are cut at the borders of the CTAs' shares.  The first piece of every
// row of a cut unit (in a decode: of every row) stands at the row's own place:
//   stat[row * Hq + head]  (maximum in log2 units, sum, first CTA, last CTA as int bits)
//   first[kv head][D / 8][row * G + g][8]
// and what CTAs first + 1 .. last add to it at their own, a unit's row each:
//   cont_ml[cta][256]  (maximum, sum), cont[cta][D / 8][256][8].
// (Threads hold neighbouring rows, so 8 values of each lie beside one another: with rows of
// D values the 256 x D store of a unit took 4 us.)
// A decode's own tokens: own_stat[row * Hq + head] (maximum, sum, as int bits where the row's
// first query head lies in its unit, -1 where no run is to be joined or kDone where the outputs
// are written by another launch), own[row * Hq + head][D].
// cuts[cta]: the cut unit that begins in that CTA, the last one of its share.
struct CutUnit {
    int32_t pos, pos_end, kvh, last_cta;   // last_cta 0: none
};
static_assert(sizeof(CutUnit) == 16, "read as one vector");
constexpr int kDone = -2;
struct RowsPartials {
    float4 *stat;
    float *first;
    float2 *cont_ml;
    float *cont;
    CutUnit *cuts;
    float *own;
    float4 *own_stat;
};

inline size_t rows_workspace_bytes(int64_t n_rows, int32_t n_q_heads, int32_t head_dim)
{
    const size_t rows = (size_t)n_rows * (size_t)n_q_heads, cont = (size_t)kMaxCtas * kUnitRows;
    return (2 * rows + cont) * (size_t)head_dim * sizeof(float) + rows * 2 * sizeof(float4) +
           cont * sizeof(float2) + kMaxCtas * sizeof(CutUnit);
}

inline RowsPartials carve_rows_workspace(void *ws, int64_t n_rows, int32_t n_q_heads, int32_t head_dim)
{
    const size_t rows = (size_t)n_rows * (size_t)n_q_heads, cont = (size_t)kMaxCtas * kUnitRows;
    RowsPartials p;
    p.cont = static_cast<float *>(ws);
    p.first = p.cont + cont * head_dim;
    p.own = p.first + rows * head_dim;
    p.stat = reinterpret_cast<float4 *>(p.own + rows * head_dim);
    p.own_stat = p.stat + rows;
    p.cuts = reinterpret_cast<CutUnit *>(p.own_stat + rows);
    p.cont_ml = reinterpret_cast<float2 *>(p.cuts + kMaxCtas);
    return p;
}

// Packed query rows, each of which sees keys of two runs, one behind the other.  Rows
// starts[g] .. starts[g + 1] - 1 are run g's; all of them see its keys 0 .. run_lens[g] - 1
// at run_tables[g].  In a decode (ctx_lens not null) row s is a sequence, which sees of its
// run's keys those below ctx_lens[s], and goes on with keys run_lens[g] .. ctx_lens[s] - 1
// of its own at tables[s].  Sequences that end before their run does (ctx_lens[s] < run_lens[g])
// are attended one by one, as they see other keys than the rest.
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
    int32_t few;                  // rows of runs of up to so many are attended one by one
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

// The run of a row, -1 for none, and what it is: the last g with starts[g] <= row, where
// row < starts[g + 1].  Asked by a whole warp: it narrows the runs down to 32 by the starts of
// 32 of them at a time, and then reads those.  (A row each for 1024 and 4096 sequences of 64
// keys: 213 and 1124 us when all starts before a row's were read, 113 and 290 so.)
__device__ __forceinline__ int32_t run_of(const int32_t *starts, const int32_t *run_lens, int32_t n_runs, int32_t n_rows,
                                          int32_t max_run_blocks, int32_t block_size, int32_t row, Run *out)
{
    const int lane = threadIdx.x & 31;
    int32_t g0 = 0, n = n_runs;                     // it is one of g0 .. g0 + n - 1
    while (n > 32) {
        const int32_t step = (int32_t)(((uint32_t)n + 31u) / 32u), at = lane * step;
        const uint32_t upto = __ballot_sync(0xffffffffu, at < n && __ldcg(starts + g0 + at) <= row);
        const int32_t skip = upto == 0 ? 0 : (31 - __clz(upto)) * step;
        g0 += skip;
        n = min(n - skip, step);
    }
    const int32_t g = g0 + lane;
    Run r{0, 0, 0, false};
    if (lane < n) r = run_at(starts, run_lens, n_rows, max_run_blocks, block_size, g);
    const uint32_t here = __ballot_sync(0xffffffffu, row - r.row0 >= 0 && row - r.row0 < r.rows);
    if (here == 0) {
        *out = Run{0, 0, 0, true};
        return -1;
    }
    const int src = __ffs(here) - 1;
    out->row0 = __shfl_sync(0xffffffffu, r.row0, src);
    out->rows = __shfl_sync(0xffffffffu, r.rows, src);
    out->len = __shfl_sync(0xffffffffu, r.len, src);
    out->good = __shfl_sync(0xffffffffu, (int)r.good, src);
    return g0 + src;
}
#endif

// The runs' keys: partials (decode), or outputs where a CTA has all of a row's keys.
cudaError_t launch_rows_tc(const RowsArgs &a, int num_sms, cudaStream_t stream);
// Behind it, a decode: the sequences' own keys, partials as well.
cudaError_t launch_rows_rest(const RowsArgs &a, int num_sms, cudaStream_t stream);
// Behind that: joins the partials.
cudaError_t launch_rows_join(const RowsArgs &a, int num_sms, cudaStream_t stream);

// The rows of runs of up to a.few, all of a row in one launch, each by itself; beside the rows
// kernel where there is one (a.few below kAllRows).
constexpr int32_t kAllRows = 0x7fffffff;
cudaError_t launch_rows_whole(const RowsArgs &a, int num_sms, cudaStream_t stream);

}  // namespace pkv
