// rows.cu -- the calls over packed query rows (pagedkv_batch.h): host checks and a
// kernel that is right for every case, a CTA for each row and query head.
#include <math.h>

#include "common.cuh"
#include "rows.h"
#include "../../include/pagedkv_batch.h"

namespace pkv {
namespace {

constexpr int kWarps = 4;

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

template <int D, bool INT8>
__global__ void __launch_bounds__(32 * kWarps) rows_plain_kernel(const RowsArgs a)
{
    constexpr int PER = D / 32;                      // elements of a lane
    __shared__ float m_s[kWarps], l_s[kWarps], o_s[kWarps][D];
    grid_dependents_launch();   // a programmatic dependent: nothing is read before the wait
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t r = (int32_t)blockIdx.x, head = (int32_t)blockIdx.y, bs = a.dims.block_size, hkv = a.dims.n_kv_heads;
    const int32_t kvh = head / (a.n_q_heads / hkv);
    if (r == 0 && head == 0)
        for (int32_t i = threadIdx.x; i <= a.n_runs && a.n_runs > 0; i += blockDim.x) {
            const int32_t x = __ldg(a.starts + i);
            if (x < 0 || x > a.n_rows || (i > 0 && x < __ldg(a.starts + i - 1))) report(a.dev_status, PKV_DEV_BAD_LENGTH);
        }
    const int32_t g = run_of(a.starts, a.n_runs, r);
    const bool decode = a.ctx_lens != nullptr;
    if (g < 0 && !decode) return;                    // a row of no sequence
    int32_t run = g < 0 ? 0 : __ldg(a.run_lens + g), ctx = decode ? __ldg(a.ctx_lens + r) : run;
    if (run < 0 || (int64_t)run > (int64_t)a.max_run_blocks * bs || ctx < 0 || (decode && (int64_t)ctx > (int64_t)a.max_blocks * bs)) {
        if (threadIdx.x == 0 && head == 0) report(a.dev_status, PKV_DEV_BAD_LENGTH);
        run = ctx = 0;
    }
    float q[PER], o[PER], m = -INFINITY, l = 0.f;
    const __nv_bfloat16 *q_row = static_cast<const __nv_bfloat16 *>(a.q) + r * a.q_stride + (int64_t)head * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        q[e] = __bfloat162float(q_row[e]) * a.softmax_scale;
        o[e] = 0.f;
    }
    for (int32_t t = warp; t < ctx; t += kWarps) {
        const int32_t *row = t < run ? a.run_tables + (int64_t)g * a.max_run_blocks : a.tables + (int64_t)r * a.max_blocks;
        const int32_t b = __ldg(row + t / bs);
        float k[PER], v[PER];
        if (b < 0 || b > a.dims.n_blocks) {
            if (lane == 0) report(a.dev_status, PKV_DEV_BAD_BLOCK_ID);
#pragma unroll
            for (int e = 0; e < PER; ++e) k[e] = v[e] = 0.f;
        } else {
            const int64_t at = ((int64_t)b * bs + t % bs) * hkv + kvh;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int64_t x = at * D + lane * PER + e;
                k[e] = INT8 ? (float)static_cast<const int8_t *>(a.k_pool)[x] * a.k_scales[at]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.k_pool)[x]);
                v[e] = INT8 ? (float)static_cast<const int8_t *>(a.v_pool)[x] * a.v_scales[at]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v_pool)[x]);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) s += q[e] * k[e];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - top), p = expf(s - top);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = o[e] * f + p * v[e];
    }
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) o_s[warp][lane * PER + e] = o[e];
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w]);
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        const float f = m_s[w] == -INFINITY ? 0.f : expf(m_s[w] - top);
        sum += l_s[w] * f;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] += o_s[w][lane * PER + e] * f;
    }
    const int64_t out_row = (int64_t)r * a.n_q_heads + head;
#pragma unroll
    for (int e = 0; e < PER; ++e)
        static_cast<__nv_bfloat16 *>(a.out)[out_row * D + lane * PER + e] = __float2bfloat16(sum > 0.f ? o[e] / sum : 0.f);
    if (lane == 0 && a.lse_out) a.lse_out[out_row] = sum > 0.f ? top + logf(sum) : -INFINITY;
}

}  // namespace

static cudaError_t launch_rows(const RowsArgs &a, int num_sms, cudaStream_t stream)
{
    if (a.kv_dtype == PKV_KV_BF16) {
        if (a.n_runs > 0) {
            const cudaError_t e = launch_rows_tc(a, num_sms, stream);
            if (e != cudaSuccess) return e;
        }
        if (a.ctx_lens) {
            const cudaError_t e = launch_shared_rest(a, num_sms, stream);
            if (e != cudaSuccess) return e;
        }
        return launch_rows_join(a, num_sms, stream);
    }
    const dim3 grid((unsigned)a.n_rows, (unsigned)a.n_q_heads);
    if (a.dims.head_dim == 128) {
        rows_plain_kernel<128, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    } else {
        rows_plain_kernel<64, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

namespace {

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
