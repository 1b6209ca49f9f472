// rope_write.cu -- rotary positions and the page write in one launch
// (pagedkv_rope.h): queries and keys turned by the angles of their positions,
// keys and values stored in the pages (bf16, or int8 codes with a scale per
// row), turned queries returned.
//
// Every element is read once and written once, so the launch is bound by
// memory (prefill chunks) or by its own latency (decode tokens).  A block takes
// one token: its threads compute the token's sines and cosines once, one pair
// each, while the rows they will turn are on their way; a warp holds several of
// the token's head rows (Hq + 2 Hkv of them) at once, D / 16 lanes a row (rope.cuh).
//
// Measured (32 query and 8 kv heads of 128, kernels back to back in a graph): a chunk
// of 8 x 512 tokens 17.2 us = 5.9 TB/s, 86 % of the copy rate, of which 2.1 us are a
// launch of one token; 64 tokens of one position each 2.4 us; 5 x 301 tokens into
// int8 pages 10.2 us, 8 x 512 of them 23 us (4.0 TB/s: 110 registers a thread leave
// 16 warps on an SM, whose instructions wait for one another).  Rows are loaded before
// the position is known, and sines and cosines shared by the block: 22.8 -> 18.6 us on
// the chunk; read and written once, so loads and stores are streamed: 18.6 -> 17.6.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "rope.cuh"
#include "window.h"
#include "write_rows.cuh"

namespace pkv {
namespace {

struct RopeWriteArgs {
    const __nv_bfloat16 *q, *k_new, *v_new;
    int64_t q_stride, k_stride, v_stride;
    int32_t n_q_heads;
    RopeArgs rope;
    __nv_bfloat16 *q_out;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales;
    pkv_dims dims;
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *start_pos;
    int32_t n_new;
    int32_t *dev_status;
};

// Warps of a block and groups of head rows that a warp holds at once.  Chunks take
// narrow blocks (4 warps, 3 groups: 48 rows of 128 elements in one go), many of
// them on an SM; a few tokens take wide ones, while all of their blocks are
// resident at once.  Measured, narrow / wide: 64 tokens 2.5 / 2.3 us (bf16 pages),
// 3.3 / 3.1 (int8); 600 tokens 3.6 / 3.4 and 4.6 / 6.5; 1024 tokens 5.5 / 6.9 and
// 7.9 / 11.6; 4096 tokens 17.2 / 19.5 and 23 / 35.
constexpr int kNarrowWarps = 4, kNarrowGroups = 3;
constexpr int kWideWarps = 8, kWideGroups = 2;
// blocks that are resident on an SM; the registers are bounded to it (narrow blocks
// for bf16 pages on 4096 tokens: 18.3 us with 5, 17.2 with 6, 17.6 with 8; one more
// for int8 pages spills)
template <bool INT8>
constexpr int wide_blocks() { return INT8 ? 2 : 4; }
template <bool INT8>
constexpr int narrow_blocks() { return INT8 ? 4 : 6; }

template <int D, bool INT8, bool WIDE>
__global__ void __launch_bounds__(32 * (WIDE ? kWideWarps : kNarrowWarps), WIDE ? wide_blocks<INT8>() : narrow_blocks<INT8>())
    rope_write_kernel(const RopeWriteArgs a)
{
    constexpr int kGroups = WIDE ? kWideGroups : kNarrowGroups;
    constexpr int SLOTS = D / 16;        // lanes per head row
    constexpr int ROWS = 32 / SLOTS;     // head rows in a group
    __shared__ __align__(16) float cos_s[D / 2], sin_s[D / 2];
    grid_dependents_launch();   // a programmatic dependent: nothing is read before the wait
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, slot = lane % SLOTS, sub = lane / SLOTS;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int hkv = a.dims.n_kv_heads, hq = a.n_q_heads;
    const int n_rows = hq + 2 * hkv;
    const int64_t tok = blockIdx.x;
    int v0, v1;
    const bool turn = rope_vectors(a.rope, slot, v0, v1);
    uint4 x0[kGroups], x1[kGroups];
    auto load = [&](int g0) {            // the warp's groups g0, g0 + warps, ...
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int r = (g0 + i * warps) * ROWS + sub;
            x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
            if (r >= n_rows) continue;
            const __nv_bfloat16 *src = r < hq         ? a.q + tok * a.q_stride + (int64_t)r * D
                                       : r < hq + hkv ? a.k_new + tok * a.k_stride + (int64_t)(r - hq) * D
                                                      : a.v_new + tok * a.v_stride + (int64_t)(r - hq - hkv) * D;
            x0[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + v0);
            x1[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + v1);
        }
    };
    load(warp);
    const int64_t s = (uint32_t)blockIdx.x / (uint32_t)a.n_new;
    const int64_t t = (int64_t)__ldg(a.start_pos + s) + (tok - s * a.n_new);
    for (int i = threadIdx.x; i < a.rope.rot_dim / 2; i += blockDim.x) rope_angle(a.rope, i, t, cos_s[i], sin_s[i]);
    const int64_t row = pool_row_of(a.tables + s * a.max_blocks, a.max_blocks, a.dims.n_blocks, a.dims.block_size, t,
                                    threadIdx.x == 0 ? a.dev_status : nullptr);
    __syncthreads();
    float c[8], sn[8];
    if (turn) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float4 *>(c + 4 * i) = *reinterpret_cast<const float4 *>(cos_s + 8 * slot + 4 * i);
            *reinterpret_cast<float4 *>(sn + 4 * i) = *reinterpret_cast<const float4 *>(sin_s + 8 * slot + 4 * i);
        }
    }
    for (int g0 = warp; g0 * ROWS < n_rows; g0 += kGroups * warps) {
        if (g0 != warp) load(g0);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int r0 = (g0 + i * warps) * ROWS, r = r0 + sub;
            if (r0 >= n_rows) break;
            const bool is_q = r < hq, is_v = r >= hq + hkv, live = r < n_rows;
            const int h = is_q ? r : is_v ? r - hq - hkv : r - hq;
            if (!INT8 || is_q) {
                if (turn && !is_v) {
                    float x[16];
                    unpack_bf16x8(x0[i], x);
                    unpack_bf16x8(x1[i], x + 8);
                    rope_turn(a.rope.interleaved, c, sn, x);
                    x0[i] = pack_bf16x8(x);
                    x1[i] = pack_bf16x8(x + 8);
                }
                if (live && (is_q || row >= 0)) {
                    __nv_bfloat16 *dst = is_q ? a.q_out + (tok * hq + h) * D
                                              : static_cast<__nv_bfloat16 *>(is_v ? a.v_pool : a.k_pool) + (row * hkv + h) * D;
                    __stcs(reinterpret_cast<uint4 *>(dst) + v0, x0[i]);
                    __stcs(reinterpret_cast<uint4 *>(dst) + v1, x1[i]);
                }
            }
            if constexpr (INT8) {
                if (r0 + ROWS <= hq) continue;        // no row of the pages in this group
                float x[16];
                unpack_bf16x8(x0[i], x);
                unpack_bf16x8(x1[i], x + 8);
                if (turn && !is_v && !is_q) rope_turn(a.rope.interleaved, c, sn, x);
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
                for (int off = 1; off < SLOTS; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                uint32_t w[4];
                const float scale = int8_codes16(x, amax, w);
                if (is_q || !live || row < 0) continue;
                int8_t *dst = static_cast<int8_t *>(is_v ? a.v_pool : a.k_pool) + (row * hkv + h) * D;
                *reinterpret_cast<uint2 *>(dst + 8 * v0) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2 *>(dst + 8 * v1) = make_uint2(w[2], w[3]);
                if (slot == 0) (is_v ? a.v_scales : a.k_scales)[row * hkv + h] = scale;
            }
        }
    }
}

}  // namespace

int check_rope(const pkv_rope *rope, int32_t head_dim)
{
    if (!rope || !rope->phases || !aligned16(rope->phases) || !std::isfinite((float)rope->magnitude))
        return PKV_ERR_INVALID_ARG;
    if (rope->rot_dim <= 0 || rope->rot_dim > head_dim) return PKV_ERR_INVALID_ARG;
    if (rope->rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

bool row_stride_ok(int64_t stride, int32_t heads, int32_t head_dim)
{
    return stride % 8 == 0 && stride >= (int64_t)heads * head_dim;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_rope_phases(int32_t rot_dim, double base, int32_t scaling, double factor, double original_context,
                    double low_turns, double high_turns, uint64_t *phases_out, double *magnitude_out)
{
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    if (!phases_out || !magnitude_out || rot_dim <= 0 || rot_dim % 16 != 0) return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(base) || !(base > 1.0)) return PKV_ERR_INVALID_ARG;
    if (scaling < PKV_ROPE_NONE || scaling > PKV_ROPE_YARN) return PKV_ERR_UNSUPPORTED;
    if (scaling != PKV_ROPE_NONE && (!std::isfinite(factor) || !(factor >= 1.0))) return PKV_ERR_INVALID_ARG;
    const bool by_turns = scaling == PKV_ROPE_BANDS || scaling == PKV_ROPE_YARN;
    if (by_turns && (!std::isfinite(original_context) || !(original_context > 0.0) || !(low_turns > 0.0) ||
                     !(high_turns > low_turns) || !std::isfinite(high_turns)))
        return PKV_ERR_INVALID_ARG;
    *magnitude_out = scaling == PKV_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    if (scaling == PKV_ROPE_NTK) base *= pow(factor, rot_dim / (rot_dim - 2.0));
    // YARN: the (real) pair index that makes n turns in the original context
    const auto pair_of = [&](double n) { return rot_dim * log(original_context / (n * kTwoPi)) / (2.0 * log(base)); };
    double lo = 0.0, hi = 0.0;
    if (scaling == PKV_ROPE_YARN) {
        lo = fmax(floor(pair_of(high_turns)), 0.0);
        hi = fmin(ceil(pair_of(low_turns)), rot_dim - 1.0);
    }
    for (int32_t i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        double divide = 0.0;                 // 0: f kept, 1: f / factor
        if (scaling == PKV_ROPE_LINEAR) divide = 1.0;
        if (scaling == PKV_ROPE_BANDS) {
            const double n = original_context * f / kTwoPi;
            divide = 1.0 - fmin(fmax((n - low_turns) / (high_turns - low_turns), 0.0), 1.0);
        }
        if (scaling == PKV_ROPE_YARN) divide = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
        if (divide != 0.0) f = f * (1.0 - divide) + f / factor * divide;
        // f <= 1 radian per position: less than a sixth of 2^64
        phases_out[i] = (uint64_t)(f / kTwoPi * 18446744073709551616.0 + 0.5);
    }
    return PKV_OK;
}

int paged_kv_write_rope(const pkv_bf16 *q, int64_t q_stride, int32_t n_q_heads, const pkv_bf16 *k_new,
                        int64_t k_stride, const pkv_bf16 *v_new, int64_t v_stride, const pkv_rope *rope,
                        pkv_bf16 *q_out, void *k_pool, void *v_pool, float *k_scales, float *v_scales,
                        int32_t kv_dtype, pkv_dims dims, const int32_t *block_tables, int32_t max_blocks,
                        const int32_t *start_pos, int32_t n_seqs, int32_t n_new, int32_t *dev_status,
                        pkv_stream_t stream)
{
    int st = check_dims(dims);
    if (st != PKV_OK) return st;
    if (n_seqs < 0 || n_new < 0 || max_blocks <= 0 || n_q_heads <= 0) return PKV_ERR_INVALID_ARG;
    if (kv_dtype != PKV_KV_BF16 && kv_dtype != PKV_KV_INT8) return PKV_ERR_UNSUPPORTED;
    st = check_rope(rope, dims.head_dim);
    if (st != PKV_OK) return st;
    if (!row_stride_ok(q_stride, n_q_heads, dims.head_dim) || !row_stride_ok(k_stride, dims.n_kv_heads, dims.head_dim) ||
        !row_stride_ok(v_stride, dims.n_kv_heads, dims.head_dim))
        return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0 || n_new == 0) return PKV_OK;
    const void *p[] = {q, k_new, v_new, q_out, k_pool, v_pool};
    for (const void *x : p)
        if (!x || !aligned16(x)) return PKV_ERR_INVALID_ARG;
    if (!block_tables || !start_pos) return PKV_ERR_INVALID_ARG;
    // a turned row may be written before another warp has read its source
    if (q_out == q && q_stride != (int64_t)n_q_heads * dims.head_dim) return PKV_ERR_INVALID_ARG;
    const bool int8 = kv_dtype == PKV_KV_INT8;
    if (int8 && (!k_scales || !v_scales ||
                 ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3u)))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)n_new > (int64_t)max_blocks * dims.block_size) return PKV_ERR_OUT_OF_RANGE;
    if ((int64_t)n_seqs * n_new > 0x7fffffffLL) return PKV_ERR_OUT_OF_RANGE;
    int sms = 0;
    st = num_sms_of_current_device(&sms);
    if (st != PKV_OK) return st;

    RopeWriteArgs a{};
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.k_new = reinterpret_cast<const __nv_bfloat16 *>(k_new);
    a.v_new = reinterpret_cast<const __nv_bfloat16 *>(v_new);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.n_q_heads = n_q_heads;
    a.rope = rope_args(rope->phases, rope->rot_dim, rope->interleaved, rope->magnitude);
    a.q_out = reinterpret_cast<__nv_bfloat16 *>(q_out);
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.dims = dims;
    a.tables = block_tables;
    a.max_blocks = max_blocks;
    a.start_pos = start_pos;
    a.n_new = n_new;
    a.dev_status = dev_status;
    const int64_t tokens = (int64_t)n_seqs * n_new;
    const int rows_at_once = 32 / (dims.head_dim / 16);
    const int64_t groups = (n_q_heads + 2 * (int64_t)dims.n_kv_heads + rows_at_once - 1) / rows_at_once;
    const bool wide = tokens <= (int64_t)sms * (int8 ? wide_blocks<true>() : wide_blocks<false>());
    const int64_t most = wide ? kWideWarps : kNarrowWarps;
    const int warps = (int)(groups < most ? groups : most);
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)tokens);
    lc.blockDim = dim3((unsigned)(32 * warps));
    lc.stream = (cudaStream_t)stream;
    lc.attrs = pdl;
    lc.numAttrs = 1;
    cudaError_t e;
    if (dims.head_dim == 128)
        e = int8 ? (wide ? cudaLaunchKernelEx(&lc, rope_write_kernel<128, true, true>, a)
                         : cudaLaunchKernelEx(&lc, rope_write_kernel<128, true, false>, a))
                 : (wide ? cudaLaunchKernelEx(&lc, rope_write_kernel<128, false, true>, a)
                         : cudaLaunchKernelEx(&lc, rope_write_kernel<128, false, false>, a));
    else
        e = int8 ? (wide ? cudaLaunchKernelEx(&lc, rope_write_kernel<64, true, true>, a)
                         : cudaLaunchKernelEx(&lc, rope_write_kernel<64, true, false>, a))
                 : (wide ? cudaLaunchKernelEx(&lc, rope_write_kernel<64, false, true>, a)
                         : cudaLaunchKernelEx(&lc, rope_write_kernel<64, false, false>, a));
    return cuda_status(e);
}

}  // extern "C"
