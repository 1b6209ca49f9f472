// write_slots.cu -- packed new K and V rows to the pool rows that a slot map names
// (pagedkv_batch.h, paged_kv_write_slots), as they are or quantised to int8.
//
// A piece is 16 elements of one head row: 32 bytes in, 32 or 16 bytes out.  A thread
// takes one piece of K or V; a warp's pieces lie behind one another in a row, and the
// row's slot is loaded beside them, so that the only dependent access is the store.
// Lanes of a head row (4 or 8 of them) share its largest element.
//
// Measured: 9550 rows of 8 heads of 128 12.5 to 13.7 us, 84 to 92 % of the copy rate; into int8
// pages 15.0 to 16.1, 55 to 58 %, with 32 warps of 64 registers on an SM; 64 rows 1.6 and 1.9.
// Not faster: K and V of a piece in one thread (14.3, 18.5), persistent threads that load a
// piece ahead (13.7, 21.8), fewer registers (spills: 23 to 30).
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"
#include "window.h"
#include "../../include/pagedkv_batch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

struct SlotArgs {
    const __nv_bfloat16 *k_new, *v_new;
    int64_t k_stride, v_stride;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales;
    const int64_t *slots;
    int64_t pool_rows, n_rows;
    int32_t n_kv_heads;
    int32_t *dev_status;
};

// int8_codes16's scale and codes without its branch: bf16 rows often hold half of their
// largest element, whose quotient is a tie, so most warps would take it.  The quotient is
// rounded as a division rounds it by Markstein's theorem (IBM J. Res. Dev. 34, 1990): with y
// the correctly rounded 1 / b and q within one ulp of a / b, the remainder r = a - b q is
// exact and q + r y, rounded once, is a / b correctly rounded.  The first step makes q such a
// one, the second rounds it.  (8 K tokens of 1024 elements in K and in V:
// 18.7 to 22.5 us -> 15.0, 64 tokens 2.5 -> 1.8.)  Scales below
// 2^-100, where r could be subnormal, and rows that are not finite go the other way.
__device__ __forceinline__ float int8_codes16_rounded(const float (&x)[16], float amax, uint32_t (&w)[4])
{
    const float scale = __fdiv_rn(amax, 127.0f);
    if (!(scale >= 7.888609e-31f && scale <= 3.0e38f)) return int8_codes16(x, amax, w);
    const float y = __frcp_rn(scale);
    uint32_t c[16];
    float sum = 0.f;                                            // no number if an element is none
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float q = __fmul_rn(x[e], y);
        q = __fmaf_rn(__fmaf_rn(-q, scale, x[e]), y, q);
        q = __fmaf_rn(__fmaf_rn(-q, scale, x[e]), y, q);
        q = __fadd_rn(q, 12582912.f);                           // 1.5 * 2^23: rounded to an integer, in the low byte
        c[e] = __float_as_uint(q);
        sum += q;
    }
    if (!(sum == sum)) return int8_codes16(x, amax, w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    return scale;
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads) write_slots_kernel(const SlotArgs a)
{
    constexpr int SLOTS = D / 16;                        // lanes per head row
    grid_dependents_launch();   // a programmatic dependent: nothing is read before the wait
    grid_dependency_wait();
    const int32_t per_row = a.n_kv_heads * SLOTS;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, half = i / per_row;
    const int32_t piece = (int32_t)(i - half * per_row);
    const int64_t r = half >> 1;
    const bool is_v = half & 1, live = r < a.n_rows;     // (alike for the lanes of a head row)
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    int64_t row = -1;
    if (live) {
        const uint4 *src = reinterpret_cast<const uint4 *>((is_v ? a.v_new + r * a.v_stride : a.k_new + r * a.k_stride) + piece * 16);
        x0 = __ldcs(src);
        x1 = __ldcs(src + 1);
        row = a.slots[r];
        if (row >= a.pool_rows) {
            if (piece == 0 && !is_v) report(a.dev_status, PKV_DEV_BAD_POSITION);
            row = -1;
        }
    }
    const int64_t at = row * a.n_kv_heads * D + (int64_t)piece * 16;
    if constexpr (!INT8) {
        if (row < 0) return;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_v ? a.v_pool : a.k_pool) + at);
        dst[0] = x0;
        dst[1] = x1;
    } else {
        float x[16];
        unpack_bf16x8(x0, x);
        unpack_bf16x8(x1, x + 8);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
        for (int off = 1; off < SLOTS; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        uint32_t w[4];
        const float scale = int8_codes16_rounded(x, amax, w);
        if (row < 0) return;
        *reinterpret_cast<uint4 *>(static_cast<int8_t *>(is_v ? a.v_pool : a.k_pool) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        if (piece % SLOTS == 0) (is_v ? a.v_scales : a.k_scales)[row * a.n_kv_heads + piece / SLOTS] = scale;
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int paged_kv_write_slots(const pkv_bf16 *k_new, int64_t k_stride, const pkv_bf16 *v_new, int64_t v_stride,
                                    void *k_pool, void *v_pool, float *k_scales, float *v_scales, int32_t kv_dtype,
                                    pkv_dims dims, const int64_t *slots, int32_t n_rows, int32_t *dev_status,
                                    pkv_stream_t stream)
{
    const int st = check_dims(dims);
    if (st != PKV_OK) return st;
    if (n_rows < 0) return PKV_ERR_INVALID_ARG;
    if (kv_dtype != PKV_KV_BF16 && kv_dtype != PKV_KV_INT8) return PKV_ERR_UNSUPPORTED;
    if (!row_stride_ok(k_stride, dims.n_kv_heads, dims.head_dim) || !row_stride_ok(v_stride, dims.n_kv_heads, dims.head_dim))
        return PKV_ERR_INVALID_ARG;
    if (n_rows == 0) return PKV_OK;
    const void *p[] = {k_new, v_new, k_pool, v_pool};
    for (const void *x : p)
        if (!x || !aligned16(x)) return PKV_ERR_INVALID_ARG;
    if (!slots || (reinterpret_cast<uintptr_t>(slots) & 7u)) return PKV_ERR_INVALID_ARG;
    const bool int8 = kv_dtype == PKV_KV_INT8;
    if (int8 && (!k_scales || !v_scales ||
                 ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3u)))
        return PKV_ERR_INVALID_ARG;
    SlotArgs a{reinterpret_cast<const __nv_bfloat16 *>(k_new), reinterpret_cast<const __nv_bfloat16 *>(v_new), k_stride,
               v_stride, k_pool, v_pool, k_scales, v_scales, slots, (int64_t)(dims.n_blocks + 1) * dims.block_size, n_rows,
               dims.n_kv_heads, dev_status};
    const int64_t pieces = 2 * (int64_t)n_rows * dims.n_kv_heads * (dims.head_dim / 16);
    const int64_t grid = (pieces + kThreads - 1) / kThreads;
    if (grid > 0x7fffffffLL) return PKV_ERR_OUT_OF_RANGE;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)grid);
    lc.blockDim = dim3(kThreads);
    lc.stream = (cudaStream_t)stream;
    lc.attrs = pdl;
    lc.numAttrs = 1;
    cudaError_t e;
    if (dims.head_dim == 128)
        e = int8 ? cudaLaunchKernelEx(&lc, write_slots_kernel<128, true>, a) : cudaLaunchKernelEx(&lc, write_slots_kernel<128, false>, a);
    else
        e = int8 ? cudaLaunchKernelEx(&lc, write_slots_kernel<64, true>, a) : cudaLaunchKernelEx(&lc, write_slots_kernel<64, false>, a);
    return cuda_status(e);
}
