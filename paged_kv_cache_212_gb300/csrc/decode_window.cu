// decode_window.cu -- decode attention under a sliding window with first tokens
// that stay visible (pagedkv_window.h), over bf16 or int8 pages, alone or as one
// layer's step with the rotary turn and the page write of the new token.
//
// The host knows how many tokens a query can see (window + sinks), so no plan
// and no workspace is needed: a (sequence, kv head) unit is the work of one
// thread-block cluster of 1 .. 8 CTAs, and its pieces are joined through the
// cluster's shared memory, all in one launch.
//
// The visible tokens of a sequence are counted through: c < first is token c,
// the rest continue at the window's first token.  Sixteen consecutive c make a
// tile; warp w of the cluster takes tiles w, w + n_warps, ...  A warp works alone:
// it looks its tiles' blocks up one tile ahead, copies their K and V rows (16
// bytes a lane, asynchronously) into a ring of its own, and contracts them with
// the G query heads of its kv head on the tensor cores (mma.sync m16n8k16):
//   S^T = K Q^T     16 tokens as M, query heads as N = 8
//   O^T += V^T P^T  head_dim as M, query heads as N, tokens as K
// with a running maximum and sum in log2 units.  No barrier but the warp's own
// until the end, where warps and then CTAs are joined by their maxima.
//
// Rounding.  bf16 pages: products are exact in binary32 when both factors are,
// so the queries of a step (turned in binary32) and the probabilities are split
// into a bf16 value and its bf16 remainder (2^-16 together).  With up to 4 query
// heads both fit in the 8 columns of the product (heads in columns 0-3,
// remainders in 4-7) and cost nothing; with 5 to 8 the remainders take a second
// product.
//
// int8 pages are contracted as fp16 (a code and the value 1152 share one
// exponent: a byte permute, and one subtraction or, for K, one correction by
// 1152 times the query's sum).  Queries and weights are rounded once to fp16
// (2^-11, eight times finer than the bf16 output).  The K scale multiplies the
// score; the V scale joins the probability as exp2(s + log2 |v_scale| - m2)
// under a maximum m2 of its own, so that the fp16 weights use their range
// whatever the scales are.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "rope.cuh"
#include "write_rows.cuh"
#include "../../include/pagedkv_window.h"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;              // tokens per tile
constexpr int kHeads = 8;              // query heads per kv head, padded
constexpr int kMaxSplits = 8;          // CTAs per cluster
constexpr int kCtasPerSm = 3;          // resident CTAs that fill an SM
constexpr float kLazyMax = 8.0f;       // the running maximum may lag by this (log2 units)

struct WindowArgs {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    int32_t n_q_heads, group;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales;
    int32_t n_blocks, block_size, n_kv_heads;
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *ctx_lens;
    float scale_log2;
    int32_t window, sinks;
    __nv_bfloat16 *out;
    float *lse_out;
    int32_t *dev_status;
    int32_t splits;                    // CTAs per cluster
    // a step: the new token's rows (k_new null: attention alone)
    const __nv_bfloat16 *k_new, *v_new;
    int64_t k_stride, v_stride;
    const int32_t *start_pos;
    RopeArgs rope;
};

template <int D, bool INT8>
struct Shape {
    static constexpr int kRow = INT8 ? D : 2 * D;                 // bytes of a head row in the pool
    static constexpr int kVecs = kRow / 16;
    static constexpr int kStage = 2 * kTile * kRow + (INT8 ? 2 * kTile * 4 : 0);
    static constexpr int kStages = 3;
    static constexpr int kAcc = D + 4;                            // floats per accumulator row
    static constexpr int kRing = kStages * kStage > kHeads * kAcc * 4 ? kStages * kStage : kHeads * kAcc * 4;
    static constexpr size_t kSmem = 256 + (size_t)kWarps * kRing + (size_t)kHeads * kAcc * 4 + 2 * kRow;
    static_assert(kRing % kRow == 0 && kStage % kRow == 0, "rows aligned to their size");
    // a row's 16-byte chunks are permuted so that chunk c of 8 consecutive rows
    // lies in 8 different bank groups
    static __device__ __forceinline__ int swizzle(int row) { return kRow >= 128 ? row & 7 : (row >> 1) & 3; }
    static __device__ __forceinline__ uint32_t at(int row, int chunk) { return row * kRow + ((chunk ^ swizzle(row)) << 4); }
};

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float of the CTA `rank` of the cluster, at the same place as local address a
__device__ __forceinline__ float ld_cluster(const float *a, uint32_t rank)
{
    uint32_t r;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(a)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
    return v;
}

// Two bytes of x (codes + 128) as the fp16 values code + 1152, and as the codes.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t biased_f16x2(uint32_t x)
{
    return __byte_perm(x, 0x64646464u, SEL);
}
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t x)
{
    const uint32_t w = biased_f16x2<SEL>(x);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(1152.f));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// a, b rounded to a pair of 16-bit values, and the pair of what the rounding left
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b)
{
    return F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}
template <bool F16>
__device__ __forceinline__ float2 unpack16(uint32_t w)
{
    if (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16_rest(float a, float b, uint32_t packed)
{
    const float2 r = unpack16<F16>(packed);
    return pack16<F16>(a - r.x, b - r.y);
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F16)
        mma_f16_16816(d, a, b0, b1);
    else
        mma_bf16_16816(d, a, b0, b1);
}

// WIDE: 5 to 8 query heads per kv head (bf16; int8 pages have one form for all).
template <int D, bool INT8, bool WIDE>
__global__ void __launch_bounds__(kThreads) decode_window_kernel(const WindowArgs a)
{
    using S = Shape<D, INT8>;
    constexpr int SLOTS = D / 16;                   // lanes per head row in the prologue
    constexpr int KS = D / 16;                      // 16-element steps over head_dim
    constexpr bool PAIRED = !INT8 && !WIDE;         // remainders in columns 4-7
    constexpr bool REST2 = !INT8 && WIDE;           // remainders in a second product
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 255) & ~uintptr_t(255));
    float *qf = reinterpret_cast<float *>(ring + (size_t)kWarps * S::kRing);          // [8][kAcc] queries
    uint8_t *new_rows = reinterpret_cast<uint8_t *>(qf + kHeads * S::kAcc);           // the step's K and V row
    __shared__ uint32_t present_s[kWarps][S::kStages];                                // tokens of the stage that are there
    __shared__ float new_scale[2], q_mul[kHeads];
    __shared__ float w_m[kWarps][kHeads], w_m2[kWarps][kHeads], w_l[kWarps][kHeads], w_f[kWarps][kHeads];
    __shared__ float c_m[kHeads], c_m2[kHeads], c_l[kHeads];                          // of the CTA

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;        // mma fragment row group / column pair
    const int mi = lane >> 3, ri = lane & 7;        // ldmatrix matrix / row within it
    const int hkv = a.n_kv_heads, G = a.group, bs = a.block_size;
    const int rank = (int)(blockIdx.x % a.splits), unit = (int)(blockIdx.x / a.splits);
    const int s = unit / hkv, h = unit % hkv;
    const bool step = a.k_new != nullptr;
    const int32_t *trow = a.tables + (int64_t)s * a.max_blocks;

    grid_dependents_launch();   // a programmatic dependent: nothing is read before the wait
    grid_dependency_wait();

    // 1. the visible tokens
    int32_t L = __ldg(a.ctx_lens + s);
    const int32_t t_new = step ? __ldg(a.start_pos + s) : -1;
    if (L < 0 || (int64_t)L > (int64_t)a.max_blocks * bs) {
        if (tid == 0 && h == 0 && rank == 0) report(a.dev_status, PKV_DEV_BAD_LENGTH);
        L = 0;
    }
    const int32_t first = min(a.sinks, L);          // seen as first tokens
    const int32_t low = max(first, L - a.window);   // and from here on
    const int32_t n_vis = first + (L - low);
    const int n_tiles = (n_vis + kTile - 1) / kTile;
    const int n_workers = kWarps * a.splits, worker = rank * kWarps + warp;

    // 2. the warp's pipeline
    uint8_t *my_ring = ring + (size_t)warp * S::kRing;
    auto token_of = [&](int tile) -> int32_t {      // of this lane (lanes 16-31 repeat 0-15); -1: none
        const int32_t c = tile * kTile + (lane & 15);
        return c >= n_vis ? -1 : c < first ? c : low + (c - first);
    };
    auto load_id = [&](int tile) -> int32_t {
        const int32_t t = token_of(tile);
        return t >= 0 ? __ldg(trow + (uint32_t)t / (uint32_t)bs) : 0;
    };
    int32_t id = worker < n_tiles ? load_id(worker) : 0;
    // copies of one tile into a stage; id is its lanes' block, and the next tile's after
    auto issue = [&](int tile, int st) {
        if (tile < n_tiles) {
            const int32_t t = token_of(tile);
            int32_t row = -1;
            if (t >= 0) {
                if (id < 0 || id > a.n_blocks)
                    report(a.dev_status, PKV_DEV_BAD_BLOCK_ID);
                else
                    row = id * bs + (int32_t)((uint32_t)t % (uint32_t)bs);
            }
            // bits 0-15: there; 16-31: the step's new token, which comes from new_rows
            const uint32_t there = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
            const uint32_t fresh = __ballot_sync(0xffffffffu, step && row >= 0 && t == t_new) & 0xffffu;
            if (lane == 0) present_s[warp][st] = there | (fresh << 16);
            id = load_id(tile + n_workers);
            const uint32_t kdst = smem_u32(my_ring + st * S::kStage), vdst = kdst + kTile * S::kRow;
#pragma unroll
            for (int i = 0; i < kTile * S::kVecs / 32; ++i) {
                const int r = (i * 32 + lane) / S::kVecs, v = (i * 32 + lane) % S::kVecs;
                const int32_t rr = __shfl_sync(0xffffffffu, row, r);
                const int64_t src = ((int64_t)max(rr, 0) * hkv + h) * S::kRow + v * 16;
                cp_async16_or_zero(kdst + S::at(r, v), static_cast<const uint8_t *>(a.k_pool) + src, rr >= 0);
                cp_async16_or_zero(vdst + S::at(r, v), static_cast<const uint8_t *>(a.v_pool) + src, rr >= 0);
            }
            if constexpr (INT8) {
                const float *sc = (lane < 16 ? a.k_scales : a.v_scales) + (int64_t)max(row, 0) * hkv + h;
                cp_async4_or_zero(kdst + 2 * kTile * S::kRow + lane * 4, sc, row >= 0);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S::kStages - 1; ++k) issue(worker + k * n_workers, k);

    // 3. the queries in binary32 (turned in a step), and a step's new rows: a head
    //    row is the work of SLOTS lanes (rope.cuh)
    const int64_t new_row = step ? pool_row_of(trow, a.max_blocks, a.n_blocks, bs, t_new,
                                               tid == 0 && h == 0 && rank == 0 ? a.dev_status : nullptr)
                                 : -1;
    {
        const int slot = tid % SLOTS;
        for (int r0 = 0; r0 < kHeads + 2; r0 += kThreads / SLOTS) {
            const int r = r0 + tid / SLOTS;          // 0 .. 7 queries, 8 the K row, 9 the V row
            int v0, v1;
            const bool turn = rope_vectors(a.rope, slot, v0, v1) && r <= kHeads;
            const __nv_bfloat16 *src = nullptr;
            if (r < kHeads) {
                if (r < G) src = a.q + s * a.q_stride + ((int64_t)h * G + r) * D;
            } else if (step && r < kHeads + 2) {
                src = r == kHeads ? a.k_new + s * a.k_stride + (int64_t)h * D : a.v_new + s * a.v_stride + (int64_t)h * D;
            }
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            if (src) {
                x0 = __ldg(reinterpret_cast<const uint4 *>(src) + v0);
                x1 = __ldg(reinterpret_cast<const uint4 *>(src) + v1);
            }
            float x[16];
            unpack_bf16x8(x0, x);
            unpack_bf16x8(x1, x + 8);
            if (turn && src) {
                float c[8], sn[8];
                rope_angles(a.rope, slot, t_new, c, sn);
                rope_turn(a.rope.interleaved, c, sn, x);
                x0 = pack_bf16x8(x);
                x1 = pack_bf16x8(x + 8);
            }
            float amax = 0.f;
            if constexpr (INT8) {
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
                for (int off = 1; off < SLOTS; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            }
            int code[16];
            float scale = 0.f;
            if constexpr (INT8) scale = int8_codes<16>(x, amax, code);
            if (r < kHeads) {
                if constexpr (INT8) {
                    // fp16 holds the query as multiples of the power of two below its largest element
                    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 0xff) - 127, -126), 126);
                    const float down = amax > 0.f ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.f;
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] *= down;
                    if (slot == 0) q_mul[r] = a.scale_log2 * (amax > 0.f ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.f);
                }
                float *dst = qf + r * S::kAcc;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    *reinterpret_cast<float4 *>(dst + 8 * v0 + 4 * k) = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                    *reinterpret_cast<float4 *>(dst + 8 * v1 + 4 * k) =
                        make_float4(x[8 + 4 * k], x[9 + 4 * k], x[10 + 4 * k], x[11 + 4 * k]);
                }
            } else if (src) {
                const int which = r - kHeads;
                uint8_t *dst = new_rows + which * S::kRow;
                uint8_t *pool = static_cast<uint8_t *>(which ? a.v_pool : a.k_pool) + (new_row * hkv + h) * S::kRow;
                const bool write = rank == 0 && new_row >= 0;
                if constexpr (INT8) {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e / 4] |= (uint32_t)(code[e] & 0xff) << (8 * (e % 4));
                    const uint2 y0 = make_uint2(w[0], w[1]), y1 = make_uint2(w[2], w[3]);
                    *reinterpret_cast<uint2 *>(dst + 8 * v0) = y0;
                    *reinterpret_cast<uint2 *>(dst + 8 * v1) = y1;
                    if (slot == 0) new_scale[which] = scale;
                    if (write) {
                        *reinterpret_cast<uint2 *>(pool + 8 * v0) = y0;
                        *reinterpret_cast<uint2 *>(pool + 8 * v1) = y1;
                        if (slot == 0) (which ? a.v_scales : a.k_scales)[new_row * hkv + h] = scale;
                    }
                } else {
                    *reinterpret_cast<uint4 *>(dst + 16 * v0) = x0;
                    *reinterpret_cast<uint4 *>(dst + 16 * v1) = x1;
                    if (write) {
                        *reinterpret_cast<uint4 *>(pool + 16 * v0) = x0;
                        *reinterpret_cast<uint4 *>(pool + 16 * v1) = x1;
                    }
                }
            }
        }
    }
    __syncthreads();

    // 4. the queries as B fragments.  bf16: column g4 is head g4 (WIDE), or head
    //    g4 % 4 with its remainders in columns 4-7.  int8: column g4 is head g4, the
    //    four bytes 4 q4 .. of a 16-byte chunk are the products' k = 2 q4, 2 q4 + 1,
    //    2 q4 + 8, 2 q4 + 9, and bias is 1152 times the sum of the rounded query.
    uint32_t qb[KS][2], qr[REST2 ? KS : 1][2];
    bool rest = false;                               // REST2: some query has a remainder
    float bias = 0.f;
    {
        const float *src = qf + (PAIRED ? (g4 & 3) : g4) * S::kAcc;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int d = 16 * kk + (INT8 ? 4 * q4 + 2 * j : 2 * q4 + 8 * j);
                const float2 x = *reinterpret_cast<const float2 *>(src + d);
                const uint32_t hi = pack16<INT8>(x.x, x.y);
                if constexpr (INT8) {
                    const float2 y = unpack16<true>(hi);
                    bias += y.x + y.y;
                    qb[kk][j] = hi;
                } else {
                    const uint32_t lo = pack16_rest<false>(x.x, x.y, hi);
                    qb[kk][j] = PAIRED && g4 >= 4 ? lo : hi;
                    if constexpr (REST2) {
                        qr[kk][j] = lo;
                        rest |= (lo & 0x7fff7fffu) != 0;
                    }
                }
            }
        }
        if constexpr (REST2) rest = __any_sync(0xffffffffu, rest);
    }
    // this lane's two heads (columns 2 q4, 2 q4 + 1 of the products)
    const int h0 = PAIRED ? (2 * q4) & 3 : 2 * q4;
    const float mul0 = INT8 ? q_mul[h0] : a.scale_log2, mul1 = INT8 ? q_mul[h0 + 1] : a.scale_log2;
    float bias0 = 0.f, bias1 = 0.f;
    if constexpr (INT8) {
        bias += __shfl_xor_sync(0xffffffffu, bias, 1);
        bias += __shfl_xor_sync(0xffffffffu, bias, 2);         // of head g4, in its four lanes
        bias0 = -1152.f * __shfl_sync(0xffffffffu, bias, 4 * h0);
        bias1 = -1152.f * __shfl_sync(0xffffffffu, bias, 4 * h0 + 4);
    }

    // 5. the tiles
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, m2[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int st = 0;
    for (int tile = worker; tile < n_tiles; tile += n_workers) {
        cp_async_wait<S::kStages - 2>();
        __syncwarp();                                // the tile is there, the stage before it is free
        issue(tile + (S::kStages - 1) * n_workers, st == 0 ? S::kStages - 1 : st - 1);
        uint8_t *kt = my_ring + st * S::kStage, *vt = kt + kTile * S::kRow;
        const float *sc = reinterpret_cast<const float *>(vt + kTile * S::kRow);     // int8: K, V scales
        const uint32_t present = present_s[warp][st];
        if (present >> 16) {                         // the step's new token
            const int i = __ffs(present >> 16) - 1;
            for (int v = lane; v < 2 * S::kVecs; v += 32) {
                uint8_t *dst = v < S::kVecs ? kt : vt;
                *reinterpret_cast<uint4 *>(dst + S::at(i, v % S::kVecs)) =
                    *reinterpret_cast<const uint4 *>(new_rows + v * 16);
            }
            if (INT8 && lane < 2) const_cast<float *>(sc)[lane * kTile + i] = new_scale[lane];
            __syncwarp();
        }

        // S^T = K Q^T
        float c[4] = {bias0, bias1, bias0, bias1}, ca[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t kaddr = smem_u32(kt) + S::at(ri + 8 * (mi & 1), mi >> 1);
        if constexpr (INT8) {
#pragma unroll
            for (int k2 = 0; k2 < KS / 2; ++k2) {
                uint32_t raw[4];
                ldmatrix_x4(raw, kaddr ^ (32u * k2));
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[i] ^= 0x80808080u;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t af[4] = {biased_f16x2<0x4140>(raw[2 * j]), biased_f16x2<0x4140>(raw[2 * j + 1]),
                                            biased_f16x2<0x4342>(raw[2 * j]), biased_f16x2<0x4342>(raw[2 * j + 1])};
                    mma16<true>(j ? ca : c, af, qb[2 * k2 + j][0], qb[2 * k2 + j][1]);
                }
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                uint32_t af[4];
                ldmatrix_x4(af, kaddr ^ (32u * kk));
                mma16<false>(kk & 1 ? ca : c, af, qb[kk][0], qb[kk][1]);
                if constexpr (REST2)
                    if (rest) mma16<false>(kk & 1 ? ca : c, af, qr[kk][0], qr[kk][1]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] += ca[e];
        if constexpr (PAIRED) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] += __shfl_xor_sync(0xffffffffu, c[e], 2);
        }

        // scores in log2 units: c[0], c[1] of token g4, c[2], c[3] of token g4 + 8
        const bool t0 = (present >> g4) & 1, t1 = (present >> (g4 + 8)) & 1;
        const float k0 = INT8 ? sc[g4] : 1.f, k1 = INT8 ? sc[g4 + 8] : 1.f;
        c[0] = t0 ? c[0] * (k0 * mul0) : -INFINITY;
        c[1] = t0 ? c[1] * (k0 * mul1) : -INFINITY;
        c[2] = t1 ? c[2] * (k1 * mul0) : -INFINITY;
        c[3] = t1 ? c[3] * (k1 * mul1) : -INFINITY;
        float w[4];                                  // int8: scores with the V scale
        float sv0 = 0.f, sv1 = 0.f;
        if constexpr (INT8) {
            sv0 = sc[kTile + g4];
            sv1 = sc[kTile + g4 + 8];
            const float lv0 = __log2f(fabsf(sv0)), lv1 = __log2f(fabsf(sv1));
            w[0] = c[0] + lv0;
            w[1] = c[1] + lv0;
            w[2] = c[2] + lv1;
            w[3] = c[3] + lv1;
            if (!t0) w[0] = w[1] = -INFINITY;
            if (!t1) w[2] = w[3] = -INFINITY;
        }
        // the maxima move (and what was summed is rescaled) only when a score
        // passes one by more than kLazyMax: no reduction in the common case
        float mx[2] = {fmaxf(c[0], c[2]), fmaxf(c[1], c[3])}, mx2[2] = {-INFINITY, -INFINITY};
        bool grow = mx[0] > m[0] + kLazyMax || mx[1] > m[1] + kLazyMax;
        if constexpr (INT8) {
            mx2[0] = fmaxf(w[0], w[2]);
            mx2[1] = fmaxf(w[1], w[3]);
            grow |= mx2[0] > m2[0] + kLazyMax || mx2[1] > m2[1] + kLazyMax;
        }
        if (__any_sync(0xffffffffu, grow)) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], off));
                const bool up = mx[k] > m[k] + kLazyMax;
                f[k] = up ? fast_exp2(m[k] - mx[k]) : 1.f;
                if (up) m[k] = mx[k];
                l[k] *= f[k];
                if constexpr (INT8) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx2[k] = fmaxf(mx2[k], __shfl_xor_sync(0xffffffffu, mx2[k], off));
                    const bool up2 = mx2[k] > m2[k] + kLazyMax;
                    f[k] = up2 ? fast_exp2(m2[k] - mx2[k]) : 1.f;
                    if (up2) m2[k] = mx2[k];
                }
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= f[e & 1];
        }
        // probabilities (0 where absent), their sum, and the weights of V
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = fast_exp2(c[e] - (e & 1 ? b1 : b0));
        l[0] += c[0] + c[2];
        l[1] += c[1] + c[3];
        if constexpr (INT8) {
            const float d0 = m2[0] == -INFINITY ? 0.f : m2[0], d1 = m2[1] == -INFINITY ? 0.f : m2[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = copysignf(fast_exp2(w[e] - (e & 1 ? d1 : d0)), e < 2 ? sv0 : sv1);
        }
        uint32_t pa = pack16<INT8>(c[0], c[1]), pb = pack16<INT8>(c[2], c[3]);
        uint32_t ra_t = 0, rb_t = 0;
        if constexpr (!INT8) {
            const uint32_t ra = pack16_rest<false>(c[0], c[1], pa), rb = pack16_rest<false>(c[2], c[3], pb);
            if constexpr (REST2) {
                ra_t = movmatrix_trans(ra);
                rb_t = movmatrix_trans(rb);
            } else if (q4 >= 2) {                    // columns 4-7: the remainders of heads 0-3
                pa = ra;
                pb = rb;
            }
        }
        const uint32_t pa_t = movmatrix_trans(pa), pb_t = movmatrix_trans(pb);

        // O^T += V^T P^T
        if constexpr (INT8) {
            const uint32_t vaddr = smem_u32(vt) + S::at(ri + 8 * (mi & 1), mi >> 1);
#pragma unroll
            for (int k2 = 0; k2 < KS / 2; ++k2) {
                uint32_t raw[4];
                ldmatrix_x4_trans(raw, vaddr ^ (32u * k2));
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[i] ^= 0x80808080u;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // rows 0-7: elements 2 g4 of the chunk, rows 8-15: 2 g4 + 1
                    const uint32_t af[4] = {codes_f16x2<0x4240>(raw[2 * j]), codes_f16x2<0x4341>(raw[2 * j]),
                                            codes_f16x2<0x4240>(raw[2 * j + 1]), codes_f16x2<0x4341>(raw[2 * j + 1])};
                    mma16<true>(o[2 * k2 + j], af, pa_t, pb_t);
                }
            }
        } else {
            const uint32_t vaddr = smem_u32(vt) + S::at(ri + 8 * (mi >> 1), mi & 1);
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                uint32_t af[4];
                ldmatrix_x4_trans(af, vaddr ^ (32u * i));
                mma16<false>(o[i], af, pa_t, pb_t);
                if constexpr (REST2) mma16<false>(o[i], af, ra_t, rb_t);
            }
        }
        st = st + 1 == S::kStages ? 0 : st + 1;
    }

    // 6. the warp's partial: sums over its tokens, remainders added to their heads
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
    float *acc = reinterpret_cast<float *>(my_ring);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (PAIRED) o[i][e] += __shfl_xor_sync(0xffffffffu, o[i][e], 2);
            const int d = 16 * i + (INT8 ? 2 * g4 + (e >> 1) : g4 + 8 * (e >> 1));
            if (!PAIRED || q4 < 2) acc[(h0 + (e & 1)) * S::kAcc + d] = o[i][e];
        }
    }
    if (g4 == 0 && (!PAIRED || q4 < 2)) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w_m[warp][h0 + k] = m[k];
            w_m2[warp][h0 + k] = INT8 ? m2[k] : m[k];
            w_l[warp][h0 + k] = l[k];
        }
    }
    __syncthreads();

    // 7. the CTA's partial
    if (tid < G) {
        float M = -INFINITY, M2 = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            M = fmaxf(M, w_m[k][tid]);
            M2 = fmaxf(M2, w_m2[k][tid]);
        }
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (w_m[k][tid] != -INFINITY) sum += fast_exp2(w_m[k][tid] - M) * w_l[k][tid];
            else sum += w_l[k][tid];                 // 0, or the NaN of a score
            w_f[k][tid] = w_m2[k][tid] == -INFINITY ? 1.f : fast_exp2(w_m2[k][tid] - M2);
        }
        c_m[tid] = M;
        c_m2[tid] = M2;
        c_l[tid] = sum;
    }
    __syncthreads();
    for (int i = tid; i < G * D; i += kThreads) {
        const int g = i / D, d = i % D;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            v += w_f[k][g] * reinterpret_cast<const float *>(ring + (size_t)k * S::kRing)[g * S::kAcc + d];
        qf[g * S::kAcc + d] = v;
    }

    // 8. joined over the cluster; each CTA writes its share of the outputs
    __nv_bfloat16 *out = a.out + ((int64_t)s * a.n_q_heads + (int64_t)h * G) * D;
    if (a.splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    for (int i = rank * kThreads + tid; i < G * D / 2; i += a.splits * kThreads) {
        const int g = i / (D / 2), d = (i % (D / 2)) * 2;
        float M = -INFINITY, M2 = -INFINITY, sum = 0.f, v0 = 0.f, v1 = 0.f;
        float rm[kMaxSplits], rm2[kMaxSplits], rl[kMaxSplits], ra[kMaxSplits], rb[kMaxSplits];
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) {
            rm[r] = rm2[r] = -INFINITY;
            rl[r] = ra[r] = rb[r] = 0.f;
            if (r >= a.splits) continue;
            rm[r] = a.splits > 1 ? ld_cluster(&c_m[g], r) : c_m[g];
            rm2[r] = a.splits > 1 ? ld_cluster(&c_m2[g], r) : c_m2[g];
            rl[r] = a.splits > 1 ? ld_cluster(&c_l[g], r) : c_l[g];
            ra[r] = a.splits > 1 ? ld_cluster(&qf[g * S::kAcc + d], r) : qf[g * S::kAcc + d];
            rb[r] = a.splits > 1 ? ld_cluster(&qf[g * S::kAcc + d + 1], r) : qf[g * S::kAcc + d + 1];
            M = fmaxf(M, rm[r]);
            M2 = fmaxf(M2, rm2[r]);
        }
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) {
            sum += rm[r] == -INFINITY ? rl[r] : fast_exp2(rm[r] - M) * rl[r];
            const float f = rm2[r] == -INFINITY ? 1.f : fast_exp2(rm2[r] - M2);
            v0 += f * ra[r];
            v1 += f * rb[r];
        }
        // o = 2^M2 v / (2^M sum); no token seen: 0
        const float inv = sum == 0.f ? 0.f : (M2 == -INFINITY ? 1.f : INT8 ? fast_exp2(M2 - M) : 1.f) / sum;
        *reinterpret_cast<uint32_t *>(out + g * D + d) = pack_bf16x2(v0 * inv, v1 * inv);
        if (a.lse_out && d == 0)
            a.lse_out[(int64_t)s * a.n_q_heads + (int64_t)h * G + g] =
                sum == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) * 0.69314718055994531f + logf(sum);
    }
    if (a.splits > 1) cluster_sync_all();            // no CTA leaves while another reads it
}

template <int D, bool INT8, bool WIDE>
cudaError_t launch_as(const WindowArgs &a, int64_t units, cudaStream_t stream)
{
    const void *kern = reinterpret_cast<const void *>(decode_window_kernel<D, INT8, WIDE>);
    const cudaError_t e = prepare_kernel(kern, kThreads, Shape<D, INT8>::kSmem, nullptr);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.splits;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(units * a.splits));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = Shape<D, INT8>::kSmem;
    lc.stream = stream;
    lc.attrs = at;
    lc.numAttrs = a.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, decode_window_kernel<D, INT8, WIDE>, a);
}

// CTAs per (sequence, kv head): enough for kCtasPerSm CTAs per SM, as long as every
// warp keeps two tiles or more of the longest window.
int choose_splits(int64_t units, int64_t tiles, int sms)
{
    int c = 1;
    while (c < kMaxSplits && units * c < kCtasPerSm * sms && tiles >= (int64_t)c * 2 * 2 * kWarps) c *= 2;
    return c;
}

cudaError_t launch_window(WindowArgs &a, int32_t head_dim, bool int8, int32_t n_seqs, int sms, cudaStream_t stream)
{
    const int64_t units = (int64_t)n_seqs * a.n_kv_heads;
    int64_t seen = (int64_t)a.max_blocks * a.block_size;
    if ((int64_t)a.window + a.sinks < seen) seen = (int64_t)a.window + a.sinks;
    a.splits = choose_splits(units, (seen + kTile - 1) / kTile, sms);
    const bool wide = a.group > 4;
    if (head_dim == 128) {
        if (int8) return launch_as<128, true, true>(a, units, stream);
        return wide ? launch_as<128, false, true>(a, units, stream) : launch_as<128, false, false>(a, units, stream);
    }
    if (int8) return launch_as<64, true, true>(a, units, stream);
    return wide ? launch_as<64, false, true>(a, units, stream) : launch_as<64, false, false>(a, units, stream);
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
    if ((int64_t)max_blocks * dims.block_size > 0x7fffffffLL) return PKV_ERR_OUT_OF_RANGE;
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
    if (rope) a.rope = RopeArgs{rope->phases, rope->rot_dim, rope->interleaved != 0, rope->magnitude};
    int sms = 0;
    st = num_sms_of_current_device(&sms);
    if (st != PKV_OK) return st;
    return cuda_status(launch_window(a, dims.head_dim, kv_dtype == PKV_KV_INT8, n_seqs, sms, (cudaStream_t)stream));
}

}  // extern "C"
