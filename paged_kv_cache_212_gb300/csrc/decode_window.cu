// decode_window.cu -- decode attention under a sliding window with first tokens
// that stay visible (pagedkv_window.h), over bf16 or int8 pages, alone or as one
// layer's step with the rotary turn and the page write of the new token.
//
// The host knows how many tokens a query can see (window + sinks), so no plan
// and no workspace is needed: a (sequence, kv head) unit is the work of one
// thread-block cluster of 1 .. 16 CTAs, whose partials are joined through the
// cluster's shared memory, all in one launch.
//
// A tile is 16 tokens from a multiple of 16 on, so it lies in one block; tokens of
// it that the query does not see are not read.  Warp w of the cluster takes the
// unit's tiles w, w + n_warps, ...  A warp works alone: it looks its tiles' blocks up
// one tile ahead, copies their K and V rows (16 bytes a lane, asynchronously) into a
// ring of its own, and contracts them with the G query heads of its kv head on the
// tensor cores (mma.sync m16n8k16):
//   S^T = K Q^T     16 tokens as M, query heads as N = 8
//   O^T += V^T P^T  head_dim as M, query heads as N, tokens as K
// with a running maximum and sum in log2 units.  Warps and CTAs meet once, at the
// end, where they are joined by their maxima in a fixed order.
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
// 1152 times the query's sum).  The K scale multiplies the score; the V scale joins
// the probability, and the weight is multiplied by a running power of two r that
// keeps the largest one in fp16's range whatever the scales are.  Weights are split
// into an fp16 value and its fp16 remainder in a second product (2^-22 together;
// 64 sequences, 64 query heads: 30.4 -> 31.4 us).  Queries are multiples of a power of
// two and rounded once to fp16: a bf16 query is exact there but for elements below
// 2^-17 of its largest one, which are held to 2^-25 of that; a step's turned query
// keeps 11 bits, where a turn written to memory between the two calls keeps 8 (its
// remainders in a second product: a step of 64 sequences 32.0 -> 34.5 us or more).
//
// Measured (one launch among others; 8 kv heads of 128, window 1024, 4 first tokens).
// 64 sequences, bf16 pages, 32 query heads: 41.4 us = 6.28 TB/s, 92 % of the copy rate;
// memory bounds it.  The same over int8 pages with 64 query heads: 31.4 us, 4.3 TB/s;
// half of the issue slots are taken and the rest is the latency of an SM's 16 warps.
// Two sequences of 16 K visible tokens, 64 query heads: 26.5 us, 5.1 TB/s.  Four
// sequences of 68 visible tokens (2 kv heads of 64): 2.7 us, a launch and three
// dependent reads.
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "rope.cuh"
#include "window.h"
#include "write_rows.cuh"
#include "../../include/pagedkv_window.h"

namespace pkv {
namespace {

constexpr int kTile = 16;              // tokens per tile
constexpr int kHeads = 8;              // query heads per kv head, padded
constexpr int kMaxSplits = 16;         // CTAs per cluster
constexpr float kMostLr = 120.f;       // int8: log2 of the largest factor on the weights
constexpr float kLazyMax = 8.0f;       // the running maximum may lag by this (log2 units); int8, 64 sequences: 33.3 -> 31.4 us

struct WindowArgs {
    const __nv_bfloat16 *q;
    int64_t q_stride;
    int32_t n_q_heads, group;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales;
    int32_t n_blocks, block_size, n_kv_heads;
    uint32_t tiles_per_block, block_magic;   // tile / tiles_per_block = the product's upper half, above one tile
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
    // 64 sequences, bf16 pages: 44.5 us with 2, 40.9 with 3, 52.2 with 4 (fewer CTAs are resident)
    static constexpr int kStages = 3;
    static constexpr int kAcc = D + 4;                            // floats per staged row
    static constexpr int kQRow = 2 * D + 16;                      // bytes of a staged query row of 16-bit elements
    static constexpr int kQueries = (INT8 ? 1 : 2) * kHeads * kQRow;   // the queries and (bf16) their remainders
    static constexpr bool kShared = INT8;                         // staged once for all warps of a CTA
    static_assert(kShared || kStage >= kQueries, "a free stage holds them");
    static constexpr size_t smem(int warps) { return 256 + (size_t)warps * kStages * kStage + (kShared ? 1 : warps) * 2 * kRow + (kShared ? kQueries : 0); }
    static_assert(kStage % kRow == 0, "rows aligned to their size");
    static_assert(kStage >= kHeads * kAcc * 4, "a free stage holds 8 rows of binary32");
    // a row's 16-byte chunks are permuted so that chunk c of 8 consecutive rows
    // lies in 8 different bank groups
    static __device__ __forceinline__ int swizzle(int row) { return kRow >= 128 ? row & 7 : (row >> 1) & 3; }
    static __device__ __forceinline__ uint32_t at(int row, int chunk) { return row * kRow + ((chunk ^ swizzle(row)) << 4); }
};

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// four floats of the CTA `rank` of the cluster, at the same place as local address a
__device__ __forceinline__ float4 ld_cluster(const float4 *a, uint32_t rank)
{
    uint32_t r;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(a)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(r)
                 : "memory");
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

// The tiles that hold the tokens seen by the query of a sequence of length L:
// tiles 0 .. n_first - 1, then those from tile w_tile on.
struct Seen {
    int32_t L, first, low, n_first, w_tile, tiles;
    __device__ __forceinline__ Seen(const WindowArgs &a, int32_t len)
    {
        L = len < 0 || (int64_t)len > (int64_t)a.max_blocks * a.block_size ? 0 : len;
        first = min(a.sinks, L);                // tokens below are seen
        low = max(first, L - a.window);         // and tokens from here on
        n_first = (first + kTile - 1) / kTile;
        w_tile = max(low / kTile, n_first);
        tiles = n_first + max(0, (L + kTile - 1) / kTile - w_tile);
    }
    // the place of tile i in the sequence, in tiles, and which of its 16 tokens are seen
    __device__ __forceinline__ int32_t place(int32_t i) const { return i < n_first ? i : w_tile + i - n_first; }
    __device__ __forceinline__ uint32_t mask(int32_t t) const
    {
        if (t >= low && L - t >= kTile) return 0xffffu;
        const uint32_t below_L = L - t >= kTile ? 0xffffu : (1u << max(L - t, 0)) - 1u;
        const uint32_t below_first = first - t >= kTile ? 0xffffu : (1u << max(first - t, 0)) - 1u;
        const uint32_t from_low = low <= t ? 0xffffu : low - t >= kTile ? 0u : 0xffffu << (low - t);
        return below_L & (below_first | from_low) & 0xffffu;
    }
};

// WIDE: 5 to 8 query heads per kv head (bf16; int8 pages have one form for all).
template <int D, bool INT8, bool WIDE, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, INT8 && WARPS == 4 ? 4 : 1) decode_window_kernel(const WindowArgs a)
{
    using S = Shape<D, INT8>;
    constexpr int SLOTS = D / 16;                   // lanes that hold a head row (rope.cuh)
    constexpr int KS = D / 16;                      // 16-element steps over head_dim
    constexpr bool PAIRED = !INT8 && !WIDE;         // remainders in columns 4-7
    constexpr bool REST2 = !INT8 && WIDE;           // the queries' remainders in a second product
    constexpr int QROWS = PAIRED ? 4 : 8;           // query rows that the products read
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 255) & ~uintptr_t(255));
    __shared__ uint32_t present_s[WARPS][S::kStages];                                 // tokens of the stage that are there
    __shared__ float new_scale[2], q_mul[kHeads], q_sum[kHeads];
    __shared__ float w_m[WARPS][kHeads], w_m2[WARPS][kHeads], w_l[WARPS][kHeads];
    __shared__ float4 c_stat[kHeads];               // of the CTA: maximum, maximum of the weights, sum

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;        // mma fragment row group / column pair
    const int mi = lane >> 3, ri = lane & 7;        // ldmatrix matrix / row within it
    const int hkv = a.n_kv_heads, G = a.group, bs = a.block_size;
    const int rank = (int)(blockIdx.x % a.splits), unit = (int)(blockIdx.x / a.splits);
    const int s = unit / hkv, h = unit % hkv;
    const bool step = a.k_new != nullptr;
    const int32_t *trow = a.tables + (int64_t)s * a.max_blocks;
    uint8_t *my_ring = ring + (size_t)warp * S::kStages * S::kStage;
    uint8_t *new_rows = ring + (size_t)WARPS * S::kStages * S::kStage + (S::kShared ? 0 : warp) * 2 * S::kRow;   // a step's K and V row

    grid_dependents_launch();   // a programmatic dependent: nothing is read before the wait
    grid_dependency_wait();

    // 1. the tiles
    const int32_t len = __ldg(a.ctx_lens + s);
    const int32_t t_new = step ? __ldg(a.start_pos + s) : -1;
    const Seen seen(a, len);
    if (tid == 0 && h == 0 && rank == 0 && len != seen.L) report(a.dev_status, PKV_DEV_BAD_LENGTH);
    const int n_workers = WARPS * a.splits, worker = rank * WARPS + warp;

    // 2. the warp's copies, which run ahead of its products by kStages - 1 tiles
    int32_t a_tile = worker, a_token = 0, a_off = 0, id = 0;
    auto look_up = [&]() {                          // the block of the next tile to copy
        if (a_tile >= seen.tiles) return;
        const uint32_t at = (uint32_t)seen.place(a_tile);
        const uint32_t blk = a.tiles_per_block == 1 ? at : __umulhi(at, a.block_magic);
        a_token = (int32_t)at * kTile;
        a_off = (int32_t)(at - blk * a.tiles_per_block) * kTile;
        id = __ldg(trow + blk);
    };
    look_up();
    const uint32_t lane_dst = S::at(lane / S::kVecs, lane % S::kVecs);   // of the lane's first vector in a tile
    const int64_t token_bytes = (int64_t)hkv * S::kRow;
    const uint8_t *k_lane = static_cast<const uint8_t *>(a.k_pool) + lane / S::kVecs * token_bytes + (int64_t)h * S::kRow +
                            (lane % S::kVecs) * 16;
    const int64_t k_to_v = static_cast<const uint8_t *>(a.v_pool) - static_cast<const uint8_t *>(a.k_pool);
    constexpr int RPI = 32 / S::kVecs;              // rows that the warp copies at once
    auto issue = [&](int st) {
        if (a_tile < seen.tiles) {
            uint32_t there = seen.mask(a_token);
            if (id < 0 || id > a.n_blocks) {
                if (lane == 0) report(a.dev_status, PKV_DEV_BAD_BLOCK_ID);
                there = 0;
            }
            const int32_t row = there ? id * bs + a_off : 0;
            // bits 0-15: there; 16-31: the step's new token, which comes from new_rows
            const uint32_t fresh = step && (uint32_t)(t_new - a_token) < (uint32_t)kTile ? there & (1u << (t_new - a_token)) : 0u;
            if (lane == 0) present_s[warp][st] = there | (fresh << 16);
            a_tile += n_workers;
            look_up();
            const uint32_t dst = smem_u32(my_ring + st * S::kStage);
            const uint8_t *src = k_lane + row * token_bytes;
            if (there == 0xffffu) {
#pragma unroll
                for (int i = 0; i < kTile / RPI; ++i) {
                    // row i * RPI + lane / kVecs, whose swizzle is that of its two parts
                    const uint32_t off = i * RPI * S::kRow + (lane_dst ^ (S::swizzle(i * RPI) << 4));
                    cp_async16(dst + off, src);
                    cp_async16(dst + kTile * S::kRow + off, src + k_to_v);
                    src += RPI * token_bytes;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kTile / RPI; ++i) {
                    const uint32_t off = i * RPI * S::kRow + (lane_dst ^ (S::swizzle(i * RPI) << 4));
                    const bool in = (there >> (i * RPI + lane / S::kVecs)) & 1;
                    cp_async16_or_zero(dst + off, in ? src : k_lane, in);
                    cp_async16_or_zero(dst + kTile * S::kRow + off, (in ? src : k_lane) + k_to_v, in);
                    src += RPI * token_bytes;
                }
            }
            if constexpr (INT8) {
                const int r = lane & 15;
                const bool in = (there >> r) & 1;
                cp_async4_or_zero(dst + 2 * kTile * S::kRow + lane * 4,
                                  (lane < 16 ? a.k_scales : a.v_scales) + (row + (in ? r : 0)) * (int64_t)hkv + h, in);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S::kStages - 1; ++k) issue(k);

    // 3. the queries (turned in a step) in 16 bits into shared memory, and a step's new
    //    rows: a head row is the work of SLOTS lanes (rope.cuh).  int8: the rounds of rows
    //    are shared out to the warps (64 sequences 31.6 -> 30.4 us, 4 of 256 tokens 6.1 ->
    //    5.5); bf16: each warp has its own, in its free stage (a barrier of all warps made
    //    the smallest call 2.8 -> 2.9 us, two sequences of 16 K tokens 26.4 -> 26.8).
    uint32_t qb[KS][2], qr[REST2 ? KS : 1][2];
    bool rest = false;                           // bf16: some query has a remainder
    const int h0 = PAIRED ? (2 * q4) & 3 : 2 * q4;   // this lane's two heads: columns 2 q4, 2 q4 + 1
    float mul0 = a.scale_log2, mul1 = a.scale_log2, bias0 = 0.f, bias1 = 0.f;
    {
        constexpr int PER = 32 / SLOTS;          // rows at once
        constexpr int NIT = (QROWS + PER - 1) / PER + 1, TEAM = S::kShared ? WARPS : 1, MINE = (NIT + TEAM - 1) / TEAM;
        const int member = S::kShared ? warp : 0;
        // 8 rows, then (bf16) their remainders
        uint8_t *q_s = S::kShared ? new_rows + 2 * S::kRow : my_ring + (S::kStages - 1) * S::kStage;
        const int slot = lane % SLOTS;
        int v0, v1;
        const bool turn = rope_vectors(a.rope, slot, v0, v1);
        // row it * PER + lane / SLOTS of the queries; the last round is K and V
        auto source = [&](int it) -> const __nv_bfloat16 * {
            const int r = it * PER + lane / SLOTS;
            if (it < NIT - 1) return r < G ? a.q + s * a.q_stride + ((int64_t)h * G + r) * D : nullptr;
            if (it > NIT - 1 || !step || lane / SLOTS > 1) return nullptr;
            return lane / SLOTS == 0 ? a.k_new + s * a.k_stride + (int64_t)h * D : a.v_new + s * a.v_stride + (int64_t)h * D;
        };
        uint4 x0[MINE], x1[MINE];
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const __nv_bfloat16 *src = source(member + i * TEAM);
            x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
            if (src) {
                x0[i] = __ldg(reinterpret_cast<const uint4 *>(src) + v0);
                x1[i] = __ldg(reinterpret_cast<const uint4 *>(src) + v1);
            }
        }
        float c[8], sn[8];
        if (turn && member < NIT) rope_angles(a.rope, slot, t_new, c, sn);
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int it = member + i * TEAM;
            if (it > NIT - 1 || (it == NIT - 1 && !step)) break;
            const int r = it * PER + lane / SLOTS;
            float x[16];
            unpack_bf16x8(x0[i], x);
            unpack_bf16x8(x1[i], x + 8);
            if (turn && (it < NIT - 1 || lane / SLOTS == 0)) {
                rope_turn(a.rope.interleaved, c, sn, x);
                x0[i] = pack_bf16x8(x);
                x1[i] = pack_bf16x8(x + 8);
            }
            float amax = 0.f;
            if constexpr (INT8) {
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
                for (int off = 1; off < SLOTS; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            }
            if (it < NIT - 1) {
                uint4 *dst = reinterpret_cast<uint4 *>(q_s + r * S::kQRow);
                uint32_t hi[8], lo[8];
                if constexpr (INT8) {
                    // fp16 holds the query as multiples of the power of two below its largest element;
                    // its products with the codes' bias are taken off by the sum of what was rounded
                    const int e = min(max((int)((__float_as_uint(amax) >> 23) & 0xff) - 127, -126), 126);
                    const float down = amax > 0.f ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.f;
                    float sum = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        hi[k] = pack16<true>(x[2 * k] * down, x[2 * k + 1] * down);
                        const float2 y = unpack16<true>(hi[k]);
                        sum += y.x + y.y;
                    }
#pragma unroll
                    for (int off = 1; off < SLOTS; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    if (slot == 0 && r < QROWS) {
                        q_mul[r] = a.scale_log2 * (amax > 0.f ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.f);
                        q_sum[r] = sum;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        hi[k] = pack16<false>(x[2 * k], x[2 * k + 1]);
                        lo[k] = pack16_rest<false>(x[2 * k], x[2 * k + 1], hi[k]);
                        rest |= (lo[k] & 0x7fff7fffu) != 0;
                    }
                }
                if (r >= QROWS) continue;
                dst[v0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                dst[v1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                if constexpr (!INT8) {
                    uint4 *low = reinterpret_cast<uint4 *>(q_s + (kHeads + r) * S::kQRow);
                    low[v0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    low[v1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                }
            } else {
                // every CTA (bf16: every warp) has the new rows, the first one writes them
                const int64_t new_row = (S::kShared ? rank : worker) == 0 ? pool_row_of(trow, a.max_blocks, a.n_blocks, bs, t_new,
                                                                lane == 0 && h == 0 ? a.dev_status : nullptr)
                                                  : -1;
                const int which = lane / SLOTS;
                uint8_t *dst = new_rows + (which & 1) * S::kRow;
                uint8_t *pool = static_cast<uint8_t *>(which ? a.v_pool : a.k_pool) + (new_row * hkv + h) * S::kRow;
                if constexpr (INT8) {
                    uint32_t w[4];
                    const float scale = int8_codes16(x, amax, w);
                    const uint2 y0 = make_uint2(w[0], w[1]), y1 = make_uint2(w[2], w[3]);
                    if (which > 1) continue;
                    *reinterpret_cast<uint2 *>(dst + 8 * v0) = y0;
                    *reinterpret_cast<uint2 *>(dst + 8 * v1) = y1;
                    if (slot == 0) new_scale[which] = scale;
                    if (new_row >= 0) {
                        *reinterpret_cast<uint2 *>(pool + 8 * v0) = y0;
                        *reinterpret_cast<uint2 *>(pool + 8 * v1) = y1;
                        if (slot == 0) (which ? a.v_scales : a.k_scales)[new_row * hkv + h] = scale;
                    }
                } else {
                    if (which > 1) continue;
                    *reinterpret_cast<uint4 *>(dst + 16 * v0) = x0[i];
                    *reinterpret_cast<uint4 *>(dst + 16 * v1) = x1[i];
                    if (new_row >= 0) {
                        *reinterpret_cast<uint4 *>(pool + 16 * v0) = x0[i];
                        *reinterpret_cast<uint4 *>(pool + 16 * v1) = x1[i];
                    }
                }
            }
        }
        if constexpr (S::kShared) {
            __syncthreads();
        } else {
            rest = __any_sync(0xffffffffu, rest);
            __syncwarp();
        }
        // as B fragments.  bf16: column g4 is head g4 (WIDE), or head g4 % 4 with
        // its remainders in columns 4-7.  int8: column g4 is head g4, the four bytes
        // 4 q4 .. of a 16-byte chunk are the products' k = 2 q4, 2 q4 + 1, 2 q4 + 8,
        // 2 q4 + 9.
        const uint8_t *src = q_s + (PAIRED ? (g4 & 3) + (rest && g4 >= 4 ? kHeads : 0) : g4) * S::kQRow;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if constexpr (INT8) {
                const uint2 x = *reinterpret_cast<const uint2 *>(src + 2 * (16 * kk + 4 * q4));
                qb[kk][0] = x.x;
                qb[kk][1] = x.y;
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = 2 * (16 * kk + 2 * q4 + 8 * j);
                    qb[kk][j] = *reinterpret_cast<const uint32_t *>(src + at);
                    if constexpr (REST2) qr[kk][j] = *reinterpret_cast<const uint32_t *>(src + kHeads * S::kQRow + at);
                }
            }
        }
        if constexpr (INT8) {
            mul0 = q_mul[h0];
            mul1 = q_mul[h0 + 1];
            bias0 = -1152.f * q_sum[h0];
            bias1 = -1152.f * q_sum[h0 + 1];
        }
        __syncwarp();                            // a free stage is read
    }

    // 4. the tiles
    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float lr[2] = {kMostLr, kMostLr}, r[2] = {fast_exp2(kMostLr), fast_exp2(kMostLr)};   // int8: log2 r, r
    int st = 0;                                  // stage of the next tile; the one before it is free
    for (int tile = worker; tile < seen.tiles; tile += n_workers) {
        cp_async_wait<S::kStages - 2>();
        __syncwarp();                                // the tile is there, the stage before it is free
        issue(st == 0 ? S::kStages - 1 : st - 1);
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
        if constexpr (PAIRED) {                      // every column's lane has its head's whole score
            if (rest) {
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] += __shfl_xor_sync(0xffffffffu, c[e], 2);
            }
        }

        // scores in log2 units: c[0], c[1] of token g4, c[2], c[3] of token g4 + 8
        const float k0 = INT8 ? sc[g4] : 1.f, k1 = INT8 ? sc[g4 + 8] : 1.f;
        c[0] *= k0 * mul0;
        c[1] *= k0 * mul1;
        c[2] *= k1 * mul0;
        c[3] *= k1 * mul1;
        if ((present & 0xffffu) != 0xffffu) {
            if (!((present >> g4) & 1)) c[0] = c[1] = -INFINITY;
            if (!((present >> (g4 + 8)) & 1)) c[2] = c[3] = -INFINITY;
        }
        // the maxima move (and what was summed is rescaled) only when a score
        // passes one by more than kLazyMax: no reduction in the common case
        float mx[2] = {fmaxf(c[0], c[2]), fmaxf(c[1], c[3])};
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kLazyMax || mx[1] > m[1] + kLazyMax)) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], off));
                const bool up = mx[k] > m[k] + kLazyMax;
                const float by = up ? mx[k] - m[k] : 0.f;
                f[k] = fast_exp2(-by);
                if (up) m[k] = mx[k];
                l[k] *= f[k];
                if constexpr (INT8) {                // r grows as the weights so far shrink
                    const float lr_new = fminf(lr[k] + ceilf(by), kMostLr);
                    f[k] = fast_exp2(lr_new - lr[k] - by);
                    lr[k] = lr_new;
                    r[k] = fast_exp2(lr_new);
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
            const float sv0 = sc[kTile + g4], sv1 = sc[kTile + g4 + 8];
            float w[4] = {c[0] * sv0, c[1] * sv0, c[2] * sv1, c[3] * sv1};
            // a weight over 2^8 moves r (which starts far too high) to the largest
            if (__any_sync(0xffffffffu, fmaxf(fabsf(w[0]), fabsf(w[2])) * r[0] > 256.f ||
                                            fmaxf(fabsf(w[1]), fabsf(w[3])) * r[1] > 256.f)) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float top = fmaxf(fabsf(w[k]), fabsf(w[k + 2]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    if (top * r[k] > 256.f) {
                        // the power of two at or below 1 / top
                        const float lr_new = 127.f - (float)min((int)(__float_as_uint(top) >> 23), 252);
                        const float by = fast_exp2(lr_new - lr[k]);
                        lr[k] = lr_new;
                        r[k] = fast_exp2(lr_new);
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[i][k] *= by;
                            o[i][k + 2] *= by;
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = w[e] * r[e & 1];
        }
        uint32_t pa = pack16<INT8>(c[0], c[1]), pb = pack16<INT8>(c[2], c[3]);
        uint32_t ra_t = 0, rb_t = 0;
        const uint32_t ra = pack16_rest<INT8>(c[0], c[1], pa), rb = pack16_rest<INT8>(c[2], c[3], pb);
        if constexpr (!PAIRED) {
            ra_t = movmatrix_trans(ra);
            rb_t = movmatrix_trans(rb);
        } else if (q4 >= 2) {                        // columns 4-7: the remainders of heads 0-3
            pa = ra;
            pb = rb;
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
                    mma16<true>(o[2 * k2 + j], af, ra_t, rb_t);
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

    // 5. the warp's partial, into its ring: sums over its tokens, remainders added
    //    to their heads
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
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
        for (int i = 0; i < 2; ++i) {
            w_m[warp][h0 + i] = m[i];
            w_m2[warp][h0 + i] = INT8 ? m[i] - lr[i] : m[i];     // int8: o holds exp2(s - m) v_scale r
            w_l[warp][h0 + i] = l[i];
        }
    }
    __syncthreads();

    // 6. joined over the warps, in place of the first warp's, then over the cluster,
    //    where each CTA writes its share of the outputs
    const int64_t head0 = (int64_t)s * a.n_q_heads + (int64_t)h * G;
    auto finish = [&](int g, int d, const float4 &v, float M, float M2, float sum) {
        // o = 2^M2 v / (2^M sum); no token seen: 0
        const float inv = sum == 0.f ? 0.f : (M2 == -INFINITY ? 1.f : INT8 ? fast_exp2(M2 - M) : 1.f) / sum;
        *reinterpret_cast<uint2 *>(a.out + (head0 + g) * D + d) =
            make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        if (a.lse_out && d == 0)
            a.lse_out[head0 + g] = sum == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) * 0.69314718055994531f + logf(sum);
    };
    // joins a partial to what was joined before it.  One without a maximum has seen
    // nothing: its sums are 0 (or the NaN of a score).
    auto join = [&](float4 &v, float &M, float &M2, float &sum, const float4 &x, float xm, float xm2, float xl) {
        const float N = fmaxf(M, xm), N2 = fmaxf(M2, xm2);
        sum = sum * (M == -INFINITY ? 1.f : fast_exp2(M - N)) + xl * (xm == -INFINITY ? 1.f : fast_exp2(xm - N));
        const float f = M2 == -INFINITY ? 1.f : fast_exp2(M2 - N2), g = xm2 == -INFINITY ? 1.f : fast_exp2(xm2 - N2);
        v = make_float4(v.x * f + x.x * g, v.y * f + x.y * g, v.z * f + x.z * g, v.w * f + x.w * g);
        M = N;
        M2 = N2;
    };
    float4 *acc0 = reinterpret_cast<float4 *>(ring);
    for (int i = tid; i < G * (D / 4); i += 32 * WARPS) {
        const int g = i / (D / 4), d = (i % (D / 4)) * 4, at = (g * S::kAcc + d) / 4;
        float4 v = acc0[at];
        float M = w_m[0][g], M2 = w_m2[0][g], sum = w_l[0][g];
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            join(v, M, M2, sum, reinterpret_cast<const float4 *>(ring + (size_t)w * S::kStages * S::kStage)[at], w_m[w][g],
                 w_m2[w][g], w_l[w][g]);
        if (a.splits == 1) {
            finish(g, d, v, M, M2, sum);
        } else {
            acc0[at] = v;
            if (d == 0) c_stat[g] = make_float4(M, M2, sum, 0.f);
        }
    }
    if (a.splits == 1) return;
    cluster_sync_all();
    for (int i = rank * 32 * WARPS + tid; i < G * (D / 4); i += a.splits * 32 * WARPS) {
        const int g = i / (D / 4), d = (i % (D / 4)) * 4, at = (g * S::kAcc + d) / 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = -INFINITY, M2 = -INFINITY, sum = 0.f;
        constexpr int kRound = 8;                    // partials in flight
        for (int r0 = 0; r0 < a.splits; r0 += kRound) {
            float4 x[kRound], stat[kRound];
#pragma unroll
            for (int k = 0; k < kRound; ++k) {
                if (r0 + k >= a.splits) break;
                x[k] = ld_cluster(acc0 + at, r0 + k);
                stat[k] = ld_cluster(&c_stat[g], r0 + k);
            }
#pragma unroll
            for (int k = 0; k < kRound; ++k) {
                if (r0 + k >= a.splits) break;
                join(v, M, M2, sum, x[k], stat[k].x, stat[k].y, stat[k].z);
            }
        }
        finish(g, d, v, M, M2, sum);
    }
    cluster_sync_all();                              // no CTA leaves while another reads it
}

struct Choice {
    int splits = 0, occupancy = 0;   // CTAs of a unit, CTAs that an SM holds
    int64_t places = 0;      // CTAs that are resident at once
    int64_t room = 0;        // units that the machine's rounds of this launch have room for
    int64_t share = 0;       // the most tiles of a warp
};

// Dynamic shared memory with which an SM (228 KB, 1 KB of them kept back for each
// CTA) holds at most `per_sm` CTAs, which may be fewer than it has room for.
constexpr size_t smem_for(size_t need, int per_sm)
{
    const size_t most = 228 * 1024 / (size_t)(per_sm + 1) - 1024 + 128;
    return most > need ? most : need;
}

template <int D, bool INT8, bool WIDE, int WARPS>
cudaLaunchConfig_t launch_config(cudaLaunchAttribute (&at)[2], int64_t units, int splits, int per_sm, cudaStream_t stream)
{
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)splits;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(units * splits));
    lc.blockDim = dim3(32 * WARPS);
    lc.dynamicSmemBytes = smem_for(Shape<D, INT8>::smem(WARPS), per_sm);
    lc.stream = stream;
    lc.attrs = at;
    lc.numAttrs = splits > 1 ? 2 : 1;
    return lc;
}

constexpr int kDevices = 16;   // whose occupancies are remembered

// How many CTAs an SM of the current device holds; asked once, when the kernel's
// limit of shared memory is raised to the most that a launch asks for.
template <int D, bool INT8, bool WIDE, int WARPS>
cudaError_t resident_ctas(int *out)
{
    static std::atomic<int> known[kDevices];   // 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && (*out = known[dev]) > 0) return cudaSuccess;
    const void *kern = reinterpret_cast<const void *>(decode_window_kernel<D, INT8, WIDE, WARPS>);
    e = prepare_kernel(kern, 32 * WARPS, smem_for(Shape<D, INT8>::smem(WARPS), 1), nullptr);
    if (e != cudaSuccess) return e;
    e = prepare_kernel(kern, 32 * WARPS, Shape<D, INT8>::smem(WARPS), out);
    if (e != cudaSuccess) return e;
    if (*out < 1) return cudaErrorInvalidConfiguration;
    if (dev < kDevices) known[dev] = *out;
    return cudaSuccess;
}

// How many clusters of `splits` CTAs are resident at once on the current device with
// at most `per_sm` CTAs on an SM (clusters stay within a GPC, so not every SM can
// hold one); asked once.
template <int D, bool INT8, bool WIDE, int WARPS>
cudaError_t resident_clusters(int splits, int per_sm, int *out)
{
    constexpr int kPerSm = 32;
    static std::atomic<int> known[kDevices][kMaxSplits + 1][kPerSm + 1];   // the number + 1; 0: not asked yet
    const auto kern = decode_window_kernel<D, INT8, WIDE, WARPS>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev < kDevices && per_sm <= kPerSm;
    if (keep && known[dev][splits][per_sm] > 0) {
        *out = known[dev][splits][per_sm] - 1;
        return cudaSuccess;
    }
    if (splits > 8) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t lc = launch_config<D, INT8, WIDE, WARPS>(at, 1, splits, per_sm, nullptr);
    lc.attrs = at + 1;
    lc.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(out, kern, &lc);
    if (e != cudaSuccess) return e;
    if (keep) known[dev][splits][per_sm] = *out + 1;
    return cudaSuccess;
}

// The most CTAs per unit with which all CTAs of WARPS warps are resident at once
// and every warp keeps two tiles of the longest window; then as few as leave the
// longest share of a warp as it is.  Measured (8 kv heads of 128, windows of 1024
// where not said): two sequences of 16 K visible tokens over bf16 pages take 26 us
// with the 13 CTAs per unit that are resident at once and 40 with 16; four sequences
// over int8 pages 9.9 us with the 8 CTAs (of 4 warps) that two tiles a warp allow, 8.2
// with the 6 that give the longest share, three tiles, as well, and 12.0 with one
// tile a warp.
template <int D, bool INT8, bool WIDE, int WARPS>
cudaError_t choose(int64_t units, int64_t tiles, int sms, Choice *c)
{
    cudaError_t e = resident_ctas<D, INT8, WIDE, WARPS>(&c->occupancy);
    if (e != cudaSuccess) return e;
    c->places = (int64_t)sms * c->occupancy;
    int64_t n = c->places / units;
    if (n > tiles / (2 * WARPS)) n = tiles / (2 * WARPS);
    if (n > kMaxSplits) n = kMaxSplits;
    for (; n > 1; --n) {
        const int64_t share = (tiles + n * WARPS - 1) / (n * WARPS);
        n = (tiles + share * WARPS - 1) / (share * WARPS);
        if (n == 1) break;
        int clusters = 0;
        e = resident_clusters<D, INT8, WIDE, WARPS>((int)n, c->occupancy, &clusters);
        if (e != cudaSuccess) return e;
        if (clusters >= units) break;
    }
    c->splits = n < 1 ? 1 : (int)n;
    c->share = (tiles + c->splits * WARPS - 1) / (c->splits * WARPS);
    c->room = (units * c->splits + c->places - 1) / c->places * c->places / c->splits;
    return cudaSuccess;
}

// CTAs that do not fill the machine are spread over it by shared memory that is
// asked for but not used: placed as they come, behind a kernel that is draining,
// some SMs take as many as they hold and others none.  Measured (windows of 1024,
// 8 kv heads of 128, int8 pages, as placed / spread): 28 sequences 19.2 / 16.7 us, no
// difference at 8 and 56; bf16 pages, bound by memory, are 0 to 4 % faster.
template <int D, bool INT8, bool WIDE, int WARPS>
cudaError_t launch_as(WindowArgs &a, const Choice &c, int64_t units, int sms, cudaStream_t stream)
{
    a.splits = c.splits;
    const int64_t even = (units * c.splits + sms - 1) / sms;
    int per_sm = even < c.occupancy ? (int)even : c.occupancy;
    cudaError_t e;
    for (; c.splits > 1 && per_sm < c.occupancy; ++per_sm) {
        int clusters = 0;
        e = resident_clusters<D, INT8, WIDE, WARPS>(c.splits, per_sm, &clusters);
        if (e != cudaSuccess) return e;
        if (clusters >= units) break;
    }
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t lc = launch_config<D, INT8, WIDE, WARPS>(at, units, c.splits, per_sm, stream);
    return cudaLaunchKernelEx(&lc, decode_window_kernel<D, INT8, WIDE, WARPS>, a);
}

// CTAs of 4 warps, of 2 or of 8.
//
// Of 2 where their rounds leave less of the machine idle: by a fifth, or by anything
// once the units are more than the larger CTAs' places.  Measured (4 warps / 2 warps;
// windows of 1024, 8 kv heads of 128): bf16 pages, 32 sequences 23.6 / 24.7 us,
// 40: 37.9 / 30.3, 64: 45.4 / 42.9, 80: 61.7 / 66.4, 128: 87.5 / 82.3; int8 pages,
// 12 sequences 10.0 / 14.7, 48: 24.6 / 25.0, 64: 30.4 / 32.1, 80: 42.8 / 41.0,
// 128: 52.6 / 69.3.
//
// Of 8, for units that are all resident, where that shortens the longest share of a
// warp (a cluster has 16 CTAs at most), where it needs no cluster and CTAs of 4 do, or
// where there are more CTAs of 4 than SMs anyway.  Measured (4 warps / 8 warps; window
// and first tokens together): bf16 pages, 4 sequences of 256 visible tokens 5.4 / 5.0
// us, 12: 6.4 / 5.4; 1024 tokens, one sequence 5.7 / 6.1, 4: 7.4 / 6.4, 16: 15.0 / 14.1;
// 16 K tokens, one 19.7 / 17.4, two 26.4 / 27.3; int8 pages, 1024 tokens, 4: 7.5 / 6.9,
// 16: 13.1 / 11.7; 16 K, one 21.2 / 16.0, two 27.0 / 24.5.
template <int D, bool INT8, bool WIDE>
cudaError_t launch_sized(WindowArgs &a, int64_t units, int64_t tiles, int sms, cudaStream_t stream)
{
    Choice c4, c2, c8;
    cudaError_t e = choose<D, INT8, WIDE, 4>(units, tiles, sms, &c4);
    if (e != cudaSuccess) return e;
    e = choose<D, INT8, WIDE, 2>(units, tiles, sms, &c2);
    if (e != cudaSuccess) return e;
    e = choose<D, INT8, WIDE, 8>(units, tiles, sms, &c8);
    if (e != cudaSuccess) return e;
    const bool alone = c8.splits == 1 && c4.splits > 1 && c8.share <= c4.share;
    if (units <= c8.places && (alone || c8.share < c4.share || (units * c4.splits > sms && c8.room <= c4.room)))
        return launch_as<D, INT8, WIDE, 8>(a, c8, units, sms, stream);
    const bool small = units > c4.places ? c2.room <= c4.room : 5 * c2.room < 4 * c4.room;
    return small ? launch_as<D, INT8, WIDE, 2>(a, c2, units, sms, stream)
                 : launch_as<D, INT8, WIDE, 4>(a, c4, units, sms, stream);
}

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
    // ceil(2^32 / n) is 2^32 / n and less than 1 more, so its product with a tile index below
    // 2^27, over 2^32, is above index / n by less than 2^27 / 2^32 = 1 / 32.  The next whole
    // number is at least 1 / n further, which is more for every n up to 32.
    static_assert(PKV_WINDOW_MAX_TOKENS / kTile < 1 << 27 && kMaxBlockSize / kTile <= 32, "the lookup's rounding");
    a->tiles_per_block = (uint32_t)dims.block_size / kTile;
    a->block_magic = (uint32_t)((0x100000000ull + a->tiles_per_block - 1) / a->tiles_per_block);
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
