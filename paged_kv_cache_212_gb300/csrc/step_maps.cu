// step_maps.cu -- block tables and slot maps of one step, from the tokens that each
// sequence holds and adds (pagedkv_batch.h, paged_step_maps).
//
// With need(s) = ceil((lens + n_new) / bs) - ceil(lens / bs), everything follows from two
// exclusive sums over the sequences: of n_new (the packed batch's starts) and of need
// (places in the free list).  One launch: every CTA sums all sequences by itself, 2048 at
// a time (in 32 bits, at 2^31 - 1 at most), and then fills its own part, 512 tokens and some of
// the table rows.  A second
// launch, or a wait between CTAs, would cost more than sums that all CTAs repeat from L2.
// A token's block comes from the free list or, in the block that its sequence holds
// already, from a table entry that the call does not write, so no CTA waits for another.
//
// Measured: a step of 64 sequences 4.0 us (the launch and three dependent reads), 500
// sequences with 65 K new tokens 7.6, 4096 sequences of one token 11.2 (two rounds of sums),
// four prompts of 30 K tokens in all 6.1.
#include "common.cuh"
#include "launch.h"
#include "window.h"
#include "../../include/pagedkv_batch.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;                    // sequences per thread and round
constexpr int kRound = kThreads * kPer;    // sequences per round

struct MapArgs {
    const int32_t *lens, *n_new;
    int32_t n_seqs;
    const int32_t *free_blocks;
    int32_t n_free;
    const int32_t *cursor;
    int32_t n_blocks, block_size;
    int32_t *tables;
    int32_t max_blocks, n_tokens;
    int32_t *ctx_lens, *token_starts, *token_seqs, *positions;
    int64_t *slots;
    int32_t *cursor_out;
    int32_t *dev_status;
};

constexpr uint32_t kMost = 0x7fffffffu;

// The sum of two numbers up to 2^31 - 1, or that.
__device__ __forceinline__ uint32_t add_clipped(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// What a sequence holds and adds, as they are or (false) 0 and 0 where its length is bad.
__device__ __forceinline__ bool good_lengths(const MapArgs &a, int32_t &len, int32_t &add)
{
    if (len < 0 || add < 0 || (int64_t)len + add > (int64_t)a.max_blocks * a.block_size) {
        len = add = 0;
        return false;
    }
    return true;
}
__device__ __forceinline__ bool sequence(const MapArgs &a, int32_t s, int32_t &len, int32_t &add)
{
    len = a.lens[s];
    add = a.n_new[s];
    return good_lengths(a, len, add);
}

__device__ __forceinline__ int32_t blocks_of(int32_t tokens, int32_t bs)
{
    return (int32_t)(((uint32_t)tokens + (uint32_t)bs - 1u) / (uint32_t)bs);
}

// Place `at` of the free list: a block, or -1 (and a status bit).
__device__ __forceinline__ int32_t free_block(const MapArgs &a, int64_t at, int32_t *dev_status)
{
    if (at < 0 || at >= a.n_free) {
        report(dev_status, PKV_DEV_OUT_OF_BLOCKS);
        return -1;
    }
    const int32_t b = a.free_blocks[at];
    if (b < 0 || b >= a.n_blocks) {
        report(dev_status, PKV_DEV_BAD_BLOCK_ID);
        return -1;
    }
    return b;
}

__global__ void __launch_bounds__(kThreads) step_maps_kernel(const MapArgs a)
{
    __shared__ uint32_t tok_s[kRound], blk_s[kRound];    // exclusive sums within the batch
    __shared__ int32_t len_s[kRound];
    __shared__ uint32_t warp_tok[kThreads / 32], warp_blk[kThreads / 32];
    grid_dependents_launch();   // a programmatic dependent: nothing is read before the wait
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t bs = a.block_size;
    const int64_t token = (int64_t)blockIdx.x * kThreads + tid;
    const int64_t cursor = a.cursor ? (int64_t)*a.cursor : 0;
    const int64_t first_free = cursor < 0 ? (int64_t)a.n_free : cursor;   // a negative one: nothing is left
    // a table row is the work of `team` warps, or a warp's are several rows
    const int64_t n_warps = (int64_t)gridDim.x * (kThreads / 32), my_warp = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int32_t team = (int32_t)max((int64_t)1, min(n_warps / max(a.n_seqs, 1), (int64_t)1024));
    const int64_t n_teams = n_warps / team, my_team = my_warp / team;
    const int32_t member = (int32_t)(my_warp - my_team * team);
    uint32_t tok0 = 0, blk0 = 0;                         // sums of the rounds before
    bool mapped = false;
    for (int64_t s0 = 0; s0 < a.n_seqs; s0 += kRound) {
        // 1. the round's sums
        int32_t len[kPer], add[kPer], need[kPer];
        uint32_t tok = 0, blk = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t s = s0 + tid * kPer + i;
            len[i] = add[i] = 0;
            if (s < a.n_seqs) {
                len[i] = a.lens[s];
                add[i] = a.n_new[s];
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!good_lengths(a, len[i], add[i]) && blockIdx.x == 0) report(a.dev_status, PKV_DEV_BAD_LENGTH);
            need[i] = blocks_of(len[i] + add[i], bs) - blocks_of(len[i], bs);
            tok = add_clipped(tok, add[i]);
            blk = add_clipped(blk, need[i]);
        }
        uint32_t tok_in = tok, blk_in = blk;             // inclusive over the warp's lanes
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, tok_in, off), b = __shfl_up_sync(0xffffffffu, blk_in, off);
            if (lane >= off) {
                tok_in = add_clipped(tok_in, t);
                blk_in = add_clipped(blk_in, b);
            }
        }
        uint32_t tok_at = __shfl_up_sync(0xffffffffu, tok_in, 1), blk_at = __shfl_up_sync(0xffffffffu, blk_in, 1);
        if (lane == 0) tok_at = blk_at = 0;
        if (lane == 31) {
            warp_tok[warp] = tok_in;
            warp_blk[warp] = blk_in;
        }
        __syncthreads();
        // (lane w has warp w's sums; those of the warps before this one, and of all)
        uint32_t t = lane < kThreads / 32 ? warp_tok[lane] : 0u, b = lane < kThreads / 32 ? warp_blk[lane] : 0u;
        uint32_t t_before = lane < warp ? t : 0u, b_before = lane < warp ? b : 0u;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            t = add_clipped(t, __shfl_xor_sync(0xffffffffu, t, off));
            b = add_clipped(b, __shfl_xor_sync(0xffffffffu, b, off));
            t_before = add_clipped(t_before, __shfl_xor_sync(0xffffffffu, t_before, off));
            b_before = add_clipped(b_before, __shfl_xor_sync(0xffffffffu, b_before, off));
        }
        tok_at = add_clipped(tok_at, add_clipped(tok0, t_before));
        blk_at = add_clipped(blk_at, add_clipped(blk0, b_before));
        tok0 = add_clipped(tok0, t);
        blk0 = add_clipped(blk0, b);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            tok_s[tid * kPer + i] = tok_at;
            blk_s[tid * kPer + i] = blk_at;
            len_s[tid * kPer + i] = len[i];
            tok_at = add_clipped(tok_at, add[i]);
            blk_at = add_clipped(blk_at, need[i]);
        }
        __syncthreads();

        // 2. this thread's token, where it is one of the round's: the last sequence that
        //    starts at or before it
        const int32_t n_here = (int32_t)min((int64_t)kRound, a.n_seqs - s0);
        if (!mapped && token < a.n_tokens && token < (int64_t)tok0) {
            mapped = true;
            int32_t lo = 0, hi = n_here;                 // tok_s[lo] <= token < tok_s[hi]
            while (hi - lo > 1) {
                const int32_t mid = (lo + hi) >> 1;
                if ((int64_t)tok_s[mid] <= token)
                    lo = mid;
                else
                    hi = mid;
            }
            const int32_t s = (int32_t)s0 + lo;
            const int32_t len = len_s[lo];
            const int32_t pos = len + (int32_t)(token - tok_s[lo]);
            const int32_t at = (int32_t)((uint32_t)pos / (uint32_t)bs), held = blocks_of(len, bs);
            int32_t b;
            if (at < held) {
                b = __ldcg(a.tables + (int64_t)s * a.max_blocks + at);   // (no old copy of a line that others write stays in the L1)
                // (a scratch block in a row that begins with another one is not an inactive sequence's:
                // an earlier step found no block for it)
                const bool none = b == a.n_blocks && __ldcg(a.tables + (int64_t)s * a.max_blocks) != b;
                if (b < 0 || b > a.n_blocks || none) {
                    report(a.dev_status, none ? PKV_DEV_OUT_OF_BLOCKS : PKV_DEV_BAD_BLOCK_ID);
                    b = -1;
                }
            } else {
                b = free_block(a, first_free + (int64_t)blk_s[lo] + (at - held), nullptr);   // reported with the table entry
            }
            a.token_seqs[token] = s;
            a.positions[token] = pos;
            a.slots[token] = b < 0 ? -1 : (int64_t)b * bs + (pos - at * bs);
        }

        // 3. the table rows, team t's t, t + n_teams, ...
        for (int64_t s_at = my_team < s0 ? my_team + (s0 - my_team + n_teams - 1) / n_teams * n_teams : my_team;
             my_team < n_teams && s_at < s0 + n_here; s_at += n_teams) {
            const int32_t s = (int32_t)s_at, i = (int32_t)(s_at - s0);
            int32_t len, n;
            const bool good = sequence(a, s, len, n);
            if (lane == 0 && member == 0) {
                a.ctx_lens[s] = len + n;
                a.token_starts[s] = (int32_t)tok_s[i];
            }
            if (!good) continue;
            const int32_t held = blocks_of(len, bs), want = blocks_of(len + n, bs);
            int32_t *row = a.tables + (int64_t)s * a.max_blocks;
            const int32_t stop = len == 0 ? a.max_blocks : want;
            for (int64_t j = held + member * 32 + lane; j < stop; j += 32 * team) {
                int32_t b = -1;
                if (j < want) b = free_block(a, first_free + (int64_t)blk_s[i] + (j - held), a.dev_status);
                row[j] = b < 0 ? a.n_blocks : b;
            }
        }
        __syncthreads();
    }
    if (!mapped && token < a.n_tokens) {
        a.token_seqs[token] = -1;
        a.positions[token] = 0;
        a.slots[token] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.token_starts[a.n_seqs] = (int32_t)tok0;
        *a.cursor_out = (int32_t)min(cursor + (int64_t)blk0, (int64_t)kMost);
        if ((int64_t)tok0 > a.n_tokens) report(a.dev_status, PKV_DEV_BAD_POSITION);
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int paged_step_maps(const int32_t *lens, const int32_t *n_new, int32_t n_seqs, const int32_t *free_blocks,
                               int32_t n_free, const int32_t *cursor, int32_t n_blocks, int32_t block_size,
                               int32_t *block_tables, int32_t max_blocks, int32_t n_tokens, int32_t *ctx_lens,
                               int32_t *token_starts, int32_t *token_seqs, int32_t *positions, int64_t *slots,
                               int32_t *cursor_out, int32_t *dev_status, pkv_stream_t stream)
{
    const int st = check_dims(pkv_dims{n_blocks, block_size, 1, 64});
    if (st != PKV_OK) return st;
    if (n_seqs < 0 || n_free < 0 || max_blocks <= 0 || n_tokens < 0) return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks * block_size > 0x7fffffffLL) return PKV_ERR_OUT_OF_RANGE;
    if (!token_starts || !cursor_out || cursor == cursor_out) return PKV_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!lens || !n_new || !block_tables || !ctx_lens || ctx_lens == lens || ctx_lens == n_new))
        return PKV_ERR_INVALID_ARG;
    if (n_free > 0 && !free_blocks) return PKV_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!token_seqs || !positions || !slots)) return PKV_ERR_INVALID_ARG;
    const void *p4[] = {lens, n_new, free_blocks, cursor, block_tables, ctx_lens, token_starts, token_seqs, positions, cursor_out};
    for (const void *x : p4)
        if (reinterpret_cast<uintptr_t>(x) & 3u) return PKV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(slots) & 7u) return PKV_ERR_INVALID_ARG;
    MapArgs a{lens, n_new, n_seqs, free_blocks, n_free, cursor, n_blocks, block_size, block_tables, max_blocks, n_tokens,
              ctx_lens, token_starts, token_seqs, positions, slots, cursor_out, dev_status};
    const int64_t for_tokens = ((int64_t)n_tokens + kThreads - 1) / kThreads;
    const int64_t for_rows = ((int64_t)n_seqs + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t grid = for_tokens > for_rows ? for_tokens : for_rows;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(grid > 0 ? grid : 1));
    lc.blockDim = dim3(kThreads);
    lc.stream = (cudaStream_t)stream;
    lc.attrs = pdl;
    lc.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&lc, step_maps_kernel, a));
}
