// prefill_window.cu -- chunked prefill attention under a sliding window with first
// tokens that stay visible (pagedkv_window.h), on the 5th-generation tensor cores.
//
// The tiles, warp roles and products are those of prefill_tc.cu: a unit is a
// (sequence, kv head, two adjacent tiles of 128 query rows), warps 0-3 and 4-7 are
// the softmax warpgroups of its two tiles, warps 8 and 10 load K, warp 11 loads V,
// warp 9 issues the products S = Q K^T and O += P V with P in TMEM.  What the window
// changes:
//
// Few keys.  A window of 1024 makes nine tiles of 128 keys, so what a unit costs
// beside its tiles (looking up the first block, loading Q and the first K, the last
// softmax, writing O: 9 us of 21 when every unit was a CTA of its own) weighs as
// much as the tiles.  The CTAs are therefore persistent, one per SM, and every role
// runs on from unit to unit: the producers load the next unit's K and V while this
// one's last tiles are computed, its Q as soon as the last S has been read, and the
// first S of the next unit is issued before the softmax warpgroups have written O.
//
// Packed keys.  The keys of a unit are the 16-key groups that hold first tokens,
// then those from the window of its first query on, packed behind one another into
// tiles of eight groups: a few first tokens or a window that starts inside a tile
// cost a group and not a tile.  Groups between the two are neither looked up nor
// loaded, and rows of loaded groups that no query sees are zeroed in V (a row of K
// needs nothing: its scores are replaced).
//
// Half units.  What is left over when the units are dealt out to the CTAs is cut into
// units of one query tile where that gives every CTA at most one more (512 units on
// 152 CTAs: three rounds and 112 halves in place of four rounds).  In a half unit both
// softmax warpgroups work on the one query tile, each on 64 of a tile's 128 keys; they
// exchange row maxima through shared memory, and S goes to the columns of the two query
// tiles in turn, so that the next S is computed during a softmax.  A tile takes 1.03 us
// there (1.47 with one warpgroup); 64 units take 22.5 us whole, 16.4 as halves,
// 192: 42.7 / 37.8, 320: 60.1 / 55.1, 512: 78.6 / 74.1.  Sums of a row are kept over the
// first and the last 64 keys of its tiles in whole units too, so that a row has the
// same bits in both and its result does not depend on the batch.
//
// O goes out from registers, a row of head_dim values a thread: the shared memory
// that could stage it holds the next unit's tiles by then.
//
// Rounding.  Scores, maxima, sums and O are binary32.  P is rounded once to bf16 (2^-8 of
// a probability at most), as in prefill_tc.cu: a product on the tensor cores takes P and
// V in one type, and P's remainder would need a second product and as many TMEM stores
// again.  Against 64 bits the outputs are 0.0021 to 0.0023 off (the norm of the difference
// over theirs), where their own rounding to bf16 makes 0.0016.
//
// Measured (32 query and 8 kv heads of 128, kernels back to back).  8 x 512 tokens,
// window 1024: 74 us with prefixes of 2 to 8 K, and 77.5 with prefixes of 0 to 8 K whose
// last sequence is the shortest (the halves are small ones then), 818 TFLOP/s of
// products that the mask asks for: a tile of 128 keys takes 1.56 us (1.63 PFLOP/s on 152
// SMs) and a unit 4.1 us beside its nine (masked tiles, O, the hand-over).  A prompt of
// 4095 tokens, window 1000: 67.9 us, 878 TFLOP/s.  2 x 37 tokens: 7.5 us, the latency of
// a launch and of one tile's chain.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "window.h"

namespace pkv {
namespace {

constexpr int kTM = 128;           // query rows per tile (TMEM lanes)
constexpr int kNQ = 2;             // query tiles per unit
constexpr int kTN = 128;           // keys per K/V tile
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTileCols = 256;        // TMEM columns per query tile: S / P, O
constexpr uint32_t kOCol = 128;            // O's column within a query tile's range
constexpr int kThreads = 384;

// Ring slots (one 128-key tile each) of K and of V that fit beside the Q tiles.
template <int D>
__host__ __device__ constexpr int k_slots() { return D == 128 ? 3 : 6; }
template <int D>
__host__ __device__ constexpr int v_slots() { return D == 128 ? 2 : 4; }

// Register split (setmaxnreg), as in prefill_tc.cu but for a wider issuing side:
// with 72 / 216 the producers spill (1.63 us per tile against 1.56).
constexpr int kLaunchRegs = 168;
constexpr int kRegsIssue = 88;
constexpr int kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= kThreads * kLaunchRegs, "register split above the launch");

struct WinParams {
    int32_t n_q_heads, group, chunk;
    int32_t n_blocks, block_size;
    int32_t pool_rows;            // (n_blocks + 1) * block_size: an out-of-range TMA row
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *prefix_lens;
    float scale_log2;
    __nv_bfloat16 *out;
    float *lse_out;
    int32_t *dev_status;
    int32_t pairs_per_seq;        // units per (sequence, kv head)
    int32_t n_kv_heads;
    int32_t n_full, n_units;      // units of two tiles, then those of one; below 2^31 - 2 * the grid
    int32_t window, sinks;
    int32_t wide_out;             // out is 32-byte aligned: one store for two (77.6 us, else 80.6)
    unsigned long long wait_ns;   // limit of the pipeline waits
};

// A unit and its keys.  Place c of the packed keys is key c below n_first (the
// groups with first tokens), else key c + skip; keys in [sinks, w_lo) are seen by
// no query of the unit.  A sequence of bad length has one tile without keys, whose
// output is not written (p_last -1), and so has a half unit past the chunk's end.
struct Unit {
    int32_t s, kvh, p0, p_last, P;
    int32_t w_lo, n_first, skip, n_places, n_kt;
};

// Unit u: sequence-major, the late positions of a sequence first, kv heads
// innermost.  One copy of it, out of line: inlined into every role it made the
// loops over the tiles a fifth slower (instruction fetches).
__device__ __noinline__ void find_unit(const WinParams &p, int32_t u, Unit *out)
{
    Unit w;
    const int32_t half = u >= p.n_full ? (u - p.n_full) & 1 : 0, tiles = u >= p.n_full ? 1 : kNQ;
    if (u >= p.n_full) u = p.n_full + (u - p.n_full) / 2;
    const int32_t per_seq = p.pairs_per_seq * p.n_kv_heads;
    w.s = u / per_seq;
    const int32_t in = u - w.s * per_seq, pair = in / p.n_kv_heads;
    w.kvh = in - pair * p.n_kv_heads;
    const int32_t positions = kTM / p.group;         // of a query tile
    w.p0 = ((p.pairs_per_seq - 1 - pair) * kNQ + half) * positions;
    w.p_last = min(w.p0 + tiles * positions, p.chunk) - 1;
    w.P = __ldg(p.prefix_lens + w.s);
    int32_t n_keys = 0;
    w.w_lo = 0;
    if (w.P < 0 || (int64_t)w.P + p.chunk > (int64_t)p.max_blocks * p.block_size) {   // alike for all units of a sequence
        w.P = 0;
        w.p_last = -1;
    } else if (w.p0 <= w.p_last) {
        n_keys = w.P + w.p_last + 1;
        // (of the whole unit: a row's keys are packed alike in both, so that its result does
        // not depend on which of the two the batch made it)
        w.w_lo = max(0, w.P + (p.pairs_per_seq - 1 - pair) * kNQ * positions - p.window + 1);
    }
    w.n_first = (min(p.sinks, n_keys) + 15) & ~15;
    w.skip = max((w.w_lo & ~15) - w.n_first, 0);
    w.n_places = n_keys - w.skip;
    w.n_kt = max(1, (w.n_places + kTN - 1) / kTN);
    *out = w;
}

// max(a, b, c) in one instruction (sm_100 and later).
__device__ __forceinline__ float fmax3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Byte of 16-byte chunk `chunk` of row `row` in a tile of 128-byte rows (128-byte swizzle).
__device__ __forceinline__ uint32_t swz128(uint32_t row, uint32_t chunk)
{
    return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// Bits 0 .. n - 1 of a word (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int32_t n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// mbar_wait in half its code (with the loop of write_o, 100 KB -> 90 of the kernel, 68.6
// -> 68.0 us on a prompt of 4095 tokens): one loop for limits that are polled for and
// for those that the hardware waits through.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int32_t *abort_flag, unsigned long long limit_ns)
{
    if (mbar_test_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (limit_ns < kWaitTimeoutNs ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (*abort_flag || global_timer_ns() - t0 > limit_ns) return false;
    }
}

// ---- products issued by one lane of a converged warp ----------------------------
// The issuing warp runs as a whole and the instructions carry the elected lane's
// predicate, so that the compiler keeps descriptors and addresses in uniform
// registers, where tcgen05 takes them from; issued from inside a branch for one
// lane, every operand is first moved there, and the moves stand between the
// products.

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

// D (TMEM) = A B over STEPS x 16 elements; descriptor words of A and B: the upper
// one and, per step, the lower one.
template <int STEPS>
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint32_t hi, const uint32_t (&a)[STEPS],
                                       const uint32_t (&b)[STEPS], uint32_t idesc)
{
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
        asm volatile(
            "{\n\t.reg .pred e, p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 e, %0, 0;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "mov.b64 da, {%2, %4};\n\t"
            "mov.b64 db, {%3, %4};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%1], da, db, %5, p;\n\t}" ::"r"(leader),
            "r"(d_tmem), "r"(a[k]), "r"(b[k]), "r"(hi), "r"(idesc), "r"(k > 0 ? 1u : 0u)
            : "memory");
}

// D (TMEM) += A (TMEM, 8 columns per step) B; accumulate 0: the first step starts D.
template <int STEPS>
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t hi,
                                       const uint32_t (&b)[STEPS], uint32_t idesc, uint32_t accumulate)
{
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
        asm volatile(
            "{\n\t.reg .pred e, p;\n\t.reg .b64 db;\n\t"
            "setp.ne.b32 e, %0, 0;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "mov.b64 db, {%3, %4};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], db, %5, p;\n\t}" ::"r"(leader),
            "r"(d_tmem), "r"(a_tmem + 8 * k), "r"(b[k]), "r"(hi), "r"(idesc), "r"(k > 0 ? 1u : accumulate)
            : "memory");
}

__device__ __forceinline__ void commit_one(uint32_t leader, uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %0, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
        "r"(smem_u32(bar))
        : "memory");
}

// 32 bytes to a 32-byte-aligned address.
__device__ __forceinline__ void st_global_32(void *dst, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// ---- a row's scores: NC keys of a tile, from column col0 on -----------------------

// The scores of keys that the row does not see become -inf (exp2 gives 0).  The seen
// keys as bits, 32 at a time: those of the window (behind n_mixed columns: the same,
// skip further on) and the first tokens up to the row.
template <int NC>
__device__ __forceinline__ void mask_scores(uint32_t (&sv)[NC], int32_t col0, int32_t key_base, int32_t qpos, int32_t n_mixed,
                                            int32_t skip, int32_t window, int32_t sinks)
{
    const int32_t back = qpos - key_base + 1, first = min(sinks - key_base, back);
    const int32_t back_w = n_mixed > 0 ? back - skip : back;
    const int32_t low = back < window ? 0 : back - window;
    const int32_t low_w = back_w < window ? 0 : back_w - window;
#pragma unroll
    for (int i0 = 0; i0 < NC; i0 += 32) {
        const int32_t at = col0 + i0;
        uint32_t seen = bits_below(back_w - at) & ~bits_below(low_w - at);
        if (n_mixed > 0) {
            const uint32_t mixed = bits_below(n_mixed - at);
            seen = (seen & ~mixed) | (mixed & bits_below(back - at) & ~bits_below(low - at));
        }
        seen |= bits_below(first - at);
        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((seen >> i) & 1)) sv[i0 + i] = __float_as_uint(-INFINITY);
    }
}

// The largest score: three-input maxima over four independent chains.
template <int NC>
__device__ __forceinline__ float largest(const uint32_t (&sv)[NC])
{
    float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NC; i += 8) {
        a0 = fmax3(a0, __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
        a1 = fmax3(a1, __uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3]));
        a2 = fmax3(a2, __uint_as_float(sv[i + 4]), __uint_as_float(sv[i + 5]));
        a3 = fmax3(a3, __uint_as_float(sv[i + 6]), __uint_as_float(sv[i + 7]));
    }
    return fmax3(a0, a1, fmaxf(a2, a3));
}

// The running maximum m (log2 units) moved by a tile's; the factor on what was summed.
__device__ __forceinline__ float move_maximum(float &m, float mx)
{
    float alpha = 1.f;
    if (m == -INFINITY) {
        m = mx;          // -inf until the first tile with a visible key
    } else if (mx > m + kRescaleThreshold) {
        alpha = fast_exp2(m - mx);
        m = mx;
    }
    return alpha;
}

// Probabilities of 64 scores from sv[I0] on (packed two-lane FMA for the exponent
// arguments), as bf16 pairs into 32 TMEM columns from taddr on; their sum.
template <int I0, int NC>
__device__ __forceinline__ float probabilities64(const uint32_t (&sv)[NC], float2 sc2, float2 nm2, uint32_t taddr)
{
    float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int k = I0 + i * 32 + 2 * e;
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), sc2, nm2);
            const float2 ee = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            if (e & 1)
                lb = __fadd2_rn(lb, ee);
            else
                la = __fadd2_rn(la, ee);
            pk[e] = pack_bf16x2(ee.x, ee.y);
        }
        tmem_st16_async(taddr + i * 16, pk);
    }
    return (la.x + la.y) + (lb.x + lb.y);
}

// The O of a row from taddr on, 32 columns at a time, times alpha.
template <int COLS>
__device__ __forceinline__ void rescale_o(uint32_t taddr, float alpha)
{
#pragma unroll 1
    for (int i = 0; i < COLS / 32; ++i) {
        uint32_t v[32];
        tmem_ld32_async(taddr + i * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
        tmem_st32(taddr + i * 32, v);
    }
}

// The O of a row from taddr on, times inv, to out where the row is live.  (Not unrolled:
// it runs once a unit, and code that runs so seldom is mostly fetched.)
template <int COLS>
__device__ __forceinline__ void write_o(uint32_t taddr, float inv, bool live, bool wide, __nv_bfloat16 *out)
{
#pragma unroll 1
    for (int i = 0; i < COLS / 32; ++i) {
        uint32_t v[32];
        tmem_ld32_async(taddr + i * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = pack_bf16x2(__uint_as_float(v[16 * q2 + 2 * e]) * inv, __uint_as_float(v[16 * q2 + 2 * e + 1]) * inv);
            if (!live) continue;
            if (wide) {
                st_global_32(out + i * 32 + q2 * 16, x);
            } else {
                *reinterpret_cast<uint4 *>(out + i * 32 + q2 * 16) = make_uint4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4 *>(out + i * 32 + q2 * 16 + 8) = make_uint4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_window_kernel(const __grid_constant__ CUtensorMap q_map,
                                                                     const __grid_constant__ CUtensorMap k_map,
                                                                     const __grid_constant__ CUtensorMap v_map,
                                                                     const __grid_constant__ WinParams p)
{
    constexpr int PANELS = D / 64;                          // 64-column (128-byte) panels of a bf16 row
    constexpr int NK = k_slots<D>(), NV = v_slots<D>();
    constexpr uint32_t kQPanel = kTM * 128u;                // 16 KiB: one panel of a 128-row Q tile
    constexpr uint32_t kQTile = PANELS * kQPanel;
    constexpr uint32_t kKVPanel = kTN * 128u;               // 16 KiB: one panel of a 128-key K tile
    constexpr uint32_t kSlotBytes = PANELS * kKVPanel;      // one K or V tile
    constexpr uint32_t kVGroup = PANELS * 2048u;            // one 16-key group of a V tile (all panels)

    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *q_s = base;                                    // kNQ Q tiles
    // K tile: [panel][128 keys][128 B]; V tile: [16-key group][panel][16 keys][128 B]
    uint8_t *k_ring = q_s + kNQ * kQTile;                   // NK K tiles
    uint8_t *v_ring = k_ring + NK * kSlotBytes;             // NV V tiles
    uint64_t *bars = reinterpret_cast<uint64_t *>(v_ring + NV * kSlotBytes);
    uint64_t *q_full = bars + 0;                            // a unit's Q tiles
    uint64_t *q_empty = bars + 1;                           // its last S products have read them
    uint64_t *k_full = bars + 2;                            // [NK]
    uint64_t *k_empty = k_full + NK;                        // [NK]
    uint64_t *v_full = k_empty + NK;                        // [NV]
    uint64_t *v_empty = v_full + NV;                        // [NV]
    uint64_t *s_full = v_empty + NV;                        // [kNQ]: S in TMEM
    uint64_t *p_full = s_full + kNQ;                        // [kNQ]: P in TMEM
    uint64_t *o_done = p_full + kNQ;                        // [kNQ]: a unit's last P V product done
    uint64_t *fin_bar = o_done + kNQ;
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(fin_bar + 1);
    volatile int32_t *abort_flag = reinterpret_cast<int32_t *>(fin_bar + 2);
    // Units: [4] of the issuer and the softmax warpgroups, written by warp 8 before it
    // loads a unit's Q (unit i at i % 4: by then everyone is past unit i - 3), and [4]
    // of warps 8-11, which run ahead of that.
    Unit *unit_s = reinterpret_cast<Unit *>(bars + 32);
    // Half units: a warp of one softmax warpgroup meets the one with the same rows of the
    // other; their maxima and sums go through the second Q tile, which a half unit leaves.
    __shared__ uint64_t pair_bar[4];
    float *pair_s = reinterpret_cast<float *>(q_s + kQTile);   // [2][2 warpgroups][128 rows]
    const int n_mine = (p.n_units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // units of this CTA
    static_assert(2 + 2 * (NK + NV) + 3 * kNQ + 3 <= 32, "barriers fit their 256 bytes");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    const int pos_per_tile = kTM / G;

    // a half unit is the last of its CTA
    auto is_half = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x >= p.n_full; };

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 2);   // the two K producers
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kNQ; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&pair_bar[i], 2);
        mbar_init(fin_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_base_s)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 8 && lane == 0) prefetch_tensormap(&q_map);
    if ((warp == 8 || warp == 10) && lane == 0) prefetch_tensormap(&k_map);
    if (warp == 11 && lane == 0) prefetch_tensormap(&v_map);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_s;
    // launched as a programmatic dependent: what is above overlaps the preceding
    // grid's end; no memory that it may write is read before the wait
    grid_dependents_launch();
    grid_dependency_wait();

    if (warp >= 4 * kNQ) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue) : "memory");
        if (warp != 9) {
            // ===================== TMA producers =====================
            const bool is_v = warp == 11;
            // this warp's 16-key groups: all eight (V) or four (each K warp)
            const int n_grp = is_v ? kTN / 16 : kTN / 32;
            const int grp = is_v ? lane : (warp == 10 ? kTN / 32 : 0) + lane;
            const int NSL = is_v ? NV : NK;
            uint64_t *full = is_v ? v_full : k_full;
            uint64_t *empty = is_v ? v_empty : k_empty;
            uint8_t *ring = is_v ? v_ring : k_ring;
            const uint32_t bytes = is_v ? kSlotBytes : kSlotBytes / 2;
            // block ids are read one tile ahead, across units, and turned into pool rows
            // when the tile is issued
            Unit *mine = unit_s + 4 + (warp - 8);
            int32_t kvh = 0, n_first = 0, skip = 0, n_places = 0, n_kt = 0;
            const int32_t *trow = nullptr;
            auto load_unit = [&](int i) {
                __syncwarp();
                if (lane == 0) find_unit(p, (int)blockIdx.x + i * (int)gridDim.x, mine);
                __syncwarp();
                const volatile Unit &w = *mine;
                kvh = w.kvh;
                n_first = w.n_first;
                skip = w.skip;
                n_places = w.n_places;
                n_kt = w.n_kt;
                trow = p.tables + (int64_t)w.s * p.max_blocks;
            };
            // the key at a place of the unit, and the block of this lane's group of tile j
            auto key_of = [&](int32_t place) { return place >= n_first ? place + skip : place; };
            auto load_block = [&](int j) -> int32_t {
                const int32_t place = j * kTN + grp * 16;
                return (lane < n_grp && place < n_places) ? __ldg(trow + key_of(place) / p.block_size) : 0;
            };
            load_unit(0);
            int32_t blk = load_block(0);
            int j = 0, issued = 0, unit = 0, q_loads = 0;   // tile of the unit, tiles so far, unit, Qs that lane 0 has issued
            while (unit < n_mine) {
                int32_t row = p.pool_rows;  // out of range: the box reads zeros
                const int32_t place = j * kTN + grp * 16;
                if (lane < n_grp && place < n_places) {
                    if (blk < 0 || blk > p.n_blocks)
                        report(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
                    else
                        row = blk * p.block_size + key_of(place) % p.block_size;
                }
                const int32_t t_kvh = kvh, t_unit = unit;          // of this tile
                const bool first = j == 0;
                if (warp == 8 && first && lane == 0) {             // handed on with the unit's Q, below
                    unit_s[unit & 3] = *mine;
                    if (mine->p_last < 0) report(p.dev_status, PKV_DEV_BAD_LENGTH);
                }
                if (++j == n_kt) {
                    j = 0;
                    if (++unit < n_mine) load_unit(unit);
                }
                if (unit < n_mine) blk = load_block(j);
                const int st = issued % NSL, use = issued / NSL;
                if (lane == 0 && !wait_for(&empty[st], (use & 1) ^ 1, abort_flag, p.wait_ns)) {
                    report(p.dev_status, PKV_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
                uint8_t *dst = ring + st * kSlotBytes;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                if (lane < n_grp) {
                    if (is_v) {
                        tma_load_3d(dst + grp * kVGroup, &v_map, 0, row, t_kvh * PANELS, &full[st]);
                    } else {
#pragma unroll
                        for (int h = 0; h < PANELS; ++h)
                            tma_load_3d(dst + h * kKVPanel + grp * 2048, &k_map, h * 64, t_kvh, row, &full[st]);
                    }
                }
                ++issued;
                if (warp == 8 && first) {   // the unit's Q, once the last unit's has been read
                    if (lane == 0) {
                        if (!wait_for(q_empty, (t_unit & 1) ^ 1, abort_flag, p.wait_ns)) {
                            report(p.dev_status, PKV_DEV_TIMEOUT);
                            *abort_flag = 1;
                        } else {
                            const Unit &w = unit_s[t_unit & 3];
                            const int n_q = is_half(t_unit) ? 1 : kNQ;
                            mbar_arrive_expect_tx(q_full, n_q * kQTile);
                            for (int i = 0; i < n_q; ++i)
                                for (int h = 0; h < PANELS; ++h)
                                    tma_load_3d(q_s + i * kQTile + h * kQPanel, &q_map, h * 64, t_kvh * G,
                                                w.s * p.chunk + w.p0 + i * pos_per_tile, q_full);
                            ++q_loads;   // (lane 0's: another role may have raised the flag by now)
                        }
                    }
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
                }
            }
            // every copy this warp issued has landed before the CTA can exit
            if (lane == 0) {
                if (warp == 8 && q_loads > 0) (void)mbar_wait(q_full, (q_loads - 1) & 1);
                for (int i = issued > NSL ? issued - NSL : 0; i < issued; ++i)
                    (void)mbar_wait(&full[i % NSL], (i / NSL) & 1);
            }
        } else {
            // ===================== MMA issuer =====================
            const uint32_t idesc_s = umma_idesc_bf16(kTM, kTN, false, false);
            const uint32_t idesc_o = umma_idesc_bf16(kTM, D, false, true);
            const uint32_t leader = elect_one();
            // The warp's waits keep the default limit, which compiles to the plain wait; when
            // another role's wait runs out, the abort flag ends these.
            auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(bar, phase, abort_flag));
            };
            auto tiles_of = [&](int unit) -> int { return const_cast<volatile Unit *>(unit_s)[unit & 3].n_kt; };
            const uint32_t q_addr = smem_u32(q_s) >> 4, k_addr = smem_u32(k_ring) >> 4, v_addr = smem_u32(v_ring) >> 4;
            const uint64_t kd = umma_desc_sw128(0, 16, 1024), vd = umma_desc_sw128(0, 2048, 1024);
            const uint32_t k_hi = (uint32_t)(kd >> 32), k_lo = (uint32_t)kd, v_hi = (uint32_t)(vd >> 32), v_lo = (uint32_t)vd;
            // S = Q_t K^T of the K in a ring slot, in the S columns of query tile `at`, then
            // the commit that hands it on; it covers the product issued before it, too
            auto issue_s = [&](int t, int at, int slot) {
                constexpr int STEPS = D / 16;
                uint32_t qa[STEPS], kb[STEPS];
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    qa[k] = k_lo | (q_addr + (t * kQTile + (k / 4) * kQPanel + (k % 4) * 32) / 16);
                    kb[k] = k_lo | (k_addr + (slot * kSlotBytes + (k / 4) * kKVPanel + (k % 4) * 32) / 16);
                }
                mma_ss<STEPS>(leader, tmem + at * kTileCols, k_hi, qa, kb, idesc_s);
                commit_one(leader, &s_full[at]);
            };
            // O_t += P V: A = P (TMEM, in the columns of query tile `at`), B = V (MN-major:
            // 16-key group k at k * kVGroup)
            auto issue_o = [&](int t, int at, int slot, bool accumulate) {
                uint32_t vb[kTN / 16];
#pragma unroll
                for (int k = 0; k < kTN / 16; ++k) vb[k] = v_lo | (v_addr + (slot * kSlotBytes + k * kVGroup) / 16);
                mma_ts<kTN / 16>(leader, tmem + t * kTileCols + kOCol, tmem + at * kTileCols, v_hi, vb, idesc_o,
                                 accumulate ? 1u : 0u);
            };
            // The tile at hand is the last of its unit's when left is 1.  The S of the next tile
            // goes out behind each P V; at a unit's end it waits for the next unit's Q, so both
            // P V go first.
            int n_kt = 0, ks = 0, vs = 0;         // ring slots of the tile's K and V, and their phases
            uint32_t k_phase = 0, v_phase = 0;
            bool ok = wait(q_full, 0) && wait(&k_full[0], 0);
            if (ok) {
                n_kt = tiles_of(0);
                tc_fence_after();
#pragma unroll 1
                for (int t = 0; t < (is_half(0) ? 1 : kNQ); ++t) issue_s(t, t, 0);
                commit_one(leader, &k_empty[0]);
                if (n_kt == 1) commit_one(leader, q_empty);
            }
            int units = 0, left = n_kt;
            uint32_t phase = 0;                   // of p_full
            auto next_k = [&]() {                 // the next tile's K
                if (++ks == NK) {
                    ks = 0;
                    k_phase ^= 1;
                }
            };
            auto next_v = [&]() {
                phase ^= 1;
                if (++vs == NV) {
                    vs = 0;
                    v_phase ^= 1;
                }
            };
            bool whole = !is_half(0);
            while (ok && whole) {
                const bool first = left == n_kt, last = left == 1;
                next_k();
                ok = wait(&v_full[vs], v_phase);
#pragma unroll
                for (int t = 0; t < kNQ; ++t) {
                    if (!ok) break;
                    ok = wait(&p_full[t], phase);
                    if (!ok) break;
                    tc_fence_after();
                    issue_o(t, t, vs, !first);
                    if (last) {
                        commit_one(leader, &o_done[t]);
                    } else {
                        if (t == 0) {
                            ok = wait(&k_full[ks], k_phase);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        issue_s(t, t, ks);
                    }
                }
                if (!ok) break;
                commit_one(leader, &v_empty[vs]);
                if (last) {
                    if (++units == n_mine) break;
                    whole = !is_half(units);
                    ok = wait(&k_full[ks], k_phase) && wait(q_full, units & 1);
                    if (!ok) break;
                    n_kt = tiles_of(units);
                    tc_fence_after();
                    // (S_t's columns hold a P that the tensor core reads before)
#pragma unroll 1
                    for (int t = 0; t < (whole ? kNQ : 1); ++t) issue_s(t, t, ks);
                    left = n_kt + 1;
                }
                commit_one(leader, &k_empty[ks]);
                if (--left == 1) commit_one(leader, q_empty);   // S of the unit's last tile is issued
                next_v();
            }
            // A half unit (the last): tile j's S, then its P, in the columns of query tile
            // j & 1, so that the next S is computed while the softmax of this one runs
            if (ok && units < n_mine) {
#pragma unroll 1
                for (int j = -1; j < n_kt; ++j) {   // P V of tile j, S of tile j + 2
                    if (j >= 0) {
                        ok = wait(&v_full[vs], v_phase) && wait(&p_full[0], phase) && wait(&p_full[1], phase);
                        if (!ok) break;
                        tc_fence_after();
                        issue_o(0, j & 1, vs, j > 0);
                        if (j + 1 == n_kt) {
                            commit_one(leader, &o_done[0]);
                            commit_one(leader, &o_done[1]);
                        }
                        commit_one(leader, &v_empty[vs]);
                        next_v();
                    }
                    if (j + 2 >= n_kt) continue;
                    next_k();
                    ok = wait(&k_full[ks], k_phase);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(0, j & 1, ks);
                    commit_one(leader, &k_empty[ks]);
                }
            }
            if (!ok) {
                if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            // every MMA issued has retired before the TMEM is released
            commit_one(leader, fin_bar);
            (void)mbar_wait(fin_bar, 0);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax) : "memory");
        // ===================== softmax warpgroups: row r = TMEM lane r =====================
        const int qt = warp / 4;
        const int r = threadIdx.x % kTM;
        const uint32_t lanes = tmem + ((uint32_t)((warp % 4) * 32) << 16);
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        // (the unit stays in shared memory: a row's scores need the registers)
        int c = 0;                               // tiles so far
        bool ok = true;
        // V rows of a tile that were loaded but that no query of the unit sees may hold
        // anything.  There are some past the last key (tail) and at places [sinks, w_lo -
        // skip), between the first tokens and the window (gap).
        auto has_tail = [&](const volatile Unit &w, bool last) { return last && (w.n_places & 15) != 0; };
        auto has_gap = [&](const volatile Unit &w, int32_t place0, int32_t skip) {
            return w.w_lo > p.sinks && place0 < w.w_lo - skip && place0 + kTN > p.sinks;
        };
        // They are zeroed once V has landed (both warpgroups write the same zeros).
        auto clean_v = [&](const volatile Unit &w, int32_t place0, bool tail, bool gap) -> bool {
            const int32_t skip = w.skip, n_places = w.n_places;
            if (!__all_sync(0xffffffffu, wait_for(&v_full[c % NV], (c / NV) & 1, abort_flag, p.wait_ns))) return false;
            uint8_t *vs = v_ring + (c % NV) * kSlotBytes;
            auto zero_rows = [&](int from, int stop) {
                for (int i = r; i < (stop - from) * PANELS * 8; i += kTM) {
                    const int row = from + i / (PANELS * 8), pc = i % (PANELS * 8);
                    *reinterpret_cast<uint4 *>(vs + (row / 16) * kVGroup + (pc / 8) * 2048 + swz128(row % 16, pc % 8)) =
                        make_uint4(0, 0, 0, 0);
                }
            };
            if (tail) zero_rows(n_places - place0, ((n_places + 15) & ~15) - place0);
            if (gap) zero_rows(max(p.sinks - place0, 0), min(w.w_lo - skip - place0, kTN));
            fence_proxy_async_smem();   // zeroed V rows visible to the tensor core
            return true;
        };
        int units = 0;
        for (; units < n_mine && !is_half(units); ++units) {
            const volatile Unit &w = unit_s[units & 3];
            const uint32_t lane_base = lanes + qt * kTileCols;   // of this warpgroup's query tile
            int n_kt = 1;                        // read with the unit's first tile
            int32_t pos = 0, qpos = 0;
            float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // sums over the first and last 64 keys of the tiles
            for (int j = 0; j < n_kt; ++j, ++c) {
                ok = __all_sync(0xffffffffu, wait_for(&s_full[qt], c & 1, abort_flag, p.wait_ns));
                if (!ok) break;
                tc_fence_after();
                uint32_t sv[kTN];
#pragma unroll
                for (int i = 0; i < kTN / 32; ++i) tmem_ld32_async(lane_base + i * 32, sv + i * 32);
                // (the first S of a unit says that the unit has been written)
                if (j == 0) {
                    n_kt = w.n_kt;
                    pos = w.p0 + qt * pos_per_tile + r / G;
                    qpos = w.P + pos;
                }
                const int32_t place0 = j * kTN, n_first = w.n_first, skip = w.skip;
                const int32_t key_base = place0 + (place0 >= n_first ? skip : 0);
                // groups with first tokens, of the tile that goes on with the window
                const int n_mixed = skip > 0 && place0 < n_first ? min(n_first - place0, kTN) : 0;
                // rows whose keys in this tile are all visible need no per-key test
                const bool masked = __any_sync(0xffffffffu, key_base + kTN - 1 > qpos || n_mixed > 0 ||
                                                                (key_base <= qpos - p.window && key_base + kTN > p.sinks));
                const bool tail = has_tail(w, j == n_kt - 1), gap = has_gap(w, place0, skip);
                tmem_wait_ld();
                if (masked) mask_scores(sv, 0, key_base, qpos, n_mixed, skip, p.window, p.sinks);
                const float alpha = move_maximum(m, largest(sv) * p.scale_log2);
                // O row rescale (rare): O holds P V up to tile j - 1, complete since this S's
                // commit came after it
                if (__any_sync(0xffffffffu, alpha != 1.f) && j > 0) rescale_o<D>(lane_base + kOCol, alpha);
                // P (bf16 pairs) over S's first 64 columns, each 16-column store after the S
                // columns it covers were read
                const float2 nm2 = m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(-m, -m);
                l0 = l0 * alpha + probabilities64<0>(sv, sc2, nm2, lane_base);
                l1 = l1 * alpha + probabilities64<64>(sv, sc2, nm2, lane_base + 32);
                tmem_wait_st();
                if (tail || gap) {
                    ok = clean_v(w, place0, tail, gap);
                    if (!ok) break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[qt]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait_for(&o_done[qt], units & 1, abort_flag, p.wait_ns));
            if (!ok) break;
            tc_fence_after();
            // row r of O, normalised.  (O is read before this warp's next P is handed over,
            // and the next unit's first product into O comes after that.)
            const bool live = pos <= w.p_last;
            const float l = l0 + l1;
            const int64_t out_row = ((int64_t)w.s * p.chunk + pos) * p.n_q_heads + w.kvh * G + r % G;
            write_o<D>(lane_base + kOCol, 1.f / l, live, p.wide_out, p.out + out_row * D);
            if (live && p.lse_out) p.lse_out[out_row] = (m + __log2f(l)) * 0.69314718055994531f;
            tc_fence_before();
        }
        // A half unit: both warpgroups work on its query tile, each on 64 keys of a tile and
        // then on half of O; maxima and sums meet as they do in a row of a whole unit, so the
        // bits are the same.
        if (ok && units < n_mine) {
            const volatile Unit &w = unit_s[units & 3];
            uint64_t *pair = &pair_bar[warp % 4];
            // hands x to the other warpgroup's thread of this row and takes its x: the n-th time
            auto swap = [&](int n, float x) -> float {
                float *at = pair_s + (n & 1) * 2 * kTM + r;
                at[qt * kTM] = x;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pair);
                ok = __all_sync(0xffffffffu, wait_for(pair, n & 1, abort_flag, p.wait_ns));
                tc_fence_after();
                return at[(1 - qt) * kTM];
            };
            const int c0 = c;
            int n_kt = 1;
            int32_t pos = 0, qpos = 0;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n_kt; ++j, ++c) {
                ok = __all_sync(0xffffffffu, wait_for(&s_full[j & 1], (c0 + j / 2) & 1, abort_flag, p.wait_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_base = lanes + (j & 1) * kTileCols;
                uint32_t sv[kTN / 2];
#pragma unroll
                for (int i = 0; i < 2; ++i) tmem_ld32_async(s_base + qt * 64 + i * 32, sv + i * 32);
                if (j == 0) {
                    n_kt = w.n_kt;
                    pos = w.p0 + r / G;
                    qpos = w.P + pos;
                }
                const int32_t place0 = j * kTN, n_first = w.n_first, skip = w.skip;
                const int32_t key_base = place0 + (place0 >= n_first ? skip : 0);
                const int n_mixed = skip > 0 && place0 < n_first ? min(n_first - place0, kTN) : 0;
                const bool masked = __any_sync(0xffffffffu, key_base + kTN - 1 > qpos || n_mixed > 0 ||
                                                                (key_base <= qpos - p.window && key_base + kTN > p.sinks));
                const bool tail = has_tail(w, j == n_kt - 1), gap = has_gap(w, place0, skip);
                tmem_wait_ld();
                if (masked) mask_scores(sv, qt * 64, key_base, qpos, n_mixed, skip, p.window, p.sinks);
                // (behind it both warps have read S, which P is written over)
                const float mine = largest(sv), other = swap(j, mine);
                if (!ok) break;
                const float alpha = move_maximum(m, fmaxf(mine, other) * p.scale_log2);
                if (__any_sync(0xffffffffu, alpha != 1.f) && j > 0) {
                    // the P V of the tile before this one frees its V
                    ok = __all_sync(0xffffffffu, wait_for(&v_empty[(c - 1) % NV], ((c - 1) / NV) & 1, abort_flag, p.wait_ns));
                    if (!ok) break;
                    tc_fence_after();
                    rescale_o<D / 2>(lanes + kOCol + qt * (D / 2), alpha);
                }
                const float2 nm2 = m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(-m, -m);
                l = l * alpha + probabilities64<0>(sv, sc2, nm2, s_base + qt * 32);
                tmem_wait_st();
                if (tail || gap) {
                    ok = clean_v(w, place0, tail, gap);
                    if (!ok) break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[qt]);
            }
            if (ok) {
                const float other = swap(n_kt, l);
                l = qt == 0 ? l + other : other + l;
            }
            if (ok) ok = __all_sync(0xffffffffu, wait_for(&o_done[qt], units & 1, abort_flag, p.wait_ns));
            if (ok) {
                tc_fence_after();
                const bool live = pos <= w.p_last;
                const int64_t out_row = ((int64_t)w.s * p.chunk + pos) * p.n_q_heads + w.kvh * G + r % G;
                write_o<D / 2>(lanes + kOCol + qt * (D / 2), 1.f / l, live, p.wide_out, p.out + out_row * D + qt * (D / 2));
                if (live && qt == 0 && p.lse_out) p.lse_out[out_row] = (m + __log2f(l)) * 0.69314718055994531f;
                tc_fence_before();
            }
        }
        if (!ok) {
            if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    }
    // everyone meets here before the TMEM is released
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace

cudaError_t launch_prefill_window(const PrefillArgs &a, int32_t window, int32_t sinks, int num_sms, cudaStream_t stream)
{
    const pkv_dims &d = a.dims;
    const int G = a.n_q_heads / d.n_kv_heads;
    if (G > 16 || kTM % G != 0) return cudaErrorInvalidValue;
    WinParams p{};
    p.n_q_heads = a.n_q_heads;
    p.group = G;
    p.chunk = a.chunk;
    p.n_blocks = d.n_blocks;
    p.block_size = d.block_size;
    p.pool_rows = (d.n_blocks + 1) * d.block_size;
    p.tables = a.tables;
    p.max_blocks = a.max_blocks;
    p.prefix_lens = a.prefix_lens;
    p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse_out = a.lse_out;
    p.dev_status = a.dev_status;
    p.wait_ns = pipeline_wait_ns();
    const int pos_per_tile = kTM / G;
    p.pairs_per_seq = (a.chunk + kNQ * pos_per_tile - 1) / (kNQ * pos_per_tile);
    p.n_kv_heads = d.n_kv_heads;
    const int64_t units = (int64_t)p.pairs_per_seq * d.n_kv_heads * a.n_seqs;
    if (units > INT32_MAX - 4 * (int64_t)num_sms) return cudaErrorInvalidValue;
    const int32_t over = (int32_t)(units % num_sms), halves = 2 * over <= num_sms ? over : 0;
    p.n_full = (int32_t)units - halves;
    p.n_units = p.n_full + 2 * halves;
    p.window = window;
    p.sinks = sinks;
    p.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;

    CUtensorMap qmap, kmap, vmap;
    {
        const uint64_t dims[3] = {(uint64_t)d.head_dim, (uint64_t)a.n_q_heads, (uint64_t)a.n_seqs * a.chunk};
        const uint64_t strides[2] = {(uint64_t)d.head_dim * 2, (uint64_t)a.n_q_heads * d.head_dim * 2};
        const uint32_t box[3] = {64u, (uint32_t)G, (uint32_t)pos_per_tile};
        if (encode_tensor_map(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const uint64_t rows = (uint64_t)(d.n_blocks + 1) * d.block_size;
    const uint64_t row_bytes = (uint64_t)d.n_kv_heads * d.head_dim * 2;
    {
        // K: {64 columns, kv head, pool row}, one head and 16 rows per box
        const uint64_t dims[3] = {(uint64_t)d.head_dim, (uint64_t)d.n_kv_heads, rows};
        const uint64_t strides[2] = {(uint64_t)d.head_dim * 2, row_bytes};
        const uint32_t box[3] = {64u, 1u, 16u};
        if (encode_tensor_map(&kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.k_pool), dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    {
        // V: {64 columns, pool row, 64-column panel of all heads}: a box of 16
        // rows and a head's panels lands as [panel][row][128 B]
        const uint32_t panels = (uint32_t)d.head_dim / 64u;
        const uint64_t dims[3] = {64u, rows, (uint64_t)d.n_kv_heads * panels};
        const uint64_t strides[2] = {row_bytes, 128u};
        const uint32_t box[3] = {64u, 16u, panels};
        if (encode_tensor_map(&vmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.v_pool), dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }

    const int slots = d.head_dim == 128 ? k_slots<128>() + v_slots<128>() : k_slots<64>() + v_slots<64>();
    const size_t smem = 1024 + (size_t)kNQ * kTM * d.head_dim * 2 + (size_t)slots * kTN * d.head_dim * 2 + 32 * sizeof(uint64_t) +
                        8 * sizeof(Unit);
    // The register split assumes the block gets kLaunchRegs per thread: refuse
    // a build whose kernel was given fewer (its setmaxnreg.inc could not complete).
    static const bool regs_ok = [] {
        cudaFuncAttributes fa128{}, fa64{};
        return cudaFuncGetAttributes(&fa128, prefill_window_kernel<128>) == cudaSuccess &&
               cudaFuncGetAttributes(&fa64, prefill_window_kernel<64>) == cudaSuccess && fa128.numRegs >= kLaunchRegs &&
               fa64.numRegs >= kLaunchRegs;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)(p.n_units < num_sms ? p.n_units : num_sms));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    lc.attrs = pdl;
    lc.numAttrs = 1;
    cudaError_t e;
    if (d.head_dim == 128) {
        e = prepare_kernel(reinterpret_cast<const void *>(prefill_window_kernel<128>), kThreads, smem, nullptr);
        if (e != cudaSuccess) return e;
        return cudaLaunchKernelEx(&lc, prefill_window_kernel<128>, qmap, kmap, vmap, p);
    }
    e = prepare_kernel(reinterpret_cast<const void *>(prefill_window_kernel<64>), kThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&lc, prefill_window_kernel<64>, qmap, kmap, vmap, p);
}

}  // namespace pkv
