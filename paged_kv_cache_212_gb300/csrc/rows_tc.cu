// rows_tc.cu -- packed query rows that all see the same keys (pagedkv_batch.h): the rows of
// a cross attention's sequence, or the queries of a group's sequences over the tokens that
// they share, on the 5th-generation tensor cores.
//
// A run (sequence or group) is the product of its rows x G query heads with its keys, one
// kv head at a time: o = softmax(q K^T) V without a mask inside.  A unit is a run, a kv head
// and up to 256 rows in two tiles of 128 (TMEM lanes); its keys go by in tiles of 128, as
// in prefill_window.cu: warps 0-3 and 4-7 are the softmax warpgroups of the two tiles,
// warps 8 and 10 load K, 11 loads V, 9 issues S = Q K^T and O += P V with P in TMEM.
//
// The split.  The units' tiles, one behind the other, are cut into equal shares, one per
// CTA, wherever the cuts fall: with few rows and long runs (64 rows behind 4096 tokens are
// 8 units) only a split over the keys fills the machine, and with many it keeps the last
// round whole.  Every CTA sums the runs' tiles by itself to find its share, since lengths
// stand in device memory.  A unit that is cut leaves partials in 32 bits (rows.h), at most
// one more per CTA.
//
// Rounding.  Scores, maxima, sums and O are binary32.  P is rounded once to bf16, as in
// prefill_window.cu; over int8 pages to fp16, as the values are (value_exponent).  Against 64
// bits outputs are 0.0023 off over bf16 pages and 0.0017 over int8 pages, where their own
// rounding to bf16 makes 0.0016.
//
// Measured.  4135 queries of 8 sequences, 1000 to 8191 keys, 32 query and 8 kv heads of 128:
// 163 us (174 to 178 under the power cap of a long run), 1.09 to 1.18 PFLOP/s of needed work; a tile of 128
// keys takes 1.52 us (1.68 PFLOP/s on 152 SMs), bound by the chain of S, softmax and P V of a
// query tile, a change of unit 3.2 us more (the output's stores, the next queries' load), the
// start 8 us and the join 8.  64 sequences behind 4096 tokens: 34 us.  1642 queries over int8
// pages, 24 and 8 heads of 64: 39.8 us; the same 4135 queries over int8 pages 338 us, 3.3 us a
// tile, bound by the warps that widen the codes.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "rows.h"
#include "softmax_tc.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kTM = 128;           // query head rows per tile (TMEM lanes)
constexpr int kNQ = 2;             // query tiles per unit
constexpr int kTN = 128;           // keys per K/V tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTileCols = 256;        // TMEM columns per query tile: S / P, O
constexpr uint32_t kOCol = 128;            // O's column within a query tile's range
constexpr int kBars = 48;          // barriers' room
constexpr int kDevices = 16;       // whose occupancies are remembered
constexpr int kScaleTiles = 4;     // int8: tiles whose scales are held
constexpr float kUp = 7.f;         // int8: log2 of what multiplies the probabilities
static_assert(kUp + kRescaleThreshold <= 15.f, "within fp16's range");
static_assert(kNQ * kTM == kUnitRows, "a unit's rows");

// What depends on the type of the pages: threads, ring slots (one 128-key tile each) of K
// and of V that fit beside the Q tiles, and the register split (setmaxnreg): bf16 as in
// prefill_window.cu; int8 has four warps more, which widen the codes.
template <int D, bool INT8>
struct Setup {
    static constexpr int kThreads = INT8 ? 512 : 384;
    static constexpr int kSlotsK = INT8 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);
    static constexpr int kSlotsV = INT8 ? (D == 128 ? 2 : 3) : (D == 128 ? 2 : 4);
    static constexpr int kLaunchRegs = INT8 ? 128 : 168;
    static constexpr int kRegsIssue = 88;
    static constexpr int kRegsWiden = 64;
    static constexpr int kRegsSoftmax = INT8 ? 176 : 208;
    static_assert(128 * kRegsIssue + (INT8 ? 128 * kRegsWiden : 0) + 256 * kRegsSoftmax <= kThreads * kLaunchRegs,
                  "register split above the launch");
    // (the scales of tile j + kScaleTiles overwrite those of tile j: its K slot is free by the
    // S of tile j + kScaleTiles - kSlotsK, which was issued behind the P of the tile before)
    static_assert(!INT8 || kScaleTiles > kSlotsK, "scales still in use");
    static constexpr size_t kSmem = 1024 + (size_t)kNQ * kTM * D * 2 + (size_t)(kSlotsK + kSlotsV) * kTN * D * 2 +
                                    kBars * sizeof(uint64_t) + 256 + (INT8 ? kScaleTiles * 2 * kTN * sizeof(float) : 0);
    static_assert(kSmem <= 227 * 1024 - 512, "shared memory");
};

struct RowsParams {
    int32_t n_q_heads, group, n_rows, n_kv_heads;
    int32_t n_blocks, block_size;
    int32_t pool_rows;            // (n_blocks + 1) * block_size: an out-of-range TMA row
    const int32_t *starts, *run_tables, *run_lens;
    int32_t n_runs, max_run_blocks;
    const int32_t *ctx_lens;      // decode: rows that end before their run does are not this kernel's; else null
    float scale_log2;
    __nv_bfloat16 *out;
    float *lse_out;
    RowsPartials part;
    const float *k_scales, *v_scales;   // int8 pages
    int32_t *dev_status;
    int32_t wide_out;             // out is 32-byte aligned
    int32_t sms;
    int32_t few;                  // runs of up to so many rows are another launch's
    float rest_weight;            // what a tile of a decode's own tokens costs an SM, in tiles of a run
    unsigned long long wait_ns;   // limit of the pipeline waits
};

// A CTA's part of a unit: tiles t0 .. t0 + n_kt - 1 of its run's keys.
struct Unit {
    int32_t g, kvh, pos, pos_end, len, t0, n_kt;
    int32_t last;                 // nothing behind it
    int32_t cut;                  // the unit has other parts
    int32_t last_cta;             // that has some of it
};

// The stream that the CTAs share: unit behind unit, each kUnitCost places and then a place
// for each of its tiles, so that a share with many short units is no longer than one with a
// few long ones.  CTA c has places [c base + min(c, more), ...) of base or (the first `more`)
// base + 1; base is above kUnitCost, so that every share holds a tile.
constexpr int kUnitCost = 2;
constexpr float kLate = 2.f;       // places by which a share's first tile is later than an own token's

struct Share {
    int64_t base, more;
    __device__ __forceinline__ int64_t start(int64_t c) const { return c * base + min(c, more); }
    __device__ __forceinline__ int32_t of(int64_t place) const
    {
        const int64_t wide = more * (base + 1);
        return (int32_t)(place < wide ? (uint64_t)place / (uint64_t)(base + 1) : more + (uint64_t)(place - wide) / (uint64_t)base);
    }
};

__device__ __forceinline__ int32_t tiles_of_run(const Run &r) { return (int32_t)(((uint32_t)r.len + kTN - 1u) / kTN); }
__device__ __forceinline__ int32_t pairs_of_run(const RowsParams &p, const Run &r)
{
    const int32_t positions = kNQ * (kTM / p.group);
    return (int32_t)(((uint32_t)r.rows + (uint32_t)positions - 1u) / (uint32_t)positions);
}
__device__ __forceinline__ int64_t places_of_run(const RowsParams &p, const Run &r)
{
    const int32_t n_kt = tiles_of_run(r);
    return n_kt == 0 ? 0 : (int64_t)pairs_of_run(p, r) * p.n_kv_heads * (n_kt + kUnitCost);
}

__device__ __forceinline__ Run run_of_params(const RowsParams &p, int32_t g)
{
    Run r = run_at(p.starts, p.run_lens, p.n_rows, p.max_run_blocks, p.block_size, g);
    if (r.rows <= p.few) r.rows = 0;
    return r;
}

// The parts of a CTA's share, one after the other, in the registers of a warp: lane i holds
// run g0 + i and the places before it.
struct Walker {
    int64_t at, stop;             // place in the stream, end of the share
    int32_t g0;
    Run run;
    int64_t before, upto;         // places before the lane's run, and with it

    __device__ __forceinline__ void load(const RowsParams &p, int64_t first)
    {
        const int lane = threadIdx.x & 31;
        run = Run{0, 0, 0, true};
        if (g0 + lane < p.n_runs) run = run_of_params(p, g0 + lane);
        const int64_t mine = places_of_run(p, run);
        upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        upto += first;
        before = upto - mine;
    }
    __device__ __forceinline__ void next(const RowsParams &p, const Share &share, Unit *u)
    {
        uint32_t here;
        while ((here = __ballot_sync(0xffffffffu, at >= before && at < upto)) == 0) {
            g0 += 32;
            if (g0 >= p.n_runs) {      // lengths that another stream changes meanwhile: an end in any case
                *u = Unit{0, 0, 0, 0, 0, 0, 1, 1, 0, 0};
                return;
            }
            load(p, __shfl_sync(0xffffffffu, upto, 31));
        }
        const int src = __ffs(here) - 1;
        const int32_t row0 = __shfl_sync(0xffffffffu, run.row0, src), rows = __shfl_sync(0xffffffffu, run.rows, src);
        const int64_t off = at - __shfl_sync(0xffffffffu, before, src);
        u->len = __shfl_sync(0xffffffffu, run.len, src);
        u->g = g0 + src;
        const Run r{row0, rows, u->len, true};
        const int32_t n_kt = tiles_of_run(r), pairs = pairs_of_run(p, r), places = n_kt + kUnitCost;
        const int32_t idx = (int32_t)((uint64_t)off / (uint32_t)places);
        const int32_t in = (int32_t)(off - (int64_t)idx * places);                      // place within the unit
        const int64_t end = at - in + places;                                           // of the unit
        u->kvh = (int32_t)((uint32_t)idx / (uint32_t)pairs);
        u->pos = row0 + (idx - u->kvh * pairs) * (kNQ * (kTM / p.group));
        u->pos_end = row0 + rows;
        u->t0 = max(in - kUnitCost, 0);
        u->n_kt = (int32_t)min((int64_t)n_kt, (int64_t)n_kt - (end - stop)) - u->t0;
        u->cut = u->n_kt < n_kt;
        u->last_cta = share.of(end - 1);
        u->last = stop - end <= kUnitCost;                                              // (no tile of the next one)
        at = end;
    }
};

// Four int8 codes as bf16: with the lower seven bits of a code as the mantissa of a bf16 of
// exponent 2^7, and 2^7 or (code < 0) 2^8 taken off, which is the code, exactly.
__device__ __forceinline__ uint2 codes_bf16x4(uint32_t x)
{
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t t = __byte_perm(x, 0x43434343u, i ? 0x4342 : 0x4140);
        const uint32_t low = t & 0xff7fff7fu, off = t & 0xff80ff80u;
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&low), *reinterpret_cast<const __nv_bfloat162 *>(&off));
        r[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint2(r[0], r[1]);
}

// Four int8 codes (code + 128 in x) times a scale as fp16: with a byte as the low one of
// the binary32 value 2^23 + byte, which the subtraction leaves as the code, exactly.
__device__ __forceinline__ uint2 scaled_f16x4(uint32_t x, float scale)
{
    const float2 bias = make_float2(-8388736.f, -8388736.f), s2 = make_float2(scale, scale);      // -(2^23 + 128)
    float2 a = make_float2(__uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7441)));
    float2 b = make_float2(__uint_as_float(__byte_perm(x, 0x4b000000u, 0x7442)), __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7443)));
    a = __fmul2_rn(__fadd2_rn(a, bias), s2);
    b = __fmul2_rn(__fadd2_rn(b, bias), s2);
    return make_uint2(pack_f16x2(a.x, a.y), pack_f16x2(b.x, b.y));
}

// int8: an exponent e with every V scale of a tile below 2^e (asked by a whole warp), and 2^e.
// Values are held as multiples of the power of two above the largest scale so far of their
// part of a unit, so that codes times scales stay within fp16's range and the largest keep
// its 11 bits; where it grows the softmax rescales O.  It is made from the same scales by the
// warps that widen and by the softmax.
__device__ __forceinline__ int value_exponent(const float *vs)
{
    const float4 x = *reinterpret_cast<const float4 *>(vs + 4 * (threadIdx.x & 31));
    float top = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    return min(max((int)(__float_as_uint(top) >> 23) - 126, -126), 126);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + max(e, -126)) << 23); }

// A box of a tensor map to the L2.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// A scale to shared memory, 0 where it is not there; and the barrier's arrival of this
// thread once its copies have landed.
__device__ __forceinline__ void copy_scale(float *dst, const float *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// int8: where in a slot the codes of 16 rows go.
// The bf16 values of a row are one piece of 128 bytes in each panel; head_dim 128: a row's
// codes lie in its piece of the second panel.  head_dim 64: the codes of 16 rows in the
// pieces of their last 8.
template <int D>
__device__ __forceinline__ uint32_t codes_at(bool is_v, uint32_t row)
{
    if (D == 64) return row / 16 * 2048 + 1024;
    return is_v ? row / 16 * 4096 + 2048 + row % 16 * 128 : kTN * 128u + row * 128;
}

template <int D, bool INT8>
__global__ void __launch_bounds__(Setup<D, INT8>::kThreads, 1) rows_kernel(const __grid_constant__ CUtensorMap q_map,
                                                           const __grid_constant__ CUtensorMap k_map,
                                                           const __grid_constant__ CUtensorMap v_map,
                                                           const __grid_constant__ RowsParams p)
{
    constexpr int PANELS = D / 64;                          // 64-column (128-byte) panels of a bf16 row
    using S = Setup<D, INT8>;
    constexpr int NK = S::kSlotsK, NV = S::kSlotsV, kThreads = S::kThreads;
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
    // int8: a tile's codes are there, at the beginning of the slot that they are widened into
    uint64_t *k_codes = INT8 ? o_done + kNQ : k_full;       // [NK]
    uint64_t *v_codes = INT8 ? k_codes + NK : v_full;       // [NV]
    uint64_t *sc_full = INT8 ? v_codes + NV : nullptr;      // [kScaleTiles]: their scales
    uint64_t *fin_bar = INT8 ? sc_full + kScaleTiles : o_done + kNQ;
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(fin_bar + 1);
    volatile int32_t *abort_flag = reinterpret_cast<int32_t *>(fin_bar + 2);
    // [4] units of the issuer and the softmax warpgroups, written by warp 8 before it
    // loads a unit's Q (unit i at i % 4: Q i - 1 was loaded, so the S of unit i - 2 were
    // issued, behind all of the P of unit i - 3 and so the epilogues of unit i - 4).
    Unit *unit_s = reinterpret_cast<Unit *>(bars + kBars);
    float *scale_s = reinterpret_cast<float *>(bars + kBars) + 64;   // int8: [kScaleTiles][K, V][128 keys]
    __shared__ int32_t tile_s[kScaleTiles];                 // int8: what a tile is
    constexpr int32_t kFirstTile = 1, kLastTile = 2;        // of a part, of the share
    static_assert(2 + (INT8 ? 3 : 2) * (NK + NV) + kScaleTiles + 3 * kNQ + 3 <= kBars && 4 * sizeof(Unit) <= 256, "their room");
    __shared__ int64_t warp_sum[kThreads / 32], warp_rest[kThreads / 32];
    __shared__ int32_t issued_s[2];                         // tiles that the K producers issued
    __shared__ CutUnit cut_s;                               // the last unit, where it goes on in the next CTA

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    const int pos_per_tile = kTM / G;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_codes[i], 2);  // the two K producers
            if (INT8) mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_codes[i], 1);
            if (INT8) mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kNQ; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        if (INT8)
            for (int i = 0; i < kScaleTiles; ++i) mbar_init(&sc_full[i], 64);   // the K producers' lanes
        mbar_init(fin_bar, 1);
        *abort_flag = 0;
        cut_s.last_cta = 0;
        issued_s[0] = issued_s[1] = 0;
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
    // launched as a programmatic dependent: what is above overlaps the preceding
    // grid's end; no memory that it may write is read before the wait.  The next grid may
    // start as soon as this one has waited: what it reads before its own wait was written
    // before this grid.
    grid_dependency_wait();
    grid_dependents_launch();

    Walker walk;                       // (the producers')
    walk.g0 = 0;
    if (warp >= 8 && warp < 12) walk.load(p, 0);
    // The share, from the runs' places and a decode's own tokens: each thread sums some runs,
    // the block sums the threads.
    Share share{0, 0};
    {
        int64_t sum = 0, rest = 0;       // places of the runs; own tokens, those that are shared taken off
        bool good = true;
        for (int32_t g = threadIdx.x; g < p.n_runs; g += kThreads) {
            const Run r = run_of_params(p, g);
            sum += places_of_run(p, r);
            good = good && r.good;
            if (p.ctx_lens) rest -= (int64_t)r.rows * r.len;
        }
        if (p.ctx_lens)
            for (int32_t i = threadIdx.x; i < p.n_rows; i += kThreads) rest += max(__ldcg(p.ctx_lens + i), 0);
        if (!good && blockIdx.x == 0) report(p.dev_status, PKV_DEV_BAD_LENGTH);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
            rest += __shfl_xor_sync(0xffffffffu, rest, off);
        }
        if (lane == 0) {
            warp_sum[warp] = sum;
            warp_rest[warp] = rest;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_s;
    {
        int64_t total = 0, rest = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            total += warp_sum[i];
            rest += warp_rest[i];
        }
        int64_t n_ctas = gridDim.x;
        if (rest > 0) {
            // n SMs for t places, the others for own tokens worth r of them, so that both are done
            // at once: t / n + kLate = r / (sms - n)
            const float r = (float)rest * p.n_kv_heads * p.rest_weight / kTN, t = (float)total, sms = (float)p.sms;
            const float h = t + r - kLate * sms, d = sqrtf(h * h + 4.f * kLate * t * sms);
            const float n = h > 0.f ? 2.f * t * sms / (d + h) : (d - h) / (2.f * kLate);
            n_ctas = min(n_ctas, max((int64_t)1, (int64_t)n));
            n_ctas = min(n_ctas + (n_ctas & 1), (int64_t)gridDim.x);   // whole TPCs (launch_as)
        }
        n_ctas = min(n_ctas, (int64_t)((uint64_t)total / (kUnitCost + 1)));
        if (blockIdx.x < n_ctas) {
            share.base = (int64_t)((uint64_t)total / (uint64_t)n_ctas);
            share.more = total - share.base * n_ctas;
        }
    }
    const bool any = share.base > 0;

    if (INT8 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsWiden) : "memory");
        // ===================== codes widened to bf16 =====================
        // K's codes as bf16, which holds them, and the softmax multiplies the scores by their
        // scales.  V's, with P in fp16, as code times scale in fp16, rounded once (2^-11), under
        // the unit's power of two (value_exponent).  (Scales of V on the probabilities, fetched by
        // every row's thread: 380 us where this takes 325; all scales rounded to bf16 here: 323,
        // but outputs twice as far off as over bf16 pages.)
        // In place: the codes of a row (head_dim 64: of 16 rows) lie where bf16 values of the
        // same rows go, so a warp reads some rows, then writes them.  (Loops, not unrolled code:
        // all reads before all writes, with 32 registers of codes, took 2.5 us a K tile.)
        constexpr int VECS = D / 16;                        // 16-byte vectors of a code row
        constexpr int AT_ONCE = D == 128 ? 4 : 2;           // vectors of a lane: 16 rows
        auto widen = [&](auto kind, uint8_t *slot, uint64_t *codes, uint64_t *full, uint32_t phase, const float *vs, float down) -> bool {
            constexpr bool is_v = decltype(kind)::value;
            if (!__all_sync(0xffffffffu, wait_for(codes, phase, abort_flag, p.wait_ns))) return false;
            const uint32_t vec = lane % VECS, odd = vec / 4 & 1, chunk = vec % 4 * 2;
#pragma unroll 1
            for (uint32_t row0 = (warp - 12) * 32; row0 < (warp - 12) * 32 + 32; row0 += 16) {
                uint4 x[AT_ONCE];
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) x[i] = *reinterpret_cast<const uint4 *>(slot + codes_at<D>(is_v, row0) + (i * 32 + lane) * 16);
                float scale[AT_ONCE];
                if constexpr (is_v) {
#pragma unroll
                    for (int i = 0; i < AT_ONCE; ++i) scale[i] = vs[row0 + (i * 32 + lane) / VECS] * down;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i) {
                    const uint32_t row = row0 + (i * 32 + lane) / VECS;
                    uint8_t *dst = slot + (is_v ? row / 16 * kVGroup + odd * 2048 + row % 16 * 128 : odd * kKVPanel + row * 128);
                    uint2 a, b, d, e;
                    if constexpr (is_v) {
                        a = scaled_f16x4(x[i].x ^ 0x80808080u, scale[i]);
                        b = scaled_f16x4(x[i].y ^ 0x80808080u, scale[i]);
                        d = scaled_f16x4(x[i].z ^ 0x80808080u, scale[i]);
                        e = scaled_f16x4(x[i].w ^ 0x80808080u, scale[i]);
                    } else {
                        a = codes_bf16x4(x[i].x);
                        b = codes_bf16x4(x[i].y);
                        d = codes_bf16x4(x[i].z);
                        e = codes_bf16x4(x[i].w);
                    }
                    const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(d.x, d.y, e.x, e.y);
                    // (the second panel's vectors in the other order: different banks)
                    *reinterpret_cast<uint4 *>(dst + (((chunk + odd) ^ (row & 7)) << 4)) = odd ? hi : lo;
                    *reinterpret_cast<uint4 *>(dst + (((chunk + 1 - odd) ^ (row & 7)) << 4)) = odd ? lo : hi;
                }
            }
            fence_proxy_async_smem();                       // visible to the tensor core
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            return true;
        };
        bool more = any;
        int exponent = 0;
        for (int c = 0; more; ++c) {
            const int ks = c % NK, vs = c % NV;
            const float *sc = scale_s + (c % kScaleTiles) * 2 * kTN + kTN;
            bool ok = widen(std::false_type{}, k_ring + ks * kSlotBytes, &k_codes[ks], &k_full[ks], (c / NK) & 1, sc, 1.f) &&
                      __all_sync(0xffffffffu, wait_for(&sc_full[c % kScaleTiles], (c / kScaleTiles) & 1, abort_flag, p.wait_ns));
            if (ok) {
                const int flags = const_cast<volatile int32_t *>(tile_s)[c % kScaleTiles], e = value_exponent(sc);
                exponent = flags & kFirstTile ? e : max(exponent, e);
                more = !(flags & kLastTile);
                ok = widen(std::true_type{}, v_ring + vs * kSlotBytes, &v_codes[vs], &v_full[vs], (c / NV) & 1, sc, power_of_two(-exponent));
            }
            if (!ok) {
                if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
                *abort_flag = 1;
                break;
            }
        }
    } else if (warp >= 4 * kNQ) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsIssue) : "memory");
        if (!any) {
        } else if (warp != 9) {
            // ===================== TMA producers =====================
            const bool is_v = warp == 11;
            // this warp's 16-key groups: all eight (V) or four (each K warp)
            const int n_grp = is_v ? kTN / 16 : kTN / 32;
            const int grp = is_v ? lane : (warp == 10 ? kTN / 32 : 0) + lane;
            const int NSL = is_v ? NV : NK;
            uint64_t *full = is_v ? v_codes : k_codes;
            uint64_t *empty = is_v ? v_empty : k_empty;
            uint8_t *ring = is_v ? v_ring : k_ring;
            const uint32_t bytes = (is_v ? kSlotBytes : kSlotBytes / 2) / (INT8 ? 2 : 1);
            // block ids are read one tile ahead, across units, and turned into pool rows
            // when the tile is issued
            Unit mine;
            walk.at = share.start(blockIdx.x);
            walk.stop = share.start((int64_t)blockIdx.x + 1);
            const int32_t *trow = nullptr;
            auto load_unit = [&]() {
                walk.next(p, share, &mine);
                trow = p.run_tables + (int64_t)mine.g * p.max_run_blocks;
            };
            // the block of this lane's group of tile j of the unit
            auto load_block = [&](int j) -> int32_t {
                const int32_t key = (mine.t0 + j) * kTN + grp * 16;
                return (lane < n_grp && key < mine.len) ? __ldcg(trow + key / p.block_size) : 0;
            };
            int q_loads = 0;                                // that lane 0 has issued
            // (a group that does not divide 128 leaves the tile's last rows as they are: rows of
            // S are independent of one another)
            auto load_q = [&](const Unit &w) {
                mbar_arrive_expect_tx(q_full, kNQ * PANELS * pos_per_tile * G * 128);
#pragma unroll 1
                for (int i = 0; i < kNQ * PANELS; ++i) {
                    const int t = i / PANELS, h = i % PANELS;
                    tma_load_3d(q_s + t * kQTile + h * kQPanel, &q_map, h * 64, w.kvh * G, w.pos + t * pos_per_tile, q_full);
                }
                ++q_loads;
            };
            auto prefetch_q = [&](const Unit &w) {          // to the L2 (a unit's switch: 1.7 us of loading)
#pragma unroll 1
                for (int i = 0; i < kNQ * PANELS; ++i)
                    tma_prefetch_3d(&q_map, i % PANELS * 64, w.kvh * G, w.pos + i / PANELS * pos_per_tile);
            };
            load_unit();
            if (warp == 8 && lane == 0) load_q(mine);       // the first unit's, before its block is known
            int32_t blk = load_block(0);
            int j = 0, issued = 0, unit = 0;                // tile of the unit, tiles so far, unit
            bool more = true;
            while (more) {
                int32_t row = p.pool_rows;  // out of range: the box reads zeros
                const int32_t key = (mine.t0 + j) * kTN + grp * 16;
                if (lane < n_grp && key < mine.len) {
                    if (blk < 0 || blk > p.n_blocks)
                        report(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
                    else
                        row = blk * p.block_size + key % p.block_size;
                }
                const int32_t t_kvh = mine.kvh, t_unit = unit;     // of this tile
                const int32_t t_here = mine.len - (mine.t0 + j) * kTN;   // int8: keys from its first on
                const bool first = j == 0;
                if (warp == 8 && first && lane == 0) {
                    unit_s[unit & 3] = mine;                       // handed on with the unit's Q, below
                    if (mine.cut && mine.t0 == 0) cut_s = CutUnit{mine.pos, mine.pos_end, mine.kvh, mine.last_cta};
                }
                if (++j == mine.n_kt) {
                    j = 0;
                    ++unit;
                    more = !mine.last;
                    if (more) load_unit();
                }
                if (more) blk = load_block(j);
                const int st = issued % NSL, use = issued / NSL;
                if (lane == 0 && !wait_for(&empty[st], (use & 1) ^ 1, abort_flag, p.wait_ns)) {
                    report(p.dev_status, PKV_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
                uint8_t *dst = ring + st * kSlotBytes;
                if (INT8 && !is_v) {                               // the scales of the warp's keys
                    const int key0 = warp == 10 ? kTN / 2 : 0;
                    float *sc = scale_s + (issued % kScaleTiles) * 2 * kTN + key0 + lane;
#pragma unroll
                    for (int i = 0; i < kTN / 2; i += 32) {
                        const int32_t r0 = __shfl_sync(0xffffffffu, row, (i + lane) / 16);
                        const bool in = key0 + i + lane < t_here && r0 != p.pool_rows;      // else 0: a row of zeros
                        const int64_t at = in ? ((int64_t)r0 + (lane & 15)) * p.n_kv_heads + t_kvh : 0;
                        copy_scale(sc + i, p.k_scales + at, in);
                        copy_scale(sc + kTN + i, p.v_scales + at, in);
                    }
                    copies_arrive(&sc_full[issued % kScaleTiles]);
                    // (ahead of the tile's codes, whose barrier hands it on)
                    if (warp == 8 && lane == 0) tile_s[issued % kScaleTiles] = (first ? kFirstTile : 0) | (more ? 0 : kLastTile);
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                if (lane < n_grp) {
                    if (INT8) {
                        tma_load_3d(dst + codes_at<D>(is_v, grp * 16), is_v ? &v_map : &k_map, 0, t_kvh, row, &full[st]);
                    } else if (is_v) {
                        tma_load_3d(dst + grp * kVGroup, &v_map, 0, row, t_kvh * PANELS, &full[st]);
                    } else {
#pragma unroll
                        for (int h = 0; h < PANELS; ++h)
                            tma_load_3d(dst + h * kKVPanel + grp * 2048, &k_map, h * 64, t_kvh, row, &full[st]);
                    }
                }
                ++issued;
                if (warp == 8 && first && t_unit > 0) {   // the unit's Q, once the last unit's has been read
                    if (lane == 0) {
                        prefetch_q(unit_s[t_unit & 3]);
                        if (!wait_for(q_empty, (t_unit & 1) ^ 1, abort_flag, p.wait_ns)) {
                            report(p.dev_status, PKV_DEV_TIMEOUT);
                            *abort_flag = 1;
                        } else {
                            load_q(unit_s[t_unit & 3]);
                        }
                    }
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
                }
            }
            // every copy this warp issued has landed before the CTA can exit (K's: all that is
            // issued is contracted, or settle_pair waits for it below)
            if (INT8) asm volatile("cp.async.wait_all;" ::: "memory");
            if (lane == 0) {
                if (warp == 8 && q_loads > 0) (void)mbar_wait(q_full, (q_loads - 1) & 1);
                if (is_v) {
                    for (int i = issued > NSL ? issued - NSL : 0; i < issued; ++i) (void)mbar_wait(&full[i % NSL], (i / NSL) & 1);
                } else {
                    issued_s[warp == 10] = issued;
                }
            }
        } else {
            // ===================== MMA issuer =====================
            const uint32_t idesc_s = umma_idesc_bf16(kTM, kTN, false, false);
            const uint32_t idesc_o = INT8 ? umma_idesc_f16(kTM, D, false, true) : umma_idesc_bf16(kTM, D, false, true);
            const uint32_t leader = elect_one();
            // The warp's waits keep the default limit, which compiles to the plain wait; when
            // another role's wait runs out, the abort flag ends these.
            auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(bar, phase, abort_flag));
            };
            // (a descriptor holds 18 bits of an address; in a cluster there is the CTA's rank above them)
            auto address = [](const void *x) -> uint32_t { return (smem_u32(x) & 0x3ffffu) >> 4; };
            const uint32_t q_addr = address(q_s), k_addr = address(k_ring), v_addr = address(v_ring);
            const uint64_t kd = umma_desc_sw128(0, 16, 1024), vd = umma_desc_sw128(0, 2048, 1024);
            const uint32_t k_hi = (uint32_t)(kd >> 32), k_lo = (uint32_t)kd, v_hi = (uint32_t)(vd >> 32), v_lo = (uint32_t)vd;
            // S = Q_t K^T of the K in a ring slot, then the commit that hands it on; it
            // covers the product issued before it, too
            auto issue_s = [&](int t, int slot) {
                constexpr int STEPS = D / 16;
                uint32_t qa[STEPS], kb[STEPS];
#pragma unroll
                for (int k = 0; k < STEPS; ++k) {
                    qa[k] = k_lo | (q_addr + (t * kQTile + (k / 4) * kQPanel + (k % 4) * 32) / 16);
                    kb[k] = k_lo | (k_addr + (slot * kSlotBytes + (k / 4) * kKVPanel + (k % 4) * 32) / 16);
                }
                mma_ss<STEPS>(leader, tmem + t * kTileCols, k_hi, qa, kb, idesc_s);
                commit_one(leader, &s_full[t]);
            };
            // O_t += P_t V: A = P (TMEM), B = V (MN-major: 16-key group k at k * kVGroup)
            auto issue_o = [&](int t, int slot, bool accumulate) {
                uint32_t vb[kTN / 16];
#pragma unroll
                for (int k = 0; k < kTN / 16; ++k) vb[k] = v_lo | (v_addr + (slot * kSlotBytes + k * kVGroup) / 16);
                mma_ts<kTN / 16>(leader, tmem + t * kTileCols + kOCol, tmem + t * kTileCols, v_hi, vb, idesc_o,
                                 accumulate ? 1u : 0u);
            };
            // The tile at hand is the last of its unit's when left is 1.  The S of the next tile
            // goes out behind each P V; at a unit's end it waits for the next unit's Q, so both
            // P V go first.
            int ks = 0, vs = 0;                   // ring slots of the tile's K and V, and their phases
            uint32_t k_phase = 0, v_phase = 0, phase = 0;
            bool ok = wait(q_full, 0) && wait(&k_full[0], 0);
            int units = 0, n_kt = 1, left = 1;
            bool last_unit = true;
            auto read_unit = [&]() {
                const volatile Unit &w = unit_s[units & 3];
                n_kt = left = w.n_kt;
                last_unit = w.last;
            };
            if (ok) {
                read_unit();
                tc_fence_after();
#pragma unroll 1
                for (int t = 0; t < kNQ; ++t) issue_s(t, 0);
                commit_one(leader, &k_empty[0]);
                if (n_kt == 1) commit_one(leader, q_empty);
            }
            while (ok) {
                const bool first = left == n_kt, last = left == 1;
                if (++ks == NK) {
                    ks = 0;
                    k_phase ^= 1;
                }
                ok = wait(&v_full[vs], v_phase);
#pragma unroll
                for (int t = 0; t < kNQ; ++t) {
                    if (!ok) break;
                    ok = wait(&p_full[t], phase);
                    if (!ok) break;
                    tc_fence_after();
                    issue_o(t, vs, !first);
                    if (last) {
                        commit_one(leader, &o_done[t]);
                    } else {
                        if (t == 0) {
                            ok = wait(&k_full[ks], k_phase);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        issue_s(t, ks);
                    }
                }
                if (!ok) break;
                commit_one(leader, &v_empty[vs]);
                if (last) {
                    if (last_unit) break;
                    ++units;
                    ok = wait(&k_full[ks], k_phase) && wait(q_full, units & 1);
                    if (!ok) break;
                    read_unit();
                    tc_fence_after();
                    // (S_t's columns hold a P that the tensor core reads before)
#pragma unroll 1
                    for (int t = 0; t < kNQ; ++t) issue_s(t, ks);
                    ++left;
                }
                commit_one(leader, &k_empty[ks]);
                if (--left == 1) commit_one(leader, q_empty);   // S of the unit's last tile is issued
                phase ^= 1;
                if (++vs == NV) {
                    vs = 0;
                    v_phase ^= 1;
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsSoftmax) : "memory");
        // ===================== softmax warpgroups: row r = TMEM lane r =====================
        const int qt = warp / 4;
        const int r = threadIdx.x % kTM;
        const uint32_t lane_base = tmem + ((uint32_t)((warp % 4) * 32) << 16) + qt * kTileCols;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        // (the unit stays in shared memory: a row's scores need the registers)
        int c = 0;                               // tiles so far
        bool ok = true, more = any;
        // V rows of the last group that lie behind the run's last key may hold anything: they
        // are zeroed once V has landed (both warpgroups write the same zeros).
        auto clean_v = [&](int from) -> bool {
            if (!__all_sync(0xffffffffu, wait_for(&v_full[c % NV], (c / NV) & 1, abort_flag, p.wait_ns))) return false;
            uint8_t *vs = v_ring + (c % NV) * kSlotBytes;
            for (int i = r; i < (((from + 15) & ~15) - from) * PANELS * 8; i += kTM) {
                const int row = from + i / (PANELS * 8), pc = i % (PANELS * 8);
                *reinterpret_cast<uint4 *>(vs + (row / 16) * kVGroup + (pc / 8) * 2048 + swz128(row % 16, pc % 8)) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();   // zeroed V rows visible to the tensor core
            return true;
        };
        for (int units = 0; more; ++units) {
            const volatile Unit &w = unit_s[units & 3];
            int n_kt = 1;                        // read with the unit's first tile
            bool live = false, warp_live = false;
            int32_t pos = 0;
            float m = -INFINITY, l = 0.f;
            int exponent = 0;                    // int8: O is in units of 2^exponent
            for (int j = 0; j < n_kt; ++j, ++c) {
                ok = __all_sync(0xffffffffu, wait_for(&s_full[qt], c & 1, abort_flag, p.wait_ns));
                if (!ok) break;
                tc_fence_after();
                // (the first S of a unit says that the unit has been written)
                if (j == 0) {
                    n_kt = w.n_kt;
                    more = !w.last;
                    pos = w.pos + qt * pos_per_tile + r / G;
                    // (every live row sees all keys of the run: a masked score would leave 0 times a
                    // value, and over int8 pages its scale, in the row's sums)
                    live = r < pos_per_tile * G && pos < w.pos_end;
                    if (live && p.ctx_lens) live = __ldcg(p.ctx_lens + pos) >= w.len;
                    warp_live = __any_sync(0xffffffffu, live);
                }
                const int32_t key0 = (w.t0 + j) * kTN, tail = w.len - key0;
                if constexpr (INT8) {
                    ok = __all_sync(0xffffffffu, wait_for(&sc_full[c % kScaleTiles], (c / kScaleTiles) & 1, abort_flag, p.wait_ns));
                    if (!ok) break;
                }
                if (warp_live) {                 // (others leave P as it is: their rows go nowhere)
                    uint32_t sv[kTN];
#pragma unroll
                    for (int i = 0; i < kTN / 32; ++i) tmem_ld32_async(lane_base + i * 32, sv + i * 32);
                    tmem_wait_ld();
                    if constexpr (INT8) {        // scores of codes times the keys' scales
                        const float *sc = scale_s + (c % kScaleTiles) * 2 * kTN;
#pragma unroll
                        for (int i = 0; i < kTN; i += 4) {
                            const float4 k = *reinterpret_cast<const float4 *>(sc + i);
                            const float2 a = __fmul2_rn(make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), make_float2(k.x, k.y));
                            const float2 b = __fmul2_rn(make_float2(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])), make_float2(k.z, k.w));
                            sv[i] = __float_as_uint(a.x);
                            sv[i + 1] = __float_as_uint(a.y);
                            sv[i + 2] = __float_as_uint(b.x);
                            sv[i + 3] = __float_as_uint(b.y);
                        }
                    }
                    if (tail < kTN) {            // the run ends in this tile
#pragma unroll
                        for (int i0 = 0; i0 < kTN; i0 += 32) {
                            const uint32_t seen = bits_below(tail - i0);
                            if (seen == 0xffffffffu) continue;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((seen >> i) & 1)) sv[i0 + i] = __float_as_uint(-INFINITY);
                        }
                    }
                    const float alpha = move_maximum(m, largest(sv) * p.scale_log2);
                    float alpha_o = alpha;
                    if constexpr (INT8) {
                        const int e = value_exponent(scale_s + (c % kScaleTiles) * 2 * kTN + kTN), old = exponent;
                        exponent = j == 0 ? e : max(old, e);
                        if (j > 0) alpha_o *= power_of_two(old - exponent);
                    }
                    // O row rescale (rare): O holds P V up to tile j - 1, complete since this S's
                    // commit came after it
                    if (__any_sync(0xffffffffu, alpha_o != 1.f) && j > 0) rescale_o<D>(lane_base + kOCol, alpha_o);
                    // P (bf16 pairs) over S's first 64 columns, each 16-column store after the S
                    // columns it covers were read
                    // (fp16: 2^kUp times them, so that the largest is below 2^15 and what is below
                    // fp16's range is below 2^-31 of it)
                    const float up = INT8 ? kUp - m : -m;
                    const float2 nm2 = m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(up, up);
                    const float l0 = probabilities64<0, INT8>(sv, sc2, nm2, lane_base);
                    const float l1 = probabilities64<64, INT8>(sv, sc2, nm2, lane_base + 32);
                    l = l * alpha + (l0 + l1);
                    tmem_wait_st();
                }
                if (!INT8 && tail < kTN && (tail & 15) != 0) {   // (int8: their scales are 0)
                    ok = clean_v(tail);
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
            // row r of O.  (O is read before this warp's next P is handed over, and the next
            // unit's first product into O comes after that.)
            const float unit_o = INT8 ? power_of_two(exponent) : 1.f;
            if (INT8) m -= kUp;
            if (warp_live) {
                const int64_t row = (int64_t)pos * p.n_q_heads + w.kvh * G + r % G;
                const bool whole = !p.ctx_lens && !w.cut;
                if (whole) {
                    const float inv = l == 0.f ? 0.f : unit_o / l;      // (a NaN stays one)
                    __nv_bfloat16 *out = p.out + row * D;
#pragma unroll 1
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t v[32];
                        tmem_ld32_async(lane_base + kOCol + i * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int q2 = 0; q2 < 2; ++q2) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                x[e] = pack_bf16x2(__uint_as_float(v[16 * q2 + 2 * e]) * inv, __uint_as_float(v[16 * q2 + 2 * e + 1]) * inv);
                            if (!live) continue;
                            if (p.wide_out) {
                                st_global_32(out + i * 32 + q2 * 16, x);
                            } else {
                                *reinterpret_cast<uint4 *>(out + i * 32 + q2 * 16) = make_uint4(x[0], x[1], x[2], x[3]);
                                *reinterpret_cast<uint4 *>(out + i * 32 + q2 * 16 + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                            }
                        }
                    }
                    if (live && p.lse_out) p.lse_out[row] = (m + __log2f(l)) * 0.69314718055994531f;
                } else {
                    const bool begins = w.t0 == 0;
                    const int64_t mine = (int64_t)blockIdx.x * kUnitRows + qt * kTM + r;
                    const int64_t rows = (int64_t)p.n_rows * G;
                    const int64_t step = begins ? rows * 8 : kUnitRows * 8;              // to a row's next 8 values
                    float *dst = begins ? p.part.first + (w.kvh * (D / 8) * rows + (int64_t)pos * G + r % G) * 8
                                        : p.part.cont + ((int64_t)blockIdx.x * (D / 8) * kUnitRows + qt * kTM + r) * 8;
#pragma unroll 1
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t v[32];
                        tmem_ld32_async(lane_base + kOCol + i * 32, v);
                        tmem_wait_ld();
                        if (!live) continue;
#pragma unroll
                        for (int q2 = 0; q2 < 4; ++q2) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = INT8 ? __float_as_uint(__uint_as_float(v[8 * q2 + e]) * unit_o) : v[8 * q2 + e];
                            st_global_32(dst + (i * 4 + q2) * step, x);
                        }
                    }
                    if (live && begins)
                        p.part.stat[row] = make_float4(m, l, __int_as_float((int)blockIdx.x), __int_as_float(w.last_cta));
                    else if (live)
                        p.part.cont_ml[mine] = make_float2(m, l);
                }
            }
            tc_fence_before();
        }
        if (!ok) {
            if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    }
    // everyone meets here before the TMEM is released
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) p.part.cuts[blockIdx.x] = cut_s;
    // (unequal without a wait that ran out: lengths that changed while the two read them)
    if ((*abort_flag || issued_s[0] != issued_s[1]) && (warp == 8 || warp == 10) && lane == 0)
        settle_pair(issued_s[warp == 10], issued_s[warp != 10], k_codes, NK);
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---- joins: a thread to 16 columns of a row, neighbouring rows to neighbouring threads --------

constexpr int kCols = 16;

struct Joined {
    float m, l, o[kCols];
};

__device__ __forceinline__ void load8(float *x, const float *src)
{
    const float4 a = __ldcg(reinterpret_cast<const float4 *>(src)), b = __ldcg(reinterpret_cast<const float4 *>(src) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Joins a piece (maximum xm, sum xl, x) to what was joined before it.  One without a
// maximum has seen nothing.
__device__ __forceinline__ void join_piece(Joined &j, float xm, float xl, const float (&x)[kCols])
{
    const float top = fmaxf(j.m, xm);
    const float a = j.m == -INFINITY ? 0.f : fast_exp2(j.m - top), b = xm == -INFINITY ? 0.f : fast_exp2(xm - top);
    j.m = top;
    j.l = j.l * a + xl * b;
#pragma unroll
    for (int e = 0; e < kCols; ++e) j.o[e] = j.o[e] * a + x[e] * b;
}

// Columns kCols part .. of the first piece of row i = pos * G + g of a kv head.
template <int D>
__device__ __forceinline__ void load_first(const RowsParams &p, int32_t kvh, int64_t i, int part, float (&x)[kCols])
{
    const int64_t rows = (int64_t)p.n_rows * p.group;
#pragma unroll
    for (int k = 0; k < kCols / 8; ++k) load8(x + 8 * k, p.part.first + ((kvh * (D / 8) + kCols / 8 * part + k) * rows + i) * 8);
}

// The pieces that CTAs c0 .. c1 have of a unit's row `place`.
template <int D>
__device__ __forceinline__ void join_pieces(const RowsParams &p, Joined &j, int32_t c0, int32_t c1, int place, int part)
{
    constexpr int kRound = 4;                       // pieces in flight
    // (within the workspace whatever a rows kernel that ran out of time has left there)
    c0 = max(c0, 0);
    c1 = min(c1, kMaxCtas - 1);
    for (; c0 <= c1; c0 += kRound) {
        float2 ml[kRound];
        float x[kRound][kCols];
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
            if (c0 + i > c1) break;
            ml[i] = __ldcg(p.part.cont_ml + (int64_t)(c0 + i) * kUnitRows + place);
#pragma unroll
            for (int k = 0; k < kCols / 8; ++k)
                load8(x[i] + 8 * k, p.part.cont + (((int64_t)(c0 + i) * (D / 8) + kCols / 8 * part + k) * kUnitRows + place) * 8);
        }
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
            if (c0 + i > c1) break;
            join_piece(j, ml[i].x, ml[i].y, x[i]);
        }
    }
}

// The columns of a row, o / l rounded once, and its log-sum-exp; no key seen: 0 and -inf.  (A sum
// that is no number, from a NaN or an infinity among what the row sees, passes on to both.)
template <int D>
__device__ __forceinline__ void write_joined(const RowsParams &p, const Joined &j, int64_t row, int part)
{
    const float inv = j.l == 0.f ? 0.f : 1.f / j.l;
    uint4 *out = reinterpret_cast<uint4 *>(p.out + row * D + kCols * part);
#pragma unroll
    for (int k = 0; k < kCols / 8; ++k)
        out[k] = make_uint4(pack_bf16x2(j.o[8 * k] * inv, j.o[8 * k + 1] * inv), pack_bf16x2(j.o[8 * k + 2] * inv, j.o[8 * k + 3] * inv),
                            pack_bf16x2(j.o[8 * k + 4] * inv, j.o[8 * k + 5] * inv), pack_bf16x2(j.o[8 * k + 6] * inv, j.o[8 * k + 7] * inv));
    if (part == 0 && p.lse_out) p.lse_out[row] = j.l == 0.f ? -INFINITY : (j.m + __log2f(j.l)) * 0.69314718055994531f;
}

// A cross attention: the cut unit that begins in CTA blockIdx.x; the last blockIdx.y writes the
// rows of empty runs.
template <int D>
__global__ void __launch_bounds__(kTM) rows_join_kernel(const __grid_constant__ RowsParams p)
{
    grid_dependents_launch();
    grid_dependency_wait();
    if (blockIdx.y == gridDim.y - 1) {
        for (int32_t g = (int32_t)blockIdx.x; g < p.n_runs; g += (int32_t)gridDim.x) {
            const Run run = run_of_params(p, g);
            if (run.len > 0) continue;
            const int64_t row0 = (int64_t)run.row0 * p.n_q_heads, rows = (int64_t)run.rows * p.n_q_heads;
            for (int64_t i = threadIdx.x; i < rows * (D / 8); i += blockDim.x)
                reinterpret_cast<uint4 *>(p.out + row0 * D)[i] = make_uint4(0, 0, 0, 0);
            if (p.lse_out)
                for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) p.lse_out[row0 + i] = -INFINITY;
        }
        return;
    }
    const int4 c = __ldcg(reinterpret_cast<const int4 *>(p.part.cuts + blockIdx.x));
    const CutUnit u{c.x, c.y, c.z, c.w};
    if (u.last_cta == 0) return;
    const int part = (int)blockIdx.y % (D / kCols), qt = (int)blockIdx.y / (D / kCols), r = threadIdx.x;
    const int G = p.group, tile = kTM / G;
    const int32_t pos = u.pos + qt * tile + r / G, head = u.kvh * G + r % G;
    if (r >= tile * G || pos >= u.pos_end) return;
    const int64_t row = (int64_t)pos * p.n_q_heads + head;
    const float4 stat = __ldcg(p.part.stat + row);
    Joined j;
    j.m = stat.x;
    j.l = stat.y;
    load_first<D>(p, u.kvh, (int64_t)pos * G + r % G, part, j.o);
    join_pieces<D>(p, j, (int32_t)blockIdx.x + 1, u.last_cta, qt * kTM + r, part);
    write_joined<D>(p, j, row, part);
}

// A decode: rows 128 blockIdx.x .. of the sequences' query heads of kv head blockIdx.y.
template <int D>
__global__ void __launch_bounds__(kTM) shared_join_kernel(const __grid_constant__ RowsParams p)
{
    grid_dependents_launch();
    grid_dependency_wait();
    const int part = (int)blockIdx.z, G = p.group;
    const int64_t i = (int64_t)blockIdx.x * kTM + threadIdx.x;
    if (i >= (int64_t)p.n_rows * G) return;
    const int32_t kvh = (int32_t)blockIdx.y, pos = (int32_t)(i / G), g = (int32_t)(i - (int64_t)pos * G);
    const int64_t row = (int64_t)pos * p.n_q_heads + kvh * G + g;
    const float4 own = __ldcg(p.part.own_stat + row), stat = __ldcg(p.part.stat + row);   // (stat: of this call where `place` says so)
    Joined j;
    float x[kCols];
    j.m = own.x;
    j.l = own.y;
#pragma unroll
    for (int k = 0; k < kCols / 8; ++k) load8(j.o + 8 * k, p.part.own + row * D + kCols * part + 8 * k);
    const int place = __float_as_int(own.z);
    if (place == kDone) return;
    if (place >= 0) {
        load_first<D>(p, kvh, i, part, x);
        join_piece(j, stat.x, stat.y, x);
        join_pieces<D>(p, j, __float_as_int(stat.z) + 1, __float_as_int(stat.w), place + g, part);
    }
    write_joined<D>(p, j, row, part);
}

// What 128 of a decode's own tokens cost an SM, in tiles of a run: the share of the SMs that
// the runs' tiles get.  Measured (weights 0.4 / 0.6 / 0.8 / 1.0 / 1.3): bf16 pages, 64
// sequences of 16 to 512 own tokens behind 4096 35.8 / 33.2 / 32.9 / 34.1 / 36.9 us, of 1000
// to 2000 80.3 / 79.0 / 77.4 / 97.9 / 97.4, 128 in four groups behind 1000 to 3000 51.8 / 49.9
// / 49.7 / 48.2 / 51.8; int8 pages (whose runs' tiles take longer), 96 sequences in two groups
// 56.6 / 59.7 / 64.7 / 70.1 / 77.5.
constexpr float kRestWeight = 0.85f, kRestWeightInt8 = 0.4f;

RowsParams params_of(const RowsArgs &a, int num_sms)
{
    const pkv_dims &d = a.dims;
    RowsParams p{};
    p.n_q_heads = a.n_q_heads;
    p.group = a.n_q_heads / d.n_kv_heads;
    p.n_rows = a.n_rows;
    p.n_kv_heads = d.n_kv_heads;
    p.n_blocks = d.n_blocks;
    p.block_size = d.block_size;
    p.pool_rows = (d.n_blocks + 1) * d.block_size;
    p.starts = a.starts;
    p.run_tables = a.run_tables;
    p.run_lens = a.run_lens;
    p.n_runs = a.n_runs;
    p.max_run_blocks = a.max_run_blocks;
    p.ctx_lens = a.ctx_lens;
    p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse_out = a.lse_out;
    p.part = a.partials;
    p.k_scales = a.k_scales;
    p.v_scales = a.v_scales;
    p.dev_status = a.dev_status;
    p.wide_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    p.sms = num_sms;
    p.few = a.few;
    p.rest_weight = a.kv_dtype == PKV_KV_INT8 ? kRestWeightInt8 : kRestWeight;
    p.wait_ns = pipeline_wait_ns();
    return p;
}

cudaLaunchConfig_t dependent(cudaLaunchAttribute (&pdl)[1], unsigned grid, unsigned threads, size_t smem, cudaStream_t stream)
{
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    lc.attrs = pdl;
    lc.numAttrs = 1;
    return lc;
}

// CTAs that the runs' tiles may be shared out to: one per SM, and no more than there can be tiles.
unsigned most_shares(const RowsArgs &a, int num_sms)
{
    const int64_t positions = kNQ * (kTM / (a.n_q_heads / a.dims.n_kv_heads));
    const int64_t units = ((int64_t)a.n_rows / positions + a.n_runs) * a.dims.n_kv_heads;
    const int64_t tiles = units * (((int64_t)a.max_run_blocks * a.dims.block_size + kTN - 1) / kTN);
    int64_t n = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    if (tiles < n) n = tiles;
    return (unsigned)(n < 1 ? 1 : n);
}

template <int D, bool INT8>
cudaError_t launch_as(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap, const RowsParams &p, unsigned grid,
                      cudaStream_t stream)
{
    using S = Setup<D, INT8>;
    // The register split assumes the block gets kLaunchRegs per thread: refuse
    // a build whose kernel was given fewer (its setmaxnreg.inc could not complete).
    static const bool regs_ok = [] {
        cudaFuncAttributes fa{};
        return cudaFuncGetAttributes(&fa, rows_kernel<D, INT8>) == cudaSuccess && fa.numRegs >= S::kLaunchRegs;
    }();
    if (!regs_ok) return cudaErrorInvalidConfiguration;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(rows_kernel<D, INT8>), S::kThreads, S::kSmem, nullptr);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t lc = dependent(reinterpret_cast<cudaLaunchAttribute(&)[1]>(at), grid, S::kThreads, S::kSmem, stream);
    // A decode's own tokens run beside this kernel.  The two SMs of a TPC share their way to
    // memory, and a CTA whose neighbour streams own tokens takes up to 1.4 times as long; as
    // clusters of two, which lie on one TPC, the CTAs with a share have each other for
    // neighbours (256 sequences in six groups: the last CTA done after 120 us, not 163).
    if (p.ctx_lens && grid % 2 == 0) {
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = 2;
        at[1].val.clusterDim.y = 1;
        at[1].val.clusterDim.z = 1;
        // (all of them have to be resident at once, as the shares are dealt out to all)
        static std::atomic<int> pairs[kDevices];     // + 1; 0: not asked yet
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        int n = dev < kDevices ? pairs[dev].load() - 1 : -1;
        if (n < 0) {
            cudaLaunchConfig_t ask = lc;
            ask.attrs = at + 1;
            e = cudaOccupancyMaxActiveClusters(&n, rows_kernel<D, INT8>, &ask);
            if (e != cudaSuccess) return e;
            if (dev < kDevices) pairs[dev] = n + 1;
        }
        if (n >= (int)grid / 2) lc.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&lc, rows_kernel<D, INT8>, qmap, kmap, vmap, p);
}

}  // namespace

cudaError_t launch_rows_tc(const RowsArgs &a, int num_sms, cudaStream_t stream)
{
    const pkv_dims &d = a.dims;
    const RowsParams p = params_of(a, num_sms);
    CUtensorMap qmap, kmap, vmap;
    {
        const uint64_t dims[3] = {(uint64_t)d.head_dim, (uint64_t)a.n_q_heads, (uint64_t)a.n_rows};
        const uint64_t strides[2] = {(uint64_t)d.head_dim * 2, (uint64_t)a.q_stride * 2};
        const uint32_t box[3] = {64u, (uint32_t)p.group, (uint32_t)(kTM / p.group)};
        if (encode_tensor_map(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const uint64_t rows = (uint64_t)(d.n_blocks + 1) * d.block_size;
    const bool int8 = a.kv_dtype == PKV_KV_INT8;
    const uint64_t row_bytes = (uint64_t)d.n_kv_heads * d.head_dim * (int8 ? 1 : 2);
    if (int8) {
        // {codes of a row, kv head, pool row}: 16 rows of one head lie behind one another
        const uint64_t dims[3] = {(uint64_t)d.head_dim, (uint64_t)d.n_kv_heads, rows};
        const uint64_t strides[2] = {(uint64_t)d.head_dim, row_bytes};
        const uint32_t box[3] = {(uint32_t)d.head_dim, 1u, 16u};
        if (encode_tensor_map(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(a.k_pool), dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
            encode_tensor_map(&vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(a.v_pool), dims, strides,
                              box, CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    } else {
        // K: {64 columns, kv head, pool row}, one head and 16 rows per box
        const uint64_t kdims[3] = {(uint64_t)d.head_dim, (uint64_t)d.n_kv_heads, rows};
        const uint64_t kstrides[2] = {(uint64_t)d.head_dim * 2, row_bytes};
        const uint32_t kbox[3] = {64u, 1u, 16u};
        // V: {64 columns, pool row, 64-column panel of all heads}: a box of 16
        // rows and a head's panels lands as [panel][row][128 B]
        const uint32_t panels = (uint32_t)d.head_dim / 64u;
        const uint64_t vdims[3] = {64u, rows, (uint64_t)d.n_kv_heads * panels};
        const uint64_t vstrides[2] = {row_bytes, 128u};
        const uint32_t vbox[3] = {64u, 16u, panels};
        if (encode_tensor_map(&kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.k_pool), kdims, kstrides,
                              kbox, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
            encode_tensor_map(&vmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.v_pool), vdims, vstrides,
                              vbox, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const unsigned grid = most_shares(a, num_sms);
    if (d.head_dim == 128)
        return int8 ? launch_as<128, true>(qmap, kmap, vmap, p, grid, stream) : launch_as<128, false>(qmap, kmap, vmap, p, grid, stream);
    return int8 ? launch_as<64, true>(qmap, kmap, vmap, p, grid, stream) : launch_as<64, false>(qmap, kmap, vmap, p, grid, stream);
}

cudaError_t launch_rows_join(const RowsArgs &a, int num_sms, cudaStream_t stream)
{
    const RowsParams p = params_of(a, num_sms);
    cudaLaunchAttribute pdl[1];
    if (a.ctx_lens) {
        const int64_t grid = ((int64_t)a.n_rows * p.group + kTM - 1) / kTM;
        cudaLaunchConfig_t lc = dependent(pdl, (unsigned)grid, kTM, 0, stream);
        lc.gridDim.y = (unsigned)a.dims.n_kv_heads;
        lc.gridDim.z = (unsigned)a.dims.head_dim / kCols;
        return a.dims.head_dim == 128 ? cudaLaunchKernelEx(&lc, shared_join_kernel<128>, p)
                                      : cudaLaunchKernelEx(&lc, shared_join_kernel<64>, p);
    }
    cudaLaunchConfig_t lc = dependent(pdl, most_shares(a, num_sms), kTM, 0, stream);
    lc.gridDim.y = kNQ * (unsigned)a.dims.head_dim / kCols + 1;
    return a.dims.head_dim == 128 ? cudaLaunchKernelEx(&lc, rows_join_kernel<128>, p) : cudaLaunchKernelEx(&lc, rows_join_kernel<64>, p);
}

}  // namespace pkv
