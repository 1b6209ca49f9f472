// softmax_tc.cuh -- what the attention kernels with P in TMEM share (prefill_window.cu,
// rows_tc.cu): products issued by one lane of a converged warp, the pipeline wait, and a
// row's maximum, probabilities and rescale.
#pragma once

#include <math.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace pkv {

constexpr float kRescaleThreshold = 8.0f;  // log2 units

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

// After a wait that ran out: the copies of two warps that fill a ring of K, half a slot each
// (full[] counts both arrivals), have landed when this returns; asked by a lane of each, behind a
// barrier of the CTA that both came to, with the tiles that it has issued and the other one has.
// Where one of them left early, it has not arrived at slots that the other one's copies are on
// their way into, and a wait for those would run its 4 s for each of them.  So whoever is ahead,
// by the ring at most, arrives there in its place.  (A slot's copies wait for its last use, which
// waited for both arrivals, so that each of these slots is in the phase that only that arrival is
// missing from; and what is further back than the ring, seen from whoever is ahead, has landed.)
static __device__ __noinline__ void settle_pair(int issued, int other, uint64_t *full, int slots)
{
    const int ahead = max(issued, other);
#pragma unroll 1
    for (int i = other; i < issued; ++i) mbar_arrive(&full[i % slots]);
#pragma unroll 1
    for (int i = max(ahead - slots, 0); i < issued; ++i) (void)mbar_wait(&full[i % slots], (i / slots) & 1);
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
// arguments), as bf16 (or fp16) pairs into 32 TMEM columns from taddr on; their sum.
template <int I0, bool F16 = false, int NC>
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
            pk[e] = F16 ? pack_f16x2(ee.x, ee.y) : pack_bf16x2(ee.x, ee.y);
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

}  // namespace pkv
