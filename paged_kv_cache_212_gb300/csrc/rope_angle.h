// rope_angle.h -- sine and cosine of a rotary angle, for the kernels; host compilers
// take it too (without contraction of products and sums), and tests check its error
// there.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#include <math.h>
#define PKV_HOST_DEVICE inline
#endif

namespace pkv {

struct RopeArgs {
    const uint64_t *phases;   // null: no turn
    int32_t rot_dim;
    int32_t interleaved;
    float mag_high, mag_low;  // the magnitude in two parts
};

inline RopeArgs rope_args(const uint64_t *phases, int32_t rot_dim, int32_t interleaved, double magnitude)
{
    return RopeArgs{phases, rot_dim, interleaved != 0, (float)magnitude, (float)(magnitude - (double)(float)magnitude)};
}

namespace rnd {   // one operation, one rounding

#ifdef __CUDA_ARCH__
__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float sub(float a, float b) { return __fsub_rn(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ float from_int(int32_t i) { return __int2float_rn(i); }
#else
PKV_HOST_DEVICE float mul(float a, float b) { return a * b; }
PKV_HOST_DEVICE float add(float a, float b) { return a + b; }
PKV_HOST_DEVICE float sub(float a, float b) { return a - b; }
PKV_HOST_DEVICE float fma(float a, float b, float c) { return fmaf(a, b, c); }
PKV_HOST_DEVICE float from_int(int32_t i) { return (float)i; }
#endif

}  // namespace rnd

// The cosine and sine (times the magnitude) of a phase at position t.  The nearest
// quarter turn is taken off in integers, which leaves up to an eighth of a turn.  Its
// bits down to 2^-58 turns (2e-17 rad) are held as two floats x + xl, then as an angle
// th + tl in twice binary32.  Sine and cosine are their Taylor series there (the first
// terms left out are below 1e-11 and 2e-10), summed with the largest term last and
// apart:
//   sin = th + (tl (1 - u / 2) + th u (-1/6 + u / 5! - ...)),  u = th^2
//   cos = (1 - u / 2) + ((rest of that difference) - ue / 2 + u^2 (1/4! - ...)).
// Both are within 1.2 steps of the last place of the exact value (measured over 160
// million angles: 0.75 at most, 0.83 with a magnitude that is no power of two, 0.25 on
// average, as rounding the exact one would be off), and next to a quarter turn, nearer
// than 2^-20 turns, within 6 steps (2.8) and 2^-58 turns.  A sine and cosine of the angle in
// binary32 are not as near, and the keys they turn would be rounded to another bf16
// twice as often; an angle cut at 2^-34 turns leaves 1 % off the sine of a pair of 1e-8
// rad a position.
PKV_HOST_DEVICE void rope_angle_of(const RopeArgs &r, unsigned long long phase, int64_t t, float &c, float &s)
{
    const unsigned long long a = phase * (unsigned long long)t;           // turns * 2^64
    const uint32_t q = (uint32_t)((a + (1ull << 61)) >> 62) & 3u;          // the nearest quarter turn
    const int64_t left = (int64_t)(a - ((unsigned long long)q << 62));
    // the nearest multiple of 2^-26 turns, in units of 2^-32, and the 32 bits behind it (signed)
    const float x = rnd::from_int(((int32_t)(left >> 32) + 32) & ~63), xl = rnd::from_int((int32_t)(uint32_t)(left >> 6));
    // times pi 2^-31, in two parts, and pi 2^-57
    constexpr double kPiExact = 3.14159265358979323846 / 2147483648.0;
    constexpr float kPi = (float)kPiExact, kPiLow = (float)(kPiExact - (double)kPi), kPiBehind = kPi / 67108864.f;
    const float th = rnd::mul(x, kPi);
    const float tl = rnd::add(rnd::fma(x, kPi, -th), rnd::fma(x, kPiLow, rnd::mul(xl, kPiBehind)));
    const float u = rnd::mul(th, th), ue = rnd::fma(2.f * th, tl, rnd::fma(th, th, -u));
    float ps = rnd::fma(u, -1.f / 39916800.f, 1.f / 362880.f);
    ps = rnd::fma(u, ps, -1.f / 5040.f);
    ps = rnd::fma(u, ps, 1.f / 120.f);
    ps = rnd::fma(u, ps, -1.f / 6.f);
    const float sin_low = rnd::fma(rnd::mul(th, u), ps, rnd::fma(-0.5f * u, tl, tl));
    float pc = rnd::fma(u, -1.f / 3628800.f, 1.f / 40320.f);
    pc = rnd::fma(u, pc, -1.f / 720.f);
    pc = rnd::fma(u, pc, 1.f / 24.f);
    const float cos_high = rnd::sub(1.f, 0.5f * u);
    const float cos_low = rnd::fma(rnd::mul(u, u), pc, rnd::fma(-0.5f, ue, rnd::sub(rnd::sub(1.f, cos_high), 0.5f * u)));
    // times the magnitude, then to their quarter
    auto scaled = [&](float high, float low) {
        const float h = rnd::mul(high, r.mag_high);
        return rnd::add(h, rnd::fma(low, r.mag_high, rnd::fma(high, r.mag_low, rnd::fma(high, r.mag_high, -h))));
    };
    const float y = scaled(th, sin_low), z = scaled(cos_high, cos_low);
    const float cq = q & 1 ? y : z, sq = q & 1 ? z : y;
    c = q == 1 || q == 2 ? -cq : cq;
    s = q >= 2 ? -sq : sq;
}

}  // namespace pkv
