// rope.cuh -- rotary positions as device functions, shared by the rotary page
// write and the windowed decode step.
//
// Angles.  A pair's phase is its turns per position in units of 2^-64, so the
// angle of position t is (t * phase mod 2^64) 2^-64 turns: an integer product,
// exact for every position, where the binary32 product t * f loses 0.06 rad at
// t = 10^6.
//
// Lanes.  A head row of D elements is the work of D / 16 lanes: lane `slot`
// holds two 16-byte vectors (16 elements, 8 pairs) so that both members of
// every pair are in one lane, in either layout; the 8 sines and cosines depend
// on the slot and the position alone and serve every head of a token.
#pragma once

#include "common.cuh"

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

// Vectors (of 8 elements) of a head row that lane `slot` of its D / 16 holds,
// and whether they are turned.  Half layout: the pair (slot, slot + rot / 16)
// of the turned part, then neighbours of the rest; interleaved: neighbours.
__device__ __forceinline__ bool rope_vectors(const RopeArgs &r, int slot, int &v0, int &v1)
{
    const int turned = r.phases ? r.rot_dim / 16 : 0;   // slots that hold turned pairs
    const bool turn = slot < turned;
    if (turn && !r.interleaved) {
        v0 = slot;
        v1 = slot + turned;
    } else {
        v0 = 2 * slot;
        v1 = v0 + 1;
    }
    return turn;
}

// The cosine and sine (times the magnitude) of a phase at position t, rounded
// once.  The nearest quarter turn is taken off in integers, which leaves an angle
// th + tl of at most an eighth of a turn, held to twice binary32; sine and cosine
// are their Taylor series there (the first terms left out are below 1e-11 and
// 2e-10), summed with the largest term last and apart:
//   sin = th + (tl (1 - u / 2) + th u (-1/6 + u / 5! - ...)),  u = th^2
//   cos = (1 - u / 2) + ((rest of that difference) - ue / 2 + u^2 (1/4! - ...)).
// Both are within 0.73 steps of the last place of the exact value (0.29 on
// average, as rounding the exact one would be); a sine and cosine of the angle in
// binary32 are not, and the keys they turn would be rounded to another bf16 twice
// as often.
__device__ __forceinline__ void rope_angle_of(const RopeArgs &r, unsigned long long phase, int64_t t, float &c, float &s)
{
    const unsigned long long a = phase * (unsigned long long)t;           // turns * 2^64
    const uint32_t q = (uint32_t)((a + (1ull << 61)) >> 62) & 3u;          // the nearest quarter turn
    const int32_t rest = (int32_t)((int64_t)(a - ((unsigned long long)q << 62)) >> 30);   // turns * 2^34
    // times pi 2^-33, in two parts
    constexpr float kPi = (float)(3.14159265358979323846 / 8589934592.0);
    constexpr float kPiLow = (float)(3.14159265358979323846 / 8589934592.0 - (double)kPi);
    const float x = (float)rest, xl = (float)(rest - __float2int_rn(x));
    const float th = __fmul_rn(x, kPi);
    const float tl = __fadd_rn(__fmaf_rn(x, kPi, -th), __fmaf_rn(x, kPiLow, __fmul_rn(xl, kPi)));
    const float u = __fmul_rn(th, th), ue = __fmaf_rn(2.f * th, tl, __fmaf_rn(th, th, -u));
    float ps = __fmaf_rn(u, -1.f / 39916800.f, 1.f / 362880.f);
    ps = __fmaf_rn(u, ps, -1.f / 5040.f);
    ps = __fmaf_rn(u, ps, 1.f / 120.f);
    ps = __fmaf_rn(u, ps, -1.f / 6.f);
    const float sin_low = __fmaf_rn(__fmul_rn(th, u), ps, __fmaf_rn(-0.5f * u, tl, tl));
    float pc = __fmaf_rn(u, -1.f / 3628800.f, 1.f / 40320.f);
    pc = __fmaf_rn(u, pc, -1.f / 720.f);
    pc = __fmaf_rn(u, pc, 1.f / 24.f);
    const float cos_high = __fsub_rn(1.f, 0.5f * u);
    const float cos_low = __fmaf_rn(__fmul_rn(u, u), pc, __fmaf_rn(-0.5f, ue, __fsub_rn(__fsub_rn(1.f, cos_high), 0.5f * u)));
    // times the magnitude, then to their quarter
    auto scaled = [&](float high, float low) {
        const float h = __fmul_rn(high, r.mag_high);
        return __fadd_rn(h, __fmaf_rn(low, r.mag_high, __fmaf_rn(high, r.mag_low, __fmaf_rn(high, r.mag_high, -h))));
    };
    const float y = scaled(th, sin_low), z = scaled(cos_high, cos_low);
    const float cq = q & 1 ? y : z, sq = q & 1 ? z : y;
    c = q == 1 || q == 2 ? -cq : cq;
    s = q >= 2 ? -sq : sq;
}

// Those of pair i.
__device__ __forceinline__ void rope_angle(const RopeArgs &r, int i, int64_t t, float &c, float &s)
{
    rope_angle_of(r, __ldg(reinterpret_cast<const unsigned long long *>(r.phases) + i), t, c, s);
}

// Those of pairs 8 slot .. 8 slot + 7.  phases is 16-byte aligned.
__device__ __forceinline__ void rope_angles(const RopeArgs &r, int slot, int64_t t, float (&c)[8], float (&s)[8])
{
    const ulonglong2 *ph = reinterpret_cast<const ulonglong2 *>(r.phases + 8 * slot);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 p = __ldg(ph + i);
        rope_angle_of(r, p.x, t, c[2 * i], s[2 * i]);
        rope_angle_of(r, p.y, t, c[2 * i + 1], s[2 * i + 1]);
    }
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 &raw, float *x)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float *x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Turns the 8 pairs of a lane's 16 elements (x[0..7] of its first vector,
// x[8..15] of its second).  The operations are spelled out so that every kernel
// gives the same bits.
__device__ __forceinline__ void rope_turn(bool interleaved, const float (&c)[8], const float (&s)[8], float (&x)[16])
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fmaf_rn(a, c[i], -__fmul_rn(b, s[i]));
            x[2 * i + 1] = __fmaf_rn(b, c[i], __fmul_rn(a, s[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = x[i + 8];
            x[i] = __fmaf_rn(a, c[i], -__fmul_rn(b, s[i]));
            x[i + 8] = __fmaf_rn(b, c[i], __fmul_rn(a, s[i]));
        }
    }
}

// The scale amax / 127 (correctly rounded) and the codes clamp(rint(fl(x / scale)),
// -127, 127) of a lane's 16 elements of a row of absolute maximum amax, four codes
// to a word; amax 0 gives scale and codes 0.
//
// With rcp = fl(1 / scale), q = fl(x rcp) is within 1.6e-5 of x / scale
// (|x / scale| < 128), whose own rounding is below 4e-6.  Added to 1.5 * 2^23, q is
// rounded to an integer, ties to even, which stands in the sum's low byte; where it
// is nearer than 3e-5 to a half, and where it is no number, the division decides.
__device__ __forceinline__ float int8_codes16(const float (&x)[16], float amax, uint32_t (&w)[4])
{
    constexpr float kInteger = 12582912.f;
    const float scale = __fdiv_rn(amax, 127.0f);
    const bool normal = scale >= 1.17549435e-38f;      // below, 1 / scale may not be finite
    const float rcp = normal ? __frcp_rn(scale) : 0.f;
    auto is_clear = [&](float q, float t) { return fabsf(__fsub_rn(q, __fsub_rn(t, kInteger))) < 0.5f - 3.0e-5f; };
    bool clear = normal;
    uint32_t c[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float q = __fmul_rn(x[e], rcp), t = __fadd_rn(q, kInteger);
        clear = clear && is_clear(q, t);
        c[e] = __float_as_uint(t);
    }
    if (!clear && amax != 0.f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float q = __fmul_rn(x[e], rcp);
            if (normal && is_clear(q, __uint_as_float(c[e]))) continue;
            c[e] = (uint32_t)max(-127, min(127, __float2int_rn(__fdiv_rn(x[e], scale))));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
        if (amax == 0.f) w[i] = 0;
    }
    return scale;
}

}  // namespace pkv
