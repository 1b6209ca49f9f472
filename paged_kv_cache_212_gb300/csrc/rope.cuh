// rope.cuh -- rotary positions as device functions, shared by the rotary page
// write and the windowed decode step.
//
// Angles.  A pair's phase is its turns per position in units of 2^-64, so the
// angle of position t is (t * phase mod 2^64) 2^-64 turns: an integer product,
// exact for every position, where the binary32 product t * f loses 0.06 rad at
// t = 10^6.  rope_angle.h makes sine and cosine of it.
//
// Lanes.  A head row of D elements is the work of D / 16 lanes: lane `slot`
// holds two 16-byte vectors (16 elements, 8 pairs) so that both members of
// every pair are in one lane, in either layout; the 8 sines and cosines depend
// on the slot and the position alone and serve every head of a token.
#pragma once

#include "common.cuh"
#include "rope_angle.h"

namespace pkv {

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

// The cosine and sine (times the magnitude) of pair i at position t.
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
