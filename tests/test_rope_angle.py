"""The kernels' sine and cosine of a rotary angle (csrc/rope_angle.h), compiled for the
host and compared with the exact ones: their error in steps of the last place, for slow
and fast pairs, near and far positions, and angles next to a quarter turn."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_212_gb300", "csrc")

# The exact value to 64 bits or more (long double): the turns are reduced in integers,
# which is exact, to within an eighth of a turn of a multiple of a quarter.
SHIM = r"""
#include "rope_angle.h"
#include <float.h>
static_assert(LDBL_MANT_DIG >= 64, "long double holds more than binary64");
// what the error is above `free`, in steps of the last place of the exact value
static double steps(float got, long double want, long double free)
{
    const long double off = fabsl((long double)got - want) - free;
    if (off <= 0) return 0;
    int e;
    frexpl(fabsl(want), &e);
    return want == 0 ? 1e30 : (double)(off / ldexpl(1, e - 24));
}
extern "C" void angle_errors(const uint64_t *phase, const int64_t *t, long n, double magnitude, double free_turns,
                             double *cos_steps, double *sin_steps, double *from_quarter)
{
    const long double kPi = 3.14159265358979323846264338327950288L;
    const pkv::RopeArgs r = pkv::rope_args(nullptr, 16, 0, magnitude);
    for (long i = 0; i < n; ++i) {
        float c, s;
        pkv::rope_angle_of(r, phase[i], t[i], c, s);
        const uint64_t turns = phase[i] * (uint64_t)t[i];
        int quarter = 0;                    // taken off until the rest is within an eighth of a turn
        int64_t rest = (int64_t)turns;      // half a turn to either side
        for (; rest > (int64_t)1 << 61; rest -= (int64_t)1 << 62) ++quarter;
        for (; rest < -((int64_t)1 << 61); rest += (int64_t)1 << 62) --quarter;
        from_quarter[i] = fabs((double)rest) / 18446744073709551616.0;
        const long double a = rest * (kPi / 9223372036854775808.0L), m = magnitude, off = free_turns * 2 * kPi * m;
        const long double x = cosl(a) * m, y = sinl(a) * m;
        const long double wc[4] = {x, -y, -x, y}, ws[4] = {y, x, -y, -x};
        cos_steps[i] = steps(c, wc[quarter & 3], off);
        sin_steps[i] = steps(s, ws[quarter & 3], off);
    }
}
"""


@pytest.fixture(scope="module")
def angles(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("angle")
    src, lib = str(d / "shim.cpp"), str(d / "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run([cxx, "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).angle_errors

    def call(phase, t, magnitude=1.0):
        phase, t = np.ascontiguousarray(phase, dtype=np.uint64), np.ascontiguousarray(t, dtype=np.int64)
        out = [np.empty(len(t)) for _ in range(3)]
        fn(phase.ctypes.data_as(ctypes.c_void_p), t.ctypes.data_as(ctypes.c_void_p), ctypes.c_long(len(t)),
           ctypes.c_double(magnitude), ctypes.c_double(TURNS), *(x.ctypes.data_as(ctypes.c_void_p) for x in out))
        return out

    return call


TURNS = 2.0 ** -58           # where the angle is cut


def _limit(from_quarter):
    """Steps.  The last addition rounds by half a step.  What it adds to the leading term
    is at most 0.111 of the result (sin, an eighth of a turn: (a - sin a) / sin a; cos:
    0.022) and has up to 5.2 roundings of 2^-24 (u, th u, the series' last two, their sum,
    the magnitude), a result being below 2^24 steps: 5.2 * 0.111 = 0.58.  The angle's low
    part, at most 2^-27 turns and never more than the leading one but where that is 0, is
    rounded four times (its conversion, its product with pi, two sums) and once with the
    magnitude: 5 2^-7 of a step from 2^-20 turns on, 5 steps nearer to the quarter."""
    return np.where(from_quarter < 2.0 ** -20, 5.6, 1.12)


def _phases(freqs):
    return np.array([int(round(f / (2 * np.pi) * 2.0 ** 64)) for f in freqs], dtype=np.uint64)


@pytest.mark.parametrize("magnitude", [1.0, 1.1386294361119891, 0.25])
@pytest.mark.parametrize("base,factor", [(1e4, 1.0), (5e5, 1.0), (5e5, 8.0), (1e6, 32.0), (1e8, 4.0)])
def test_near_positions(angles, base, factor, magnitude):
    """Positions 0 .. 199 of every pair, the slowest ones among them (down to 1e-9 rad a position)."""
    ph = _phases(base ** (-2.0 * np.arange(64) / 128) / factor)
    p, t = np.repeat(ph, 200), np.tile(np.arange(200), 64)
    *both, near = angles(p, t, magnitude)
    for x in both:
        assert (x <= _limit(near)).all(), (x.max(), t[x.argmax()])


def test_far_positions_and_any_phase(angles):
    rng = np.random.default_rng(5)
    n = 2_000_000
    t = (2.0 ** rng.uniform(0, 31, n)).astype(np.int64) * rng.choice([1, 1, 1, -1], n)
    p = (2.0 ** rng.uniform(0, 61.3, n)).astype(np.uint64)
    *both, near = angles(p, t)
    for x in both:
        assert (x <= _limit(near)).all() and x[near > 2.0 ** -20].mean() <= 0.3


def test_next_to_quarter_turns(angles):
    """Angles 2^-64 to 2^-2 turns beside the multiples of a quarter, where one of the two is small."""
    beside = np.concatenate([np.uint64(1) << np.arange(62, dtype=np.uint64), (np.uint64(3) << np.arange(60, dtype=np.uint64)) + np.uint64(1)])
    quarter = np.uint64(1) << np.uint64(62)
    p = np.concatenate([quarter * np.uint64(k) + s * beside for k in range(4) for s in (np.uint64(1), np.uint64(2 ** 64 - 1))])
    p = np.concatenate([p, quarter * np.arange(4, dtype=np.uint64)])      # and the multiples themselves
    *both, near = angles(p, np.ones(len(p)))
    for x in both:
        assert (x <= _limit(near)).all(), (x.max(), hex(int(p[x.argmax()])))
