"""64-bit references of the rotary page write and the sliding-window attention,
and the error that their kernels may have, derived from the roundings they make.

u16 = 2^-8 (bf16), u32 = 2^-24: half a step relative to the value."""
import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, orig=4096.0, low=None, high=None):
    """Radians per position of each pair and the magnitude, as Python floats."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    inv, magnitude = [base ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if scaling == "linear":
        inv = [f / factor for f in inv]
    elif scaling == "bands":
        low, high = low or 1.0, high or 4.0
        out = []
        for f in inv:
            turns = orig / (2 * math.pi / f)
            if turns >= high:
                out.append(f)
            elif turns <= low:
                out.append(f / factor)
            else:
                keep = (turns - low) / (high - low)
                out.append((1 - keep) * f / factor + keep * f)
        inv = out
    elif scaling == "yarn":
        low, high = low or 1.0, high or 32.0
        def pair(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        ramp = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        inv = [f / factor * r + f * (1 - r) for f, r in zip(inv, ramp)]
        magnitude = 0.1 * math.log(factor) + 1.0
    return inv, magnitude


def turn(x, pos, inv, magnitude, interleaved):
    """x [..., heads, D] float64 turned at pos [...] (integers), and |a| + |b| of
    each element's pair (0 where kept)."""
    rot = 2 * len(inv)
    f = torch.tensor(inv, dtype=torch.float64)
    ang = torch.remainder(pos.double()[..., None] * f, 2 * math.pi)[..., None, :]
    c, s = torch.cos(ang) * magnitude, torch.sin(ang) * magnitude
    y, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * magnitude
    return y, size


# A turned element in binary32: the angle is off by 2^-32 turns, by its conversion
# (2^-25 half turns) and, here, by the reference's own product (positions below
# 2^20: 2^-53 * 2^20 radians); sine and cosine by 2 u32 each, the magnitude and
# the two products and the sum by u32 each: below 2^-21 (|a| + |b|).
TURN = 2.0 ** -21


def page_rows(pool, tables, s, n, bs):
    """The first n rows [n, Hkv, ...] of sequence s as stored."""
    t = torch.arange(n)
    return pool.reshape(-1, *pool.shape[2:])[tables[s].long()[t // bs] * bs + t % bs]


def visible(q_pos, n, window, sinks):
    t = torch.arange(n)
    return (t <= q_pos) & ((t < sinks) | (t > q_pos - window))


def attend(q, k, v, seen, scale):
    """One kv head: q [m, G, D], k / v [n, D], seen [m, n] -> o [m, G, D], lse
    [m, G] and, for the error bound, sum p |v| [m, G, D], the largest scale *
    sum |q| |k| [m, G] and the largest p max |v| of a token [m, G]; float64.  A
    row that sees nothing gives 0 and -inf."""
    k, v = (torch.where(seen.any(0)[:, None], x, torch.zeros_like(x)) for x in (k, v))
    s = torch.einsum("mgd,nd->mgn", q, k) * scale
    s = s.masked_fill(~seen[:, None, :], -math.inf)
    lse = torch.logsumexp(s, dim=-1)
    p = torch.exp(s - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[..., None])
    size = torch.einsum("mgd,nd->mgn", q.abs(), k.abs()).masked_fill(~seen[:, None, :], 0).amax(-1) * scale
    return p @ v, lse, p @ v.abs(), size, (p * v.abs().amax(-1)).amax(-1)


def score_error(d, size):
    """Natural units: d products summed in binary32 (a tensor core may truncate:
    2 u32 an addition), the scalings by u32 each, the exponential's 2^-22."""
    return (2 * d + 8) * U32 * size + 2.0 ** -22


def decode_tolerance(o, absum, size, d, n, int8_top=None):
    """Absolute error of one output: the final rounding to bf16; scores' errors
    twice (weights and their sum); sums of n / 16 products of 16 and the joins,
    16 truncated additions each.  bf16 pages hold queries and probabilities to
    2^-16 (a bf16 value and its remainder).  int8 pages (int8_top: the largest
    p |v| of a token) round queries and weights to fp16 once: 2^-11, and 2^-25 of
    2^8 times the largest weight for weights below fp16's normal range; their
    scores are summed under a bias of 1152 / 127 times the largest key."""
    if int8_top is None:
        held, low, scores = 2.0 ** -16, 0.0, score_error(d, size)
    else:
        held, low, scores = 2.0 ** -11, n * 2.0 ** -17 * int8_top[..., None], 10 * score_error(d, size)
    return U16 * o.abs() + low + absum * (2 * (scores + held * size)[..., None] + 2 * held + (n / 16 + 32) * 32 * U32)


def prefill_tolerance(o, absum, size, d, n):
    """As decode_tolerance, with probabilities rounded once to bf16."""
    return U16 * o.abs() + absum * (2 * score_error(d, size)[..., None] + U16 * (1 + U16) + (n / 16 + 32) * 32 * U32)


def lse_tolerance(lse, size, d, n, int8=False):
    scores = 10 * score_error(d, size) + 2.0 ** -11 * size if int8 else score_error(d, size) + 2.0 ** -16 * size
    return scores + (n / 16 + 32) * 32 * U32 + 4 * U32 * lse.abs()
