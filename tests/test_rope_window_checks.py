"""The rotary write and the windowed attention on the CPU: phases against their
formulas, refusals of the C calls before anything is launched, refusals of the
binding, and the 64-bit references against a plain loop."""
import ctypes
import math

import pytest
import torch

import window_reference as R

FAKE, MISALIGNED = 0x1000, 0x1008      # never dereferenced


@pytest.fixture(scope="module")
def P():
    from paged_kv_cache_212_gb300 import build as B
    try:
        B.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    B.build()
    import paged_kv_cache_212_gb300 as P
    P.load_library()
    return P


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="bands", factor=8.0, orig=8192.0), dict(scaling="yarn", factor=4.0, orig=4096.0),
            dict(scaling="bands", factor=2.0, orig=1000.0, low=2.0, high=9.5),
            dict(scaling="yarn", factor=1.0, orig=2048.0), dict(scaling="yarn", factor=32.0, orig=300.0, low=0.5, high=3.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 500000.0), (128, 1.5)])
def test_phases_match_the_formulas(P, kw, rot, base):
    inv, magnitude = R.frequencies(rot, base, **kw)
    named = {{"orig": "original_context", "low": "low_turns", "high": "high_turns"}.get(k, k): v for k, v in kw.items()}
    rope = P.Rope(rot, base=base, device="cpu", **named)
    assert rope.phases.shape == (rot // 2,) and rope.rot_dim == rot and not rope.interleaved
    assert abs(rope.magnitude - magnitude) <= 2.0 ** -50 * magnitude
    for ph, f in zip(rope.phases.tolist(), inv):
        turns = (ph % 2 ** 64) / 2.0 ** 64
        # a power, a few products and sums in binary64, each side its own: 2^-47 relative at most
        assert abs(turns - f / (2 * math.pi)) <= 2.0 ** -47 * f / (2 * math.pi) + 2.0 ** -64


def test_rope_refusals(P):
    for kw in (dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=-16), dict(base=1.0), dict(base=float("nan")),
               dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("inf")),
               dict(scaling="bands", factor=2.0, original_context=-1.0),
               dict(scaling="yarn", factor=2.0, original_context=4096, low_turns=4.0, high_turns=4.0),
               dict(scaling="bands", factor=2.0, original_context=4096, low_turns=0.0)):
        args = dict(dict(rot_dim=64, device="cpu"), **kw)
        with pytest.raises(P.PagedKVError) as e:
            P.Rope(**args)
        assert e.value.status == 1, kw
    with pytest.raises(ValueError):
        P.Rope(64, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        P.Rope(64, scaling="yarn", factor=2.0, device="cpu")
    lib = P.load_library()
    buf, mag = (ctypes.c_uint64 * 8)(), ctypes.c_double()
    assert lib.pkv_rope_phases(16, 1e4, 9, 1.0, 0.0, 1.0, 2.0, buf, ctypes.byref(mag)) == 2
    assert lib.pkv_rope_phases(16, 1e4, 0, 1.0, 0.0, 1.0, 2.0, None, ctypes.byref(mag)) == 1
    assert lib.pkv_rope_phases(16, 1e4, 0, 1.0, 0.0, 1.0, 2.0, buf, None) == 1


def _rope(P, phases=FAKE, rot=64, magnitude=1.0):
    return ctypes.pointer(P._RopeC(phases, rot, 0, magnitude))


def _write_args(P, **kw):
    d = kw.get("dims", P.Dims(8, 16, 2, 64))
    return [kw.get("q", FAKE), kw.get("qs", 8 * 64), kw.get("hq", 8), kw.get("k", FAKE), kw.get("ks", 128),
            kw.get("v", FAKE), kw.get("vs", 128), kw.get("rope", _rope(P)), kw.get("qo", FAKE + 0x100), kw.get("kp", FAKE),
            FAKE, kw.get("ksc"), kw.get("vsc"), kw.get("dt", 0), d, kw.get("tab", FAKE), kw.get("mb", 4),
            kw.get("sp", FAKE), kw.get("n", 2), kw.get("n_new", 3), None, None]


def test_rope_write_argument_checks(P):
    f = P.load_library().paged_kv_write_rope
    D = P.Dims
    assert f(*_write_args(P, n=0)) == 0 and f(*_write_args(P, n_new=0)) == 0
    for kw in (dict(q=None), dict(q=MISALIGNED), dict(k=None), dict(v=MISALIGNED), dict(qo=None), dict(kp=None),
               dict(tab=None), dict(sp=None), dict(n=-1), dict(n_new=-1), dict(mb=0), dict(hq=0), dict(rope=None),
               dict(qs=8 * 64 - 8), dict(qs=8 * 64 + 4), dict(ks=120), dict(vs=-128),
               dict(rope=_rope(P, phases=None)), dict(rope=_rope(P, phases=MISALIGNED)), dict(rope=_rope(P, rot=0)),
               dict(rope=_rope(P, rot=80)), dict(rope=_rope(P, magnitude=float("nan"))), dict(dt=1),
               dict(dt=1, ksc=FAKE, vsc=FAKE + 2), dict(qo=FAKE, qs=8 * 64 + 128), dict(dims=D(-1, 16, 2, 64))):
        assert f(*_write_args(P, **kw)) == 1, kw
    for kw in (dict(dt=2), dict(dims=D(8, 16, 2, 96)), dict(dims=D(8, 24, 2, 64)), dict(rope=_rope(P, rot=24))):
        assert f(*_write_args(P, **kw)) == 2, kw
    assert f(*_write_args(P, n_new=65)) == 3
    assert f(*_write_args(P, n=1 << 30)) == 3


def _decode_args(P, **kw):
    d = kw.get("dims", P.Dims(8, 16, 2, 64))
    return [kw.get("q", FAKE), kw.get("hq", 8), FAKE, kw.get("vp", FAKE), kw.get("ksc"), kw.get("vsc"), kw.get("dt", 0), d,
            kw.get("tab", FAKE), kw.get("mb", 4), kw.get("ctx", FAKE), kw.get("n", 2), kw.get("sc", 0.125),
            kw.get("win", 10), kw.get("sinks", 2), kw.get("out", FAKE), None, None, None]


def test_window_decode_argument_checks(P):
    f = P.load_library().paged_decode_attention_window
    D = P.Dims
    assert f(*_decode_args(P, n=0)) == 0
    for kw in (dict(q=None), dict(q=MISALIGNED), dict(vp=None), dict(tab=None), dict(ctx=None), dict(out=None),
               dict(out=MISALIGNED), dict(n=-1), dict(mb=0), dict(hq=7), dict(win=0), dict(win=-5), dict(sinks=-1),
               dict(sc=0.0), dict(sc=float("inf")), dict(sc=float("nan")), dict(dt=1), dict(dt=1, ksc=FAKE + 2, vsc=FAKE)):
        assert f(*_decode_args(P, **kw)) == 1, kw
    for kw in (dict(hq=18), dict(dt=7), dict(dims=D(8, 16, 2, 32)), dict(dims=D(8, 512, 2, 64))):
        assert f(*_decode_args(P, **kw)) == 2, kw
    for kw in (dict(mb=1 << 30), dict(mb=0x7fffff00 // 16 + 1), dict(n=1 << 30)):
        assert f(*_decode_args(P, **kw)) == 3, kw


def test_window_step_argument_checks(P):
    f = P.load_library().paged_decode_step_window

    def args(**kw):
        a = _decode_args(P, **kw)
        return [kw.get("k", FAKE), kw.get("ks", 128), kw.get("v", FAKE), kw.get("vs", 128), kw.get("sp", FAKE), a[0],
                kw.get("qs", 512), a[1], kw.get("rope", _rope(P)), *a[2:]]

    assert f(*args(n=0)) == 0
    for kw in (dict(k=None), dict(v=MISALIGNED), dict(sp=None), dict(ks=64), dict(vs=132), dict(qs=504), dict(win=0),
               dict(rope=_rope(P, rot=128)), dict(rope=_rope(P, phases=None)), dict(q=None)):
        assert f(*args(**kw)) == 1, kw
    assert f(*args(rope=_rope(P, rot=40))) == 2


def test_window_prefill_argument_checks(P):
    f = P.load_library().paged_prefill_attention_window
    d = P.Dims(8, 16, 2, 64)

    def args(**kw):
        return [kw.get("q", FAKE), kw.get("hq", 8), FAKE, FAKE, d, FAKE, kw.get("mb", 4), FAKE, kw.get("n", 1), kw.get("chunk", 16), 0.1,
                kw.get("win", 9), kw.get("sinks", 0), kw.get("out", FAKE), None, None, None]

    assert f(*args(n=0)) == 0 and f(*args(chunk=0)) == 0
    for kw in (dict(win=0), dict(sinks=-1), dict(q=None), dict(out=MISALIGNED), dict(hq=7), dict(n=-1)):
        assert f(*args(**kw)) == 1, kw
    assert f(*args(hq=6)) == 2
    assert f(*args(chunk=65)) == 3
    assert f(*args(mb=0x7fffff00 // 16 + 1)) == 3


def test_token_strides(P):
    x = torch.zeros((3, 5, 12, 64), dtype=torch.bfloat16)
    q, k, v = x.split((8, 2, 2), dim=2)
    assert [P._token_stride(t, "t", 4, -1) for t in (q, k, v)] == [768] * 3
    assert P._token_stride(x[:, :1, :8], "t", 4, -1) == 5 * 768     # one token of each sequence
    assert P._token_stride(x[1:2, 2:3, 3:5], "t", 4, -1) == 128     # a single token: its own length
    assert P._token_stride(x[:, 0, :8], "t", 3, -1) == 5 * 768
    assert P._token_stride(x[:, :, 3:4], "t", 4, -1) == 768
    for bad in (x.transpose(1, 2), x[:, ::2], x[..., ::2], x[:, :, ::2], x.float()):
        with pytest.raises(ValueError):
            P._token_stride(bad, "t", 4, -1)
    with pytest.raises(ValueError):
        P._token_stride(x, "t", 4, 0)             # another device
    with pytest.raises(ValueError):
        P._token_stride(x[0], "t", 4, -1)
    with pytest.raises(TypeError):
        P._token_stride(None, "t", 4, -1)


def test_counts(P):
    assert P._count(5, "window") == 5 and P._count(2 ** 40 + 7, "window") == 2 ** 31 - 1
    with pytest.raises(ValueError):
        P._count(-1, "sinks")


def test_host_tensors_are_refused(P):
    q, pool = torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    tab, lens = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    rope = P.Rope(64, device="cpu")
    with pytest.raises(ValueError):
        P.paged_decode_attention_window(q, pool, pool, tab, lens, 0.1, 8)
    with pytest.raises(ValueError):
        P.paged_prefill_attention_window(q[:, None], pool, pool, tab, lens, 0.1, 8)
    with pytest.raises(ValueError):
        P.paged_kv_write_rope(q[:, None], q[:, None, :2], q[:, None, :2], rope, pool, pool, tab, lens)
    with pytest.raises(ValueError):
        P.paged_decode_step_window(q[:, None, :2], q[:, None, :2], lens, q, pool, pool, tab, lens, 0.1, 8, rope=rope)
    with pytest.raises(ValueError):
        P.WindowDecodePlan(pool, pool, tab, lens, 0.1, 8, 8)


def test_reference_turn_is_a_rotation():
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((4, 2, 64), generator=gen, dtype=torch.float64)
    inv, _ = R.frequencies(32)
    pos = torch.tensor([0, 1, 1000, 7])
    for inter in (False, True):
        y, _ = R.turn(x, pos, inv, 1.0, inter)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 32:], x[..., 32:])
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1), rtol=1e-12)
        # scores depend on the distance alone
        a, _ = R.turn(x[:1].expand(4, 2, 64), pos, inv, 1.0, inter)
        b, _ = R.turn(x[1:2].expand(4, 2, 64), pos + 3, inv, 1.0, inter)
        dots = (a * b).sum(-1)
        assert torch.allclose(dots, dots[:1].expand_as(dots), rtol=1e-9)


def test_reference_attention_against_a_loop():
    gen = torch.Generator().manual_seed(6)
    n, d, window, sinks = 9, 4, 3, 2
    k, v = (torch.randn((n, d), generator=gen, dtype=torch.float64) for _ in range(2))
    q = torch.randn((n, 1, d), generator=gen, dtype=torch.float64)
    seen = torch.stack([R.visible(i, n, window, sinks) for i in range(n)])
    o, lse, _, _, _ = R.attend(q, k, v, seen, 0.3)
    for i in range(n):
        ts = [t for t in range(n) if t <= i and (t < sinks or t > i - window)]
        w = [math.exp(0.3 * float(q[i, 0] @ k[t])) for t in ts]
        assert abs(math.log(sum(w)) - float(lse[i, 0])) < 1e-12
        assert torch.allclose(sum(x * v[t] for x, t in zip(w, ts)) / sum(w), o[i, 0], atol=1e-12)


def test_native_marshalling_refuses_what_it_does_not_know(P):
    """The native part of the binding answers None, without a call, to anything but
    CUDA tensors of the right kinds; the Python part then says what is wrong."""
    n = P._native
    assert n is not None
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    pool, tab, lens = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    rope = P.Rope(64, device="cpu")
    args = [q, kv, kv, rope._address, rope.phases, pool, pool, tab, lens, None, None, None, None]
    assert n.write_rope(*args) is None and n.write_rope() is None
    for i in range(len(args)):
        assert n.write_rope(*args[:i], "x", *args[i + 1:]) is None
    args = [q, pool, pool, tab, lens, 0.1, 8, 0, None, None, None]
    assert n.prefill_window(*args) is None and n.prefill_window(None) is None
    for i in range(len(args)):
        assert n.prefill_window(*args[:i], None, *args[i + 1:]) is None
    assert n.prefill_window(*args[:6], 2 ** 70, *args[7:]) is None
    with pytest.raises(ValueError):
        n.run_plan(None, q, None, None, None)
    plan = n.make_plan(0, 4, 0, 1, 1, 0, 0, 0, 2, 16, 2, 64, 1, 2, 1, 1, 0.1, 8, 0, 1, 0, 0)
    for a in ((None, None, None, None), (q[:, 0], None, None, None), (q[:, 0], kv, kv, lens)):
        assert n.run_plan(plan, *a) is None
