"""The windowed and rotary calls where something is wrong with a call or its
neighbour: waits that run out with another call behind them, chunks that run past
the table, and the calls around them, which have to stay right."""
import pytest
import torch

import window_reference as R

from test_gpu_window import P, _cuda, _paged  # noqa: F401  (P: the fixture)

pytestmark = pytest.mark.gpu


# d, n_seqs, hkv, group, chunk, window, sinks: units of at most the tiles that the rings
# hold, one unit or two halves a CTA; then about three units a CTA, of one tile each
@pytest.mark.parametrize("d,n,hkv,group,chunk,window,sinks", [(128, 2, 4, 4, 60, 100, 4), (64, 8, 8, 4, 448, 32, 0)])
def test_prefill_behind_one_whose_waits_ran_out(P, d, n, hkv, group, chunk, window, sinks):  # noqa: F811
    """A call that gives up has no copy on its way into shared memory when it ends: the
    call behind it, which takes over its SMs, gives the bits that it gives alone."""
    bs = 16
    lens = [chunk + 13 * s for s in range(n)]
    pools, _, tables, _ = _paged(d + n, lens, window, sinks, chunk, hkv, d, bs, False)
    gen = torch.Generator().manual_seed(8)
    q, other = (torch.randn((n, chunk, hkv * group, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor([x - chunk for x in lens], dtype=torch.int32).cuda()
    call = lambda x, st, out: P.paged_prefill_attention_window(x, kp, vp, tab, pre, d ** -0.5, window, sinks, out=out,
                                                               dev_status=st)
    bad, good = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    want = call(q, good, torch.empty_like(q)).clone()
    lost, got = torch.empty_like(q), torch.empty_like(q)
    lib = P.load_library()
    for ns in (1, 100, 1000, 1, 3000, 300, 1):
        got.zero_()
        torch.cuda.synchronize()
        try:
            lib.pkv_set_pipeline_wait_ns(ns)               # read when a launch is prepared
            call(other, bad, lost)
        finally:
            lib.pkv_set_pipeline_wait_ns(0)
        call(q, good, got)
        torch.cuda.synchronize()
        assert int(good.item()) == 0 and torch.equal(got, want), ns
    assert int(bad.item()) & ~16 == 0 and int(bad.item()) == 16


# hkv, group, d, chunk: whole units, and halves (one sequence), of which only the last
# reach past the table
@pytest.mark.parametrize("n", [1, 3, 25])
@pytest.mark.parametrize("hkv,group,d,chunk", [(2, 4, 64, 300), (8, 8, 128, 130)])
def test_prefill_chunk_that_ends_past_the_table(P, hkv, group, d, chunk, n):  # noqa: F811
    """A chunk whose end alone is past the table is a bad length for all of it: its
    rows stay as they were, whatever its units are, and the other sequences' are right."""
    bs, window, sinks, bad = 16, 70, 4, n // 2
    lens = [chunk + 29 * s for s in range(n)]
    pools, _, tables, _ = _paged(n + d, lens, window, sinks, chunk, hkv, d, bs, False)
    q = torch.randn((n, chunk, hkv * group, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor([x - chunk for x in lens], dtype=torch.int32).cuda()
    capacity = tables.shape[1] * bs

    def call(prefix):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:3], 7.0, device="cuda")
        P.paged_prefill_attention_window(q, kp, vp, tab, prefix, d ** -0.5, window, sinks, out=out, lse_out=lse, dev_status=st)
        torch.cuda.synchronize()
        return int(st.item()), out, lse

    st, want, want_lse = call(pre)
    assert st == 0 and torch.isfinite(want.float()).all()
    others = [s for s in range(n) if s != bad]
    for past in (1, chunk // 2, chunk - 1):
        pre[bad] = capacity - chunk + past                 # the first chunk - past rows are inside
        # (the bad sequence's blocks are not looked up either: its table entries are ids outside the pool)
        tab[bad] = pools[0].shape[0]
        st, out, lse = call(pre)
        assert st == 4, (past, st)
        assert (out[bad] == 3.0).all() and (lse[bad] == 7.0).all(), past
        assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others]), past


@pytest.mark.parametrize("interleaved", [False, True])
def test_slow_pairs_near_position_0(P, interleaved):  # noqa: F811
    """The sine of a pair of 1e-12 rad a position is right relative to itself: a pair
    (1, 0) becomes (cos, sin), each rounded once to bf16."""
    d, bs, n_new, base, factor = 128, 16, 9, 1e10, 32.0
    rope = P.Rope(d, base=base, interleaved=interleaved, scaling="linear", factor=factor)
    inv, _ = R.frequencies(d, base, "linear", factor)
    x = torch.zeros((1, n_new, 1, d), dtype=torch.bfloat16)
    x[..., 0::2] = 1
    if not interleaved:
        x = torch.cat((x[..., 0::2], x[..., 1::2]), dim=-1)
    new, pool = torch.zeros((1, n_new, 1, d), dtype=torch.bfloat16), torch.zeros((2, bs, 1, d), dtype=torch.bfloat16)
    x, k, v, kp, vp = _cuda(x, new, new, pool, pool)
    tab, start = torch.zeros((1, 1), dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    out = P.paged_kv_write_rope(x, k, v, rope, kp, vp, tab, start).cpu().double()[0, :, 0]
    cos, sin = (out[:, 0::2], out[:, 1::2]) if interleaved else (out[:, :d // 2], out[:, d // 2:])
    angle = torch.arange(n_new).double()[:, None] * torch.tensor(inv, dtype=torch.float64)
    for got, want in ((cos, angle.cos()), (sin, angle.sin())):
        # bf16's rounding, and 6 steps of binary32
        assert ((got - want).abs() <= (R.U16 + 12 * R.U32) * want.abs()).all()


@pytest.mark.parametrize("d,hkv,group,n", [(128, 2, 8, 1), (128, 8, 4, 66), (64, 1, 1, 3), (64, 4, 3, 40), (128, 8, 2, 20)])
def test_int8_weights_keep_their_bits(P, d, hkv, group, n):  # noqa: F811
    """Two tokens of the same score and opposite V codes, whose V scales differ by less
    than 2^-9: what is left is a difference of weights, which shows their rounding."""
    bs, hq = 16, hkv * group
    gen = torch.Generator().manual_seed(d + n)
    row = torch.randint(1, 128, (n, hkv, d), generator=gen, dtype=torch.int8)
    row[..., 5] = 127
    kp, vp = (torch.zeros((n + 1, bs, hkv, d), dtype=torch.int8) for _ in range(2))
    ks, vs = torch.ones((n + 1, bs, hkv)) * 0.01, torch.ones((n + 1, bs, hkv))
    kp[:n, :2], vp[:n, 0], vp[:n, 1] = row[:, None], row, -row
    scales = 0.01 * (1 + torch.rand((n, 2, hkv), generator=gen) * 2.0 ** -9)
    vs[:n, :2] = scales
    q = torch.randn((n, hq, d), generator=gen).to(torch.bfloat16)
    tab, ctx = torch.arange(n, dtype=torch.int32)[:, None], torch.full((n,), 2, dtype=torch.int32)
    q, kp, vp, ks, vs, tab, ctx = _cuda(q, kp, vp, ks, vs, tab, ctx)
    out = P.paged_decode_attention_window(q, kp, vp, tab, ctx, d ** -0.5, 64, k_scales=ks, v_scales=vs)
    sc = scales.double()[..., None]
    want = (sc[:, 0] - sc[:, 1]) * row.double() / 2               # [n, hkv, d]
    size = (sc[:, 0] + sc[:, 1]) * row.double() / 2
    # the output's rounding; weights held to 2^-22, and sums of one tile and the joins (as
    # window_reference.decode_tolerance has them), against a rounding to fp16 of 2^-12 on average
    tol = R.U16 * want.abs() + size * (2.0 ** -22 + (2 / 16 + 32) * 32 * R.U32)
    got = out.cpu().double().view(n, hkv, group, d)
    assert ((got - want[:, :, None]).abs() <= tol[:, :, None]).all()
