"""paged_kv_write_rope on the GPU against the 64-bit turn: layouts, parts of the
head, scalings, strides, int8 pages, bad blocks and positions, far positions."""
import pytest
import torch

import window_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_212_gb300 import build
    build.build()
    import paged_kv_cache_212_gb300 as P
    P.load_library()
    return P


def _inputs(seed, starts, n_new, hq, hkv, d, bs, int8, packed=True, far=None):
    gen = torch.Generator().manual_seed(seed)
    n = len(starts)
    blocks = [-(-(p + n_new) // bs) for p in starts]
    n_blocks = sum(blocks) + 2
    perm = torch.randperm(n_blocks, generator=gen).to(torch.int32)
    tables, at = torch.full((n, max(blocks)), n_blocks, dtype=torch.int32), 0
    for s, b in enumerate(blocks):
        tables[s, :b] = perm[at:at + b]
        at += b
    qkv = torch.randn((n, n_new, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16)
    shape = (n_blocks + 1, bs, hkv, d)
    if int8:
        pools = [torch.randint(-127, 128, shape, generator=gen, dtype=torch.int8) for _ in range(2)]
        scales = [torch.rand(shape[:3], generator=gen) for _ in range(2)]
    else:
        pools, scales = [torch.randn(shape, generator=gen).to(torch.bfloat16) for _ in range(2)], [None, None]
    return qkv, tables, torch.tensor(starts, dtype=torch.int32), pools, scales


def _run(P, qkv, tables, start, pools, scales, hq, hkv, rope, packed=True, **kw):
    x = qkv.cuda()
    q, k, v = x.split((hq, hkv, hkv), dim=2)
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    g = [p.cuda() for p in pools]
    sc = [None if t is None else t.cuda() for t in scales]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = P.paged_kv_write_rope(q, k, v, rope, g[0], g[1], tables.cuda(), start.cuda(), k_scales=sc[0], v_scales=sc[1],
                                dev_status=st, **kw)
    torch.cuda.synchronize()
    return out.cpu(), [t.cpu() for t in g], [None if t is None else t.cpu() for t in sc], int(st.item())


def _check(qkv, tables, start, pools, scales, hq, hkv, inv, mag, inter, got):
    out, gp, gs, status = got
    assert status == 0
    n, n_new = qkv.shape[:2]
    bs = pools[0].shape[1]
    pos = start.long()[:, None] + torch.arange(n_new)
    x = qkv.double()
    want, size = R.turn(x[:, :, :hq], pos, inv, mag, inter)
    assert ((out.double() - want).abs() <= R.U16 * want.abs() + R.TURN * size).all()
    rows = tables.long().gather(1, pos // bs) * bs + pos % bs
    kw, ksize = R.turn(x[:, :, hq:hq + hkv], pos, inv, mag, inter)
    vw = x[:, :, hq + hkv:]
    for which, (w, size) in enumerate(((kw, ksize), (vw, torch.zeros_like(vw)))):
        flat = gp[which].reshape(-1, *gp[which].shape[2:])
        if scales[0] is None:
            assert ((flat[rows].double() - w).abs() <= R.U16 * w.abs() + R.TURN * size).all()
            if which == 1:
                assert torch.equal(flat[rows], qkv[:, :, hq + hkv:])
        else:
            sc = gs[which].reshape(-1, hkv)[rows].double()[..., None]
            err = R.TURN * size
            amax = w.abs().amax(-1, keepdim=True)
            assert ((sc * 127 - amax).abs() <= 4 * R.U32 * amax + err.amax(-1, keepdim=True)).all()
            # nearest code of the turned row: half a step, the step's own rounding over 127 steps
            deq = flat[rows].double() * sc
            assert ((deq - w).abs() <= sc * (0.5 + 2.0 ** -14) + err).all()
        # nothing else was written
        kept = torch.ones(flat.shape[0], dtype=torch.bool)
        kept[rows.reshape(-1)] = False
        assert torch.equal(flat[kept], pools[which].reshape(flat.shape)[kept])
        if scales[0] is not None:
            assert torch.equal(gs[which].reshape(-1, hkv)[kept], scales[which].reshape(-1, hkv)[kept])


CASES = [
    # starts, n_new, hq, hkv, d, bs, rot, inter, int8, packed, scaling
    ([0], 1, 1, 1, 64, 16, 64, False, False, True, dict()),
    ([5, 0, 33], 1, 8, 2, 64, 16, 64, True, False, True, dict(scaling="linear", factor=4.0)),
    ([5, 0, 33], 7, 8, 2, 128, 48, 128, False, False, True, dict(scaling="bands", factor=8.0, orig=8192.0)),
    ([100, 17], 31, 6, 3, 128, 16, 32, False, False, False, dict(scaling="ntk", factor=2.0)),
    ([9, 4, 4], 19, 5, 5, 64, 32, 16, True, False, True, dict()),
    ([9, 4, 4], 19, 7, 1, 128, 16, 96, True, False, True, dict(scaling="yarn", factor=4.0, orig=4096.0)),
    ([0], 1, 8, 1, 128, 16, 128, False, True, True, dict()),
    ([3, 70], 21, 4, 3, 128, 16, 64, True, True, True, dict(scaling="yarn", factor=4.0, orig=4096.0)),
    ([3, 70], 21, 4, 2, 64, 16, 48, False, True, False, dict()),
    ([0, 250], 150, 32, 8, 128, 16, 128, False, True, True, dict()),
    ([0, 11, 800], 200, 32, 8, 128, 16, 128, False, False, True, dict()),
    ([40, 1], 320, 40, 8, 128, 16, 128, True, False, True, dict()),           # chunks: narrow blocks, two rounds
    ([40, 1], 160, 40, 8, 128, 16, 128, False, True, True, dict()),
    ([7], 700, 8, 8, 64, 16, 32, False, True, False, dict(scaling="linear", factor=2.0)),
]


@pytest.mark.parametrize("starts,n_new,hq,hkv,d,bs,rot,inter,int8,packed,scaling", CASES)
def test_rows_are_turned_and_stored(P, starts, n_new, hq, hkv, d, bs, rot, inter, int8, packed, scaling):
    inv, mag = R.frequencies(rot, **scaling)
    named = {{"orig": "original_context"}.get(k, k): v for k, v in scaling.items()}
    rope = P.Rope(rot, interleaved=inter, **named)
    x = _inputs(n_new + hq, starts, n_new, hq, hkv, d, bs, int8)
    _check(*x, hq, hkv, inv, mag, inter, _run(P, *x, hq, hkv, rope, packed))


def test_far_positions(P):
    """Positions near 2^20: a product in binary32 would be off by 0.06 radians."""
    d, bs, hq, hkv, rot = 64, 256, 2, 1, 64
    starts = [2 ** 20 - 300, 2 ** 19 + 12345]
    inv, mag = R.frequencies(rot)
    gen = torch.Generator().manual_seed(3)
    n_new, width = 4, 2 ** 20 // bs
    tables = torch.full((2, width), 4, dtype=torch.int32)
    for s, p in enumerate(starts):
        tables[s, p // bs] = s
    qkv = torch.randn((2, n_new, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16)
    pools = [torch.randn((5, bs, hkv, d), generator=gen).to(torch.bfloat16) for _ in range(2)]
    x = (qkv, tables, torch.tensor(starts, dtype=torch.int32), pools, [None, None])
    _check(*x, hq, hkv, inv, mag, False, _run(P, *x, hq, hkv, P.Rope(rot)))


def test_queries_in_place_and_out_given(P):
    hq, hkv = 4, 2
    x = _inputs(11, [3, 40], 9, hq, hkv, 128, 16, False)
    rope = P.Rope(128)
    want = _run(P, *x, hq, hkv, rope)
    qkv, tables, start, pools, scales = x
    q, k, v = (t.contiguous().cuda() for t in qkv.split((hq, hkv, hkv), dim=2))
    g = [p.cuda() for p in pools]
    got = P.paged_kv_write_rope(q, k, v, rope, g[0], g[1], tables.cuda(), start.cuda(), q_out=q)
    assert got is q and torch.equal(q.cpu(), want[0]) and torch.equal(g[0].cpu(), want[1][0])


def test_int8_values_are_those_of_the_page_write(P):
    """Values are not turned: their codes and scales are paged_kv_write_int8's."""
    hq, hkv = 8, 2
    qkv, tables, start, pools, scales = _inputs(12, [3, 40, 0], 33, hq, hkv, 128, 16, True)
    _, gp, gs, st = _run(P, qkv, tables, start, pools, scales, hq, hkv, P.Rope(128))
    k, v = (t.contiguous().cuda() for t in qkv.split((hq, hkv, hkv), dim=2)[1:])
    p2, s2 = [p.cuda() for p in pools], [t.cuda() for t in scales]
    P.paged_kv_write_int8(k, v, p2[0], p2[1], s2[0], s2[1], tables.cuda(), start.cuda())
    assert st == 0 and torch.equal(p2[1].cpu(), gp[1]) and torch.equal(s2[1].cpu(), gs[1])


def test_int8_codes_next_to_halves_and_of_odd_rows(P):
    """Ties (x / scale exactly between two codes go to the even one), rows of one
    element, of the smallest normal and of subnormal numbers, with infinities and NaN:
    the codes are paged_kv_write_int8's, and keys turned by an angle of 0 too."""
    hq, hkv, d = 2, 4, 64
    qkv, tables, start, pools, scales = _inputs(16, [0], 12, hq, hkv, d, 16, True)
    half = (torch.arange(d) - 31.5).to(torch.bfloat16)           # absmax 127: the scale is 1
    half[5] = 127
    tiny = torch.finfo(torch.bfloat16).tiny
    one = torch.zeros(d, dtype=torch.bfloat16)
    one[17] = -3.25
    rows = [half, -half, half * 2 ** -20, half * 2 ** 40, one, half * tiny, half * tiny / 128, one * 0 + tiny,
            torch.where(torch.arange(d) == 9, torch.inf, half.float()).to(torch.bfloat16),
            torch.where(torch.arange(d) == 9, torch.nan, half.float()).to(torch.bfloat16)]
    for i, x in enumerate(rows):
        qkv[0, i, hq:] = x
    rope = P.Rope(16, base=10000.0)
    rope.phases.zero_()                                          # no turn at any position
    _, gp, gs, st = _run(P, qkv, tables, start, pools, scales, hq, hkv, rope)
    k, v = (t.contiguous().cuda() for t in qkv.split((hq, hkv, hkv), dim=2)[1:])
    p2, s2 = [p.cuda() for p in pools], [t.cuda() for t in scales]
    P.paged_kv_write_int8(k, v, p2[0], p2[1], s2[0], s2[1], tables.cuda(), start.cuda())
    assert st == 0
    assert torch.equal(p2[1].cpu(), gp[1]) and torch.equal(s2[1].cpu(), gs[1])
    pos = torch.arange(8)                                        # the finite rows (0 times inf is NaN in a turn)
    at = tables[0, 0].long() * 16 + pos
    assert torch.equal(p2[0].cpu().view(-1, hkv, d)[at], gp[0].view(-1, hkv, d)[at])
    assert torch.equal(s2[0].cpu().view(-1, hkv)[at], gs[0].view(-1, hkv)[at])


@pytest.mark.parametrize("int8", [False, True])
def test_bad_rows_are_reported_and_skipped(P, int8):
    hq, hkv = 4, 2
    qkv, tables, start, pools, scales = _inputs(13, [3, 20, 0, 5], 4, hq, hkv, 64, 16, int8)
    rope, n_blocks = P.Rope(64), pools[0].shape[0] - 1
    good = _run(P, qkv, tables, start, pools, scales, hq, hkv, rope)
    bad_tables = tables.clone()
    bad_tables[0, 0] = n_blocks + 1                       # an id outside the pool
    bad_start = start.clone()
    bad_start[2] = -2                                     # two rows before the first position
    bad_start[3] = tables.shape[1] * 16 - 1               # three rows behind the last one
    out, gp, gs, st = _run(P, qkv, bad_tables, bad_start, pools, scales, hq, hkv, rope)
    assert st == 1 | 2
    assert torch.equal(out[:2], good[0][:2])              # the query of a skipped row is turned all the same
    flat, ref, old = (t.reshape(-1, hkv, 64) for t in (gp[0], good[1][0], pools[0]))
    own = tables[1, 20 // 16].long() * 16 + 20 % 16 + torch.arange(4)
    assert torch.equal(flat[own], ref[own])
    lost = tables[0, 0].long() * 16 + 3 + torch.arange(4)
    assert torch.equal(flat[lost], old[lost])


def test_zero_and_non_finite_rows_int8(P):
    hq, hkv = 2, 2
    qkv, tables, start, pools, scales = _inputs(14, [0], 3, hq, hkv, 64, 16, True)
    qkv[0, 1, hq:] = 0
    _, gp, gs, st = _run(P, qkv, tables, start, pools, scales, hq, hkv, P.Rope(64))
    row = int(tables[0, 0]) * 16 + 1
    assert st == 0
    for which in range(2):
        assert not gp[which].reshape(-1, hkv, 64)[row].any() and not gs[which].reshape(-1, hkv)[row].any()


def test_on_another_stream_and_in_a_graph(P):
    hq, hkv = 8, 2
    qkv, tables, start, pools, scales = _inputs(15, [3, 40], 5, hq, hkv, 128, 16, False)
    rope = P.Rope(128)
    want = _run(P, qkv, tables, start, pools, scales, hq, hkv, rope)
    x, g, tab, sp = qkv.cuda(), [p.cuda() for p in pools], tables.cuda(), start.cuda()
    q, k, v = x.split((hq, hkv, hkv), dim=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = P.paged_kv_write_rope(q, k, v, rope, g[0], g[1], tab, sp, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(g[0].cpu(), want[1][0])
    out2 = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.paged_kv_write_rope(q, k, v, rope, g[0], g[1], tab, sp, q_out=out2)
    for p, src in zip(g, pools):
        p.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2.cpu(), want[0]) and torch.equal(g[1].cpu(), want[1][1])
