"""Sliding-window attention on the GPU against the 64-bit reference: decode over
bf16 and int8 pages, steps, chunks.  Rows that no query sees hold NaN (int8: NaN
scales), and table entries of blocks without a visible token hold ids outside
the pool: neither may show."""
import pytest
import torch

import window_reference as R

pytestmark = pytest.mark.gpu

GARBAGE_ID = -12345


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_212_gb300 import build
    build.build()
    import paged_kv_cache_212_gb300 as P
    P.load_library()
    return P


def _paged(seed, lens, window, sinks, m, hkv, d, bs, int8, spare=2):
    """Pools holding rows 0 .. len - 1 of each sequence where one of its last m
    queries sees them, NaN elsewhere; tables; the stored values in 64 bits
    (0 where unseen) and which rows are seen."""
    gen = torch.Generator().manual_seed(seed)
    n = len(lens)
    blocks = [-(-x // bs) for x in lens]
    n_blocks, width = sum(blocks) + 1, max(max(blocks), 1) + spare
    perm = torch.randperm(n_blocks, generator=gen).to(torch.int32)
    tables, at = torch.full((n, width), GARBAGE_ID, dtype=torch.int32), 0
    shape = (n_blocks + 1, bs, hkv, d)
    if int8:
        pools = [torch.full(shape, 127, dtype=torch.int8) for _ in range(2)]
        scales = [torch.full(shape[:3], float("nan")) for _ in range(2)]
    else:
        pools, scales = [torch.full(shape, float("nan"), dtype=torch.bfloat16) for _ in range(2)], [None, None]
    values = []
    for s, x in enumerate(lens):
        seen = torch.zeros(x, dtype=torch.bool)
        for i in range(m):
            if x - m + i >= 0:
                seen |= R.visible(x - m + i, x, window, sinks)
        for b in range(blocks[s]):
            if seen[b * bs:(b + 1) * bs].any():
                tables[s, b] = perm[at + b]
        t = torch.nonzero(seen).flatten()
        rows = perm[at:at + blocks[s]].long()[t // bs] * bs + t % bs
        at += blocks[s]
        pair = []
        for which in range(2):
            full = torch.zeros((x, hkv, d), dtype=torch.float64)
            if int8:
                code = torch.randint(-127, 128, (len(t), hkv, d), generator=gen, dtype=torch.int8)
                code[..., 3] = 127                # a quantised row's largest code
                # scales spread over three powers of ten, some rows of zeros
                sc = 10.0 ** (torch.rand((len(t), hkv), generator=gen) * 3 - 4.5)
                sc[torch.rand((len(t), hkv), generator=gen) < 0.03] = 0
                pools[which].view(-1, hkv, d)[rows] = code
                scales[which].view(-1, hkv)[rows] = sc
                full[t] = code.double() * sc.double()[..., None]
            else:
                val = torch.randn((len(t), hkv, d), generator=gen).to(torch.bfloat16)
                pools[which].view(-1, hkv, d)[rows] = val
                full[t] = val.double()
            pair.append(full)
        values.append(pair)
    return pools, scales, tables, values


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check_decode(out, lse, q, values, lens, window, sinks, hkv, scale, int8, q_values=None):
    """out [n, Hq, D], lse [n, Hq] against the reference; q bf16 (or q_values in 64 bits)."""
    n, hq, d = out.shape
    g = hq // hkv
    out, lse = out.cpu().double(), lse.cpu().double()
    qd = (q.cpu().double() if q_values is None else q_values).view(n, hkv, g, d)
    for s, x in enumerate(lens):
        if x == 0:
            assert not out[s].any() and (lse[s] == -torch.inf).all()
            continue
        seen = R.visible(x - 1, x, window, sinks)[None]
        count = int(seen.sum())
        for h in range(hkv):
            o, ls, absum, size, top = (x[0] for x in R.attend(qd[s, h][None], values[s][0][:, h], values[s][1][:, h],
                                                              seen, scale))
            got = out[s].view(hkv, g, d)[h]
            assert torch.isfinite(got).all(), (s, h)
            over = (got - o).abs() - R.decode_tolerance(o, absum, size, d, count, top if int8 else None)
            assert (over <= 0).all(), (s, h, float(over.max()))
            over = (lse[s].view(hkv, g)[h] - ls).abs() - R.lse_tolerance(ls, size, d, count, int8)
            assert (over <= 0).all(), (s, h, float(over.max()))


# lens, window, sinks, hkv, group, d, bs
DECODE = [
    ([1], 1, 0, 1, 1, 64, 16),
    ([0, 1, 2, 15, 16, 17, 31, 33], 5, 0, 2, 4, 64, 16),
    ([0, 1, 3, 63, 64, 65, 68, 69, 255], 64, 4, 2, 4, 64, 16),
    ([1, 40, 41, 200, 333], 40, 37, 1, 8, 128, 16),
    ([100, 517, 90], 128, 1, 3, 3, 128, 48),
    ([700, 20, 0], 1, 16, 4, 2, 128, 32),
    ([300, 301], 2 ** 31 - 1, 0, 2, 1, 128, 16),          # a window beyond every length
    ([300, 77], 16, 2 ** 31 - 1, 2, 5, 128, 16),          # every token a first one
    ([64], 33, 1, 1, 7, 64, 64),
    ([2500, 1300], 1024, 4, 2, 6, 128, 16),               # split over a cluster
    ([4100], 4000, 5, 1, 4, 128, 256),
    ([3000, 2999, 50], 2048, 0, 1, 8, 64, 16),
    ([500 + 7 * i for i in range(40)], 256, 4, 8, 4, 128, 16),   # one CTA a unit
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,window,sinks,hkv,group,d,bs", DECODE)
def test_decode(P, lens, window, sinks, hkv, group, d, bs, int8):
    pools, scales, tables, values = _paged(len(lens) + window % 97, lens, window, sinks, 1, hkv, d, bs, int8)
    gen = torch.Generator().manual_seed(77)
    hq, scale = hkv * group, d ** -0.5
    q = torch.randn((len(lens), hq, d), generator=gen).to(torch.bfloat16)
    kp, vp, ks, vs, tab = _cuda(*pools, *scales, tables)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    lse = torch.full((len(lens), hq), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = P.paged_decode_attention_window(q.cuda(), kp, vp, tab, ctx, scale, window, sinks, k_scales=ks, v_scales=vs,
                                          lse_out=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check_decode(out, lse, q, values, lens, window, sinks, hkv, scale, int8)
    # a second call gives the same bits (no order of summation is left to chance)
    again = P.paged_decode_attention_window(q.cuda(), kp, vp, tab, ctx, scale, window, sinks, k_scales=ks, v_scales=vs)
    assert torch.equal(again, out)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [3, 11, 20, 33, 40, 52, 66])
def test_decode_batches(P, n, int8):
    """Batches between one that leaves most of the machine idle and one that overfills
    it: clusters of several sizes, CTAs of both, spread over the SMs or not."""
    lens = [300 + 37 * (i % 10) for i in range(n)]
    window, sinks, hkv, group, d = 500, 4, 8, 2, 128
    pools, scales, tables, values = _paged(n, lens, window, sinks, 1, hkv, d, 16, int8)
    q = torch.randn((n, hkv * group, d), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
    kp, vp, ks, vs, tab = _cuda(*pools, *scales, tables)
    lse = torch.empty((n, hkv * group), device="cuda")
    plan = P.WindowDecodePlan(kp, vp, tab, torch.tensor(lens, dtype=torch.int32).cuda(), d ** -0.5, hkv * group, window,
                              sinks, k_scales=ks, v_scales=vs, lse_out=lse)
    out = plan.run(q.cuda()).clone()
    _check_decode(out, lse, q, values, lens, window, sinks, hkv, d ** -0.5, int8)
    for _ in range(3):                       # calls behind one another
        assert torch.equal(plan.run(q.cuda()), out)


@pytest.mark.parametrize("int8", [False, True])
def test_decode_agrees_with_the_unwindowed_decode(P, int8):
    """A window of the whole context: the split-KV decode's result within both tolerances."""
    lens, hkv, group, d, bs = [700, 33, 256], 4, 4, 128, 16
    pools, scales, tables, _ = _paged(5, lens, 2 ** 31 - 1, 0, 1, hkv, d, bs, int8)
    tables[tables == GARBAGE_ID] = pools[0].shape[0] - 1
    q = torch.randn((3, hkv * group, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    kp, vp, ks, vs, tab = _cuda(*pools, *scales, tables)
    if int8:
        ks, vs = ks.clamp(max=0.02), vs.clamp(max=0.02)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    a = P.paged_decode_attention(q, kp, vp, tab, ctx, d ** -0.5, k_scales=ks, v_scales=vs)
    b = P.paged_decode_attention_window(q, kp, vp, tab, ctx, d ** -0.5, 4096, k_scales=ks, v_scales=vs)
    assert float((a.double() - b.double()).abs().max()) <= (2e-2 if int8 else 1e-2)


@pytest.mark.parametrize("d,group", [(128, 8), (64, 3)])
def test_int8_scales_far_apart(P, d, group):
    """Tokens whose V scales differ by up to 2^60 and whose scores by hundreds: each
    head's weights have to stay in fp16's range whichever token leads."""
    lens, hkv, bs, scale = [400, 90, 257], 2, 16, 0.5
    pools, scales, tables, values = _paged(31, lens, 300, 4, 1, hkv, d, bs, True)
    gen = torch.Generator().manual_seed(9)
    factor = 2.0 ** torch.randint(-30, 31, scales[1].shape, generator=gen).float()
    scales[1] *= factor
    # keys grow along the sequence, so that the maximum moves again and again
    for s, x in enumerate(lens):
        t = torch.arange(x)
        rows = tables[s].long()[t // bs].clamp(min=0) * bs + t % bs
        scales[0].view(-1, hkv)[rows] *= (1 + t[:, None] / 20.0)
        for which in range(2):
            sc = scales[which].view(-1, hkv)[rows].double()
            values[s][which] = torch.nan_to_num(pools[which].view(-1, hkv, d)[rows].double() * sc[..., None])
    q = torch.randn((3, hkv * group, d), generator=gen).to(torch.bfloat16)
    kp, vp, ks, vs, tab = _cuda(*pools, *scales, tables)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    lse = torch.zeros((3, hkv * group), device="cuda")
    out = P.paged_decode_attention_window(q.cuda(), kp, vp, tab, ctx, scale, 300, 4, k_scales=ks, v_scales=vs, lse_out=lse)
    _check_decode(out, lse, q, values, lens, 300, 4, hkv, scale, True)


@pytest.mark.parametrize("int8", [False, True])
def test_bad_blocks_and_lengths_are_reported(P, int8):
    lens, window, sinks, hkv, group, d, bs = [100, 100, 100], 40, 4, 2, 4, 64, 16
    pools, scales, tables, values = _paged(9, lens, window, sinks, 1, hkv, d, bs, int8)
    q = torch.randn((3, hkv * group, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    tables[1, 5] = pools[0].shape[0]                       # a needed entry outside the pool
    kp, vp, ks, vs, tab = _cuda(*pools, *scales, tables)
    ctx = torch.tensor([100, 100, tables.shape[1] * bs + 1], dtype=torch.int32).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros((3, hkv * group), device="cuda")
    out = P.paged_decode_attention_window(q.cuda(), kp, vp, tab, ctx, 0.125, window, sinks, k_scales=ks, v_scales=vs,
                                          lse_out=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 1 | 4
    _check_decode(out[:1], lse[:1], q[:1], values[:1], lens[:1], window, sinks, hkv, 0.125, int8)
    assert torch.isfinite(out.float()).all() and not out[2].any()
    # the bad block's tokens are absent from the second sequence
    k, v = values[1]
    seen = R.visible(99, 100, window, sinks)
    seen[5 * bs:6 * bs] = False
    for h in range(hkv):
        o, _, absum, size, top = (x[0] for x in R.attend(q[1].double().view(hkv, group, d)[h][None], k[:, h], v[:, h],
                                                         seen[None], 0.125))
        assert ((out[1].cpu().double().view(hkv, group, d)[h] - o).abs()
                <= R.decode_tolerance(o, absum, size, d, int(seen.sum()), top if int8 else None)).all()


# starts (tokens before the new one), window, sinks, hkv, group, d, bs, rot (0: no turn), interleaved, packed
STEPS = [
    ([0], 1, 0, 1, 1, 64, 16, 64, False, True),
    ([17, 64, 100, 255], 64, 4, 2, 4, 64, 16, 64, False, True),
    ([0, 15, 16, 31, 47, 400], 40, 3, 2, 8, 128, 48, 64, True, True),
    ([999, 2047, 1], 1024, 4, 2, 6, 128, 16, 128, False, True),
    ([77, 300], 100, 0, 4, 1, 128, 32, 32, False, False),
    ([5, 130], 33, 2, 2, 3, 64, 16, 0, False, True),
    ([300 + i for i in range(20)], 128, 4, 8, 4, 128, 16, 128, False, True),
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("starts,window,sinks,hkv,group,d,bs,rot,inter,packed", STEPS)
def test_step_is_turn_write_attend(P, starts, window, sinks, hkv, group, d, bs, rot, inter, packed, int8):
    lens = [x + 1 for x in starts]
    n, hq, scale = len(starts), hkv * group, d ** -0.5
    pools, scales, tables, values = _paged(n + rot, lens, window, sinks, 1, hkv, d, bs, int8)
    gen = torch.Generator().manual_seed(4)
    qkv = torch.randn((n, 1, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16)
    start = torch.tensor(starts, dtype=torch.int32)
    # the new rows' places hold what a freed block would: they must come from the call
    for s, x in enumerate(starts):
        row = int(tables[s, x // bs]) * bs + x % bs
        for which in range(2):
            if int8:
                scales[which].view(-1, hkv)[row] = float("nan")
            else:
                pools[which].view(-1, hkv, d)[row] = float("nan")
    rope = P.Rope(rot, interleaved=inter) if rot else None
    kp, vp, ks, vs, tab, sp = _cuda(*pools, *scales, tables, start)
    x = qkv.cuda()
    q, k, v = x.split((hq, hkv, hkv), dim=2)
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    lse = torch.zeros((n, hq), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    out = P.paged_decode_step_window(k, v, sp, q[:, 0], kp, vp, tab, ctx, scale, window, sinks, rope=rope, k_scales=ks,
                                     v_scales=vs, lse_out=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # the pages are those of the rotary write (or the page write), bit for bit
    kp2, vp2, ks2, vs2 = _cuda(*pools, *scales)
    kc, vc = k.contiguous(), v.contiguous()
    if rope is not None:
        P.paged_kv_write_rope(q, k, v, rope, kp2, vp2, tab, sp, k_scales=ks2, v_scales=vs2)
    elif int8:
        P.paged_kv_write_int8(kc, vc, kp2, vp2, ks2, vs2, tab, sp)
    else:
        P.paged_kv_write(kc, vc, kp2, vp2, tab, sp)
    bits = (lambda t: t.view(torch.int16)) if not int8 else (lambda t: t)
    assert torch.equal(bits(kp), bits(kp2)) and torch.equal(bits(vp), bits(vp2))
    if int8:
        assert torch.equal(ks.view(torch.int32), ks2.view(torch.int32))
        assert torch.equal(vs.view(torch.int32), vs2.view(torch.int32))
    # attention over what the pages now hold, with the turned query in 64 bits
    qd = qkv[:, :, :hq].double()
    if rot:
        inv, mag = R.frequencies(rot)
        qd, _ = R.turn(qd, start.long()[:, None], inv, mag, inter)
    for s, y in enumerate(starts):
        row = int(tables[s, y // bs]) * bs + y % bs
        for which, (pool, sc) in enumerate(((kp, ks), (vp, vs))):
            new = pool.view(-1, hkv, d)[row].cpu().double()
            values[s][which][y] = new * sc.view(-1, hkv)[row].cpu().double()[:, None] if int8 else new
    _check_decode(out, lse, None, values, lens, window, sinks, hkv, scale, int8, qd[:, 0])


# prefix, chunk, window, sinks, hkv, group, d, bs
PREFILL = [
    ([0], 1, 1, 0, 1, 1, 64, 16),
    ([0, 5, 300], 37, 100, 3, 2, 4, 64, 16),
    ([0, 17], 64, 1, 0, 2, 4, 128, 16),
    ([130, 0, 700], 50, 16, 130, 1, 8, 128, 32),
    ([1000, 129], 200, 128, 4, 2, 4, 128, 16),
    ([511], 300, 250, 0, 1, 2, 128, 48),
    ([0], 700, 129, 20, 1, 16, 128, 16),
    ([40], 520, 2 ** 31 - 1, 0, 1, 4, 128, 16),
    ([40, 900], 130, 7, 2 ** 31 - 1, 1, 4, 64, 16),
    ([2000], 70, 300, 129, 2, 1, 64, 256),
]


@pytest.mark.parametrize("prefix,chunk,window,sinks,hkv,group,d,bs", PREFILL)
def test_prefill(P, prefix, chunk, window, sinks, hkv, group, d, bs):
    lens = [x + chunk for x in prefix]
    n, hq, scale = len(prefix), hkv * group, d ** -0.5
    pools, _, tables, values = _paged(chunk + n, lens, window, sinks, chunk, hkv, d, bs, False)
    gen = torch.Generator().manual_seed(8)
    q = torch.randn((n, chunk, hq, d), generator=gen).to(torch.bfloat16)
    kp, vp, tab = _cuda(*pools, tables)
    lse = torch.zeros((n, chunk, hq), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pre = torch.tensor(prefix, dtype=torch.int32).cuda()
    out = P.paged_prefill_attention_window(q.cuda(), kp, vp, tab, pre, scale, window, sinks, lse_out=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got, gl = out.cpu().double().view(n, chunk, hkv, group, d), lse.cpu().double().view(n, chunk, hkv, group)
    for s, x in enumerate(lens):
        seen = torch.stack([R.visible(prefix[s] + i, x, window, sinks) for i in range(chunk)])
        count = int(seen.sum(1).max())
        for h in range(hkv):
            o, ls, absum, size, _ = R.attend(q[s].double().view(chunk, hkv, group, d)[:, h], values[s][0][:, h],
                                          values[s][1][:, h], seen, scale)
            assert torch.isfinite(got[s, :, h]).all()
            over = (got[s, :, h] - o).abs() - R.prefill_tolerance(o, absum, size, d, count)
            assert (over <= 0).all(), (s, h, float(over.max()))
            over = (gl[s, :, h] - ls).abs() - R.lse_tolerance(ls, size, d, count)
            assert (over <= 0).all(), (s, h, float(over.max()))


def test_prefill_of_many_units_and_odd_addresses(P):
    """More units than CTAs, some of bad length among them, and an output on a
    16-byte boundary: the same bits as one sequence at a time, wide stores or not."""
    hkv, group, d, bs, window, sinks, chunk = 8, 4, 128, 16, 70, 5, 200
    prefix = [0, 300, 5, 77, 1000, 16, 450, 123]
    lens = [x + chunk for x in prefix]
    pools, _, tables, _ = _paged(6, lens, window, sinks, chunk, hkv, d, bs, False)
    q = torch.randn((8, chunk, hkv * group, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor(prefix, dtype=torch.int32).cuda()
    pre[2], pre[5] = -1, tables.shape[1] * bs
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    P.paged_prefill_attention_window(q, kp, vp, tab, pre, d ** -0.5, window, sinks, out=out, dev_status=st)
    odd = torch.full((q.numel() + 8,), 3.0, dtype=torch.bfloat16, device="cuda")[8:].view(q.shape)
    assert odd.data_ptr() % 32 == 16
    P.paged_prefill_attention_window(q, kp, vp, tab, pre, d ** -0.5, window, sinks, out=odd)
    torch.cuda.synchronize()
    assert int(st.item()) == 4 and torch.equal(out, odd)
    assert (out[[2, 5]] == 3.0).all()                      # a bad length leaves its rows as they were
    for s in (0, 1, 3, 4, 6, 7):
        one = P.paged_prefill_attention_window(q[s:s + 1], kp, vp, tab[s:s + 1], pre[s:s + 1], d ** -0.5, window, sinks)
        assert torch.equal(one[0], out[s]), s


@pytest.mark.parametrize("d,hkv,group,chunk,window,sinks", [(128, 8, 4, 512, 500, 4), (64, 4, 2, 300, 133, 20),
                                                           (128, 2, 8, 130, 77, 0), (128, 1, 16, 70, 2 ** 31 - 1, 0)])
def test_prefill_rows_do_not_depend_on_the_batch(P, d, hkv, group, chunk, window, sinks):
    """A row's bits are the same whatever else is in the call (and so whether its unit
    was computed whole or as two halves)."""
    gen = torch.Generator().manual_seed(chunk)
    n, bs = 20, 16
    prefix = torch.randint(0, 1500, (n,), generator=gen, dtype=torch.int32)
    width = (1500 + chunk) // bs + 1
    pools = [torch.randn((n * width + 1, bs, hkv, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    tables = torch.randperm(n * width, generator=gen).to(torch.int32).view(n, width).cuda()
    # large scores, so that maxima move
    q = (torch.randn((n, chunk, hkv * group, d), generator=gen) * 4).to(torch.bfloat16).cuda()
    prefix = prefix.cuda()

    def call(a, b):
        lse = torch.empty((b - a, chunk, hkv * group), device="cuda")
        out = P.paged_prefill_attention_window(q[a:b].contiguous(), *pools, tables[a:b].contiguous(), prefix[a:b].contiguous(),
                                               d ** -0.5, window, sinks, lse_out=lse)
        return out, lse

    whole = call(0, n)
    assert torch.isfinite(whole[0].float()).all()
    for m in (1, 2, 3, 5, 11):
        for a in range(0, n - m, m + 2):
            for x, y in zip(call(a, a + m), whole):
                assert torch.equal(x, y[a:a + m]), (m, a)


def test_prefill_wait_runs_out_then_recovers(P):
    """With a limit of 1 ns on its pipeline waits the kernel reports the timeout and
    returns; the next call on the stream is right."""
    hkv, group, d, bs, window, sinks, chunk = 4, 4, 128, 16, 300, 4, 300
    lens = [chunk + 500, chunk]
    pools, _, tables, _ = _paged(6, lens, window, sinks, chunk, hkv, d, bs, False)
    q = torch.randn((2, chunk, hkv * group, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor([500, 0], dtype=torch.int32).cuda()
    run = lambda st: P.paged_prefill_attention_window(q, kp, vp, tab, pre, d ** -0.5, window, sinks, dev_status=st)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(st)
    lib = P.load_library()
    try:
        lib.pkv_set_pipeline_wait_ns(1)
        for _ in range(5):                                 # at least one of them must run out
            run(st)
        torch.cuda.synchronize()
    finally:
        lib.pkv_set_pipeline_wait_ns(0)
    assert int(st.item()) & 16
    st.zero_()
    got = run(st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(got, want)


def test_prefill_reports_bad_blocks_and_lengths(P):
    prefix, chunk, window, sinks, hkv, group, d, bs = [200, 200, 200], 40, 50, 4, 1, 4, 64, 16
    pools, _, tables, _ = _paged(3, [x + chunk for x in prefix], window, sinks, chunk, hkv, d, bs, False)
    q = torch.randn((3, chunk, 4, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    tables[1, 12] = pools[0].shape[0]
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor([200, 200, tables.shape[1] * bs], dtype=torch.int32).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = P.paged_prefill_attention_window(q, kp, vp, tab, pre, 0.125, window, sinks, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 1 | 4 and torch.isfinite(out[:2].float()).all()


def test_plan_stream_and_graph(P):
    """A plan's steps of two layers, captured once and replayed with new inputs in
    place, on another stream than the tensors' own."""
    lens, window, sinks, hkv, group, d, bs = [50, 300, 2], 64, 4, 2, 4, 128, 16
    hq, n = hkv * group, 3
    rope = P.Rope(128)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    start = ctx - 1
    layers = []
    for layer in range(2):
        pools, _, tables, _ = _paged(20 + layer, lens, window, sinks, 1, hkv, d, bs, False)
        kp, vp, tab = _cuda(*pools, tables)
        layers.append((P.WindowDecodePlan(kp, vp, tab, ctx, d ** -0.5, hq, window, sinks, rope=rope), kp, vp, tab))
    gen = torch.Generator().manual_seed(6)
    xs = [torch.randn((n, 1, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    x = xs[0].clone()
    q, k, v = x.split((hq, hkv, hkv), dim=2)

    def step():
        return [plan.run(q[:, 0], k, v, start) for plan, *_ in layers]

    want = []
    for y in xs:
        x.copy_(y)
        want.append([o.clone() for o in step()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for y, w in zip(xs, want):
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    side = torch.cuda.Stream()
    x.copy_(xs[0])
    side.wait_stream(torch.cuda.current_stream())
    plan, kp, vp, tab = layers[0]
    out = P.paged_decode_step_window(k, v, start, q[:, 0], kp, vp, tab, ctx, d ** -0.5, window, sinks, rope=rope, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0][0])


def test_wrappers_refuse_mismatched_tensors(P):
    hkv, group, d, bs = 2, 4, 64, 16
    pools, _, tables, _ = _paged(1, [30, 40], 8, 0, 1, hkv, d, bs, False)
    kp, vp, tab = _cuda(*pools, tables)
    q = torch.zeros((2, 8, d), dtype=torch.bfloat16, device="cuda")
    ctx = torch.tensor([30, 40], dtype=torch.int32, device="cuda")
    new = torch.zeros((2, 1, hkv, d), dtype=torch.bfloat16, device="cuda")
    rope = P.Rope(64)
    f, g = P.paged_decode_attention_window, P.paged_decode_step_window
    for bad in (lambda: f(q, kp, vp, tab, ctx[:1], 0.1, 8), lambda: f(q, kp, vp[:-1], tab, ctx, 0.1, 8),
                lambda: f(q[:1], kp, vp, tab, ctx, 0.1, 8), lambda: f(q, kp, vp, tab, ctx, 0.1, 8, out=q[:, :4]),
                lambda: f(q, kp, vp, tab, ctx, 0.1, 8, lse_out=torch.zeros((2, 7), device="cuda")),
                lambda: f(q, kp, vp, tab, ctx, 0.1, -1), lambda: f(q.float(), kp, vp, tab, ctx, 0.1, 8),
                lambda: g(new[:, :, :1], new, ctx - 1, q, kp, vp, tab, ctx, 0.1, 8),
                lambda: g(new, new, (ctx - 1)[:1], q, kp, vp, tab, ctx, 0.1, 8),
                lambda: g(torch.cat((new, new), 1), torch.cat((new, new), 1), ctx - 1, q, kp, vp, tab, ctx, 0.1, 8),
                lambda: g(new, new, ctx - 1, q, kp, vp, tab, ctx, 0.1, 8, rope=P.Rope(128)),
                lambda: g(new, new, ctx - 1, q, kp, vp, tab, ctx, 0.1, 8, rope=P.Rope(64, device="cpu")),
                lambda: P.WindowDecodePlan(kp, vp, tab, ctx, 0.1, 8, 8, rope=rope).run(q),
                lambda: P.WindowDecodePlan(kp, vp, tab, ctx, 0.1, 8, 8).run(q, start_pos=ctx),
                lambda: P.paged_prefill_attention_window(q[:, None], kp, vp, tab, ctx, 0.1, 8, out=q),
                lambda: P.paged_kv_write_rope(q[:, None], new, new, rope, kp, vp, tab, ctx, q_out=q)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(P.PagedKVError) as e:
        f(q, kp, vp, tab, ctx, 0.1, 0)                     # a window holds the query itself
    assert e.value.status == 1


def test_native_and_python_marshalling_agree(P, monkeypatch):
    """The calls give the same bits through either part of the binding."""
    assert P._native is not None
    lens, window, sinks, hkv, group, d, bs = [50, 300], 64, 4, 2, 4, 128, 16
    hq, n = hkv * group, 2
    pools, _, tables, _ = _paged(2, lens, window, sinks, 40, hkv, d, bs, False)
    x = torch.randn((n, 40, hq + 2 * hkv, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    rope = P.Rope(128)
    got = []
    for native in (P._native, None):
        monkeypatch.setattr(P, "_native", native)
        kp, vp, tab = _cuda(*pools, tables)
        q, k, v = x.split((hq, hkv, hkv), dim=2)
        qt = P.paged_kv_write_rope(q, k, v, rope, kp, vp, tab, ctx - 40)
        o = P.paged_prefill_attention_window(qt, kp, vp, tab, ctx - 40, d ** -0.5, window, sinks)
        plan = P.WindowDecodePlan(kp, vp, tab, ctx, d ** -0.5, hq, window, sinks, rope=rope)
        step = plan.run(q[:, -1], k[:, -1:], v[:, -1:], ctx - 1).clone()
        plain = P.WindowDecodePlan(kp, vp, tab, ctx, d ** -0.5, hq, window, sinks).run(qt[:, -1].contiguous())
        got.append((qt, o, step, plain.clone(), kp.view(torch.int16), vp.view(torch.int16)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("int8", [False])
def test_prompt_in_chunks_then_steps(P, int8):
    """A run of the operators as a server uses them: a prompt written and attended
    in chunks, then steps, blocks behind the window freed (their table entries
    overwritten) as the sequence grows; against one 64-bit attention over all."""
    window, sinks, hkv, group, d, bs, rot = 48, 4, 2, 4, 64, 16, 32
    hq, scale, n, prompt, steps = hkv * group, d ** -0.5, 2, [70, 45], 30
    total = [p + steps for p in prompt]
    gen = torch.Generator().manual_seed(44)
    qkv = [torch.randn((t, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16) for t in total]
    width = max(-(-t // bs) for t in total)
    n_blocks = n * width
    pool = torch.full((n_blocks + 1, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kp, vp = pool, pool.clone()
    tables = torch.randperm(n_blocks, generator=gen).to(torch.int32).view(n, width)
    inv, mag = R.frequencies(rot)
    rope, st = P.Rope(rot), torch.zeros(1, dtype=torch.int32, device="cuda")

    def free_behind(next_pos):
        for s in range(n):
            for b in range(width):
                toks = range(b * bs, (b + 1) * bs)
                if not any(t < sinks or t > next_pos[s] - window for t in toks):
                    tables[s, b] = GARBAGE_ID
        return tables.cuda()

    got = [[None] * t for t in total]
    chunk = 23
    for s in range(n):                       # each prompt in chunks
        for c0 in range(0, prompt[s], chunk):
            m = min(chunk, prompt[s] - c0)
            tab = tables[s:s + 1].cuda()
            x = qkv[s][None, c0:c0 + m].cuda()
            q, k, v = x.split((hq, hkv, hkv), dim=2)
            pre = torch.tensor([c0], dtype=torch.int32, device="cuda")
            qt = P.paged_kv_write_rope(q, k, v, rope, kp, vp, tab, pre, dev_status=st)
            o = P.paged_prefill_attention_window(qt, kp, vp, tab, pre, scale, window, sinks, dev_status=st)
            for i in range(m):
                got[s][c0 + i] = o[0, i].cpu().double()
    start = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    ctx = start + 1
    tab = free_behind(prompt)
    plan = P.WindowDecodePlan(kp, vp, tab, ctx, scale, hq, window, sinks, rope=rope, dev_status=st)
    for i in range(steps):
        pos = [p + i for p in prompt]
        tab.copy_(free_behind(pos))
        x = torch.stack([qkv[s][pos[s]] for s in range(n)])[:, None].cuda()
        q, k, v = x.split((hq, hkv, hkv), dim=2)
        o = plan.run(q[:, 0], k, v, start)
        for s in range(n):
            got[s][pos[s]] = o[s].cpu().double()
        start += 1
        ctx += 1
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for s in range(n):
        t = torch.arange(total[s])
        x = qkv[s].double()
        qt, qsize = R.turn(x[:, :hq], t, inv, mag, False)
        kt, _ = R.turn(x[:, hq:hq + hkv], t, inv, mag, False)
        kt, vt = kt.to(torch.bfloat16).double(), x[:, hq + hkv:]
        seen = torch.stack([R.visible(i, total[s], window, sinks) for i in range(total[s])])
        out = torch.stack(got[s]).view(total[s], hkv, group, d)
        for h in range(hkv):
            o, _, absum, size, _ = R.attend(qt.view(total[s], hkv, group, d)[:, h], kt[:, h], vt[:, h], seen, scale)
            # queries of the chunks, and keys where the two sides round across a step, are
            # off by up to a bf16 rounding each: 2 (u16 + u16) more on every score
            tol = R.prefill_tolerance(o, absum, size, d, window + sinks) + absum * 4 * R.U16 * size[..., None]
            assert ((out[:, h] - o).abs() <= tol).all()
