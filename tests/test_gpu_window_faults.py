"""The windowed and rotary calls where something is wrong with a call or its
neighbour: waits that run out with another call behind them, chunks that run past
the table, and the calls around them, which have to stay right."""
import threading

import pytest
import torch

import window_reference as R

from test_gpu_window import GARBAGE_ID, P, _check_decode, _cuda, _paged  # noqa: F401  (P: the fixture)

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


def _quantised(x):
    """Rows [..., D] (64 bits) as the values of their int8 codes."""
    step = x.abs().amax(-1, keepdim=True) / 127
    return torch.where(step > 0, torch.round(x / step.clamp(min=1e-300)).clamp(-127, 127) * step, torch.zeros_like(x))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("hkv,group,d", [(2, 4, 64), (4, 6, 128)])
def test_step_with_bad_positions_blocks_and_inactive_sequences(P, hkv, group, d, int8):  # noqa: F811
    """A new row without a place is reported, written nowhere and not attended; inactive
    sequences share the scratch block; the other sequences and blocks are as ever."""
    bs, window, sinks, hq, scale = 16, 40, 4, hkv * group, d ** -0.5
    #       good  before 0  past the table  bad block  inactive (two)
    lens = [100, 100, 70, 65, 1, 3]
    n = len(lens)
    pools, scales, tables, values = _paged(d, lens, window, sinks, 1, hkv, d, bs, int8)
    scratch, bad = pools[0].shape[0] - 1, 3
    start = torch.tensor([x - 1 for x in lens], dtype=torch.int32)
    start[1], start[2] = -1, tables.shape[1] * bs
    tables[bad, 64 // bs] = scratch + 1
    tables[4:] = scratch
    gen = torch.Generator().manual_seed(7)
    x = torch.randn((n, 1, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16)
    q, k, v = x.cuda().split((hq, hkv, hkv), dim=2)
    kp, vp, ks, vs, tab, sp = _cuda(*pools, *scales, tables, start)
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros((n, hq), device="cuda")
    out = P.paged_decode_step_window(k, v, sp, q[:, 0], kp, vp, tab, ctx, scale, window, sinks, k_scales=ks, v_scales=vs,
                                     lse_out=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 1 | 2
    # every block but the scratch one and the good sequence's row is as it was
    place = int(tables[0, 99 // bs]) * bs + 99 % bs
    for got, was in ((kp, pools[0]), (vp, pools[1]), (ks, scales[0]), (vs, scales[1])):
        if was is not None:
            a, b = (t.cpu().contiguous().view(torch.uint8).view(scratch + 1, bs, -1)[:scratch].reshape(scratch * bs, -1) for t in (got, was))
            kept = torch.arange(scratch * bs) != place
            assert torch.equal(a[kept], b[kept])
    # the good sequence sees its new row, those without a position what the pages held before
    for which, new in enumerate((k, v)):
        new = new[0, 0].cpu().double()
        values[0][which][99] = _quantised(new) if int8 else new
    pick = [0, 1, 2]
    _check_decode(out[pick], lse[pick], x[pick, 0, :hq], [values[s] for s in pick], [lens[s] for s in pick], window, sinks, hkv,
                  scale, int8)
    # the bad block's tokens are absent
    seen = R.visible(64, 65, window, sinks)
    seen[64:] = False
    for h in range(hkv):
        o, _, absum, size, top = (t[0] for t in R.attend(x[bad, 0, :hq].double().view(hkv, group, d)[h][None], values[bad][0][:, h],
                                                         values[bad][1][:, h], seen[None], scale))
        assert ((out[bad].cpu().double().view(hkv, group, d)[h] - o).abs()
                <= R.decode_tolerance(o, absum, size, d, int(seen.sum()), top if int8 else None)).all()


@pytest.mark.parametrize("native", [True, False])
def test_calls_from_two_threads_on_two_streams(P, native, monkeypatch):  # noqa: F811
    """Two threads, each with pages, plan and stream of its own, run write, chunk and
    steps at the same time: the bits of the same calls one after another."""
    if not native:
        monkeypatch.setattr(P, "_native", None)
    bs, window, sinks, hkv, group, d, chunk, steps = 16, 70, 4, 4, 4, 128, 90, 40
    hq, scale, rope = hkv * group, d ** -0.5, P.Rope(d)
    # (a sequence more in the second: other cluster and unit counts)
    inputs = []
    for n in (2, 3):
        gen = torch.Generator().manual_seed(n)
        width = -(-(chunk + steps) // bs)
        tab = torch.randperm(n * width, generator=gen).to(torch.int32).view(n, width).cuda()
        xs = torch.randn((steps + 1, n, chunk, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16).cuda()
        inputs.append((n, width, tab, xs))

    def work(n, width, tab, xs):
        kp, vp = (torch.zeros((n * width + 1, bs, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        start = torch.zeros(n, dtype=torch.int32, device="cuda")
        q, k, v = xs[0].split((hq, hkv, hkv), dim=2)
        qt = P.paged_kv_write_rope(q, k, v, rope, kp, vp, tab, start)
        outs = [P.paged_prefill_attention_window(qt, kp, vp, tab, start, scale, window, sinks)]
        start += chunk
        ctx = start + 1
        plan = P.WindowDecodePlan(kp, vp, tab, ctx, scale, hq, window, sinks, rope=rope)
        for x in xs[1:]:
            q, k, v = x[:, :1].split((hq, hkv, hkv), dim=2)
            outs.append(plan.run(q[:, 0], k, v, start).clone())
            start += 1
            ctx += 1
        return outs + [kp, vp]

    want = [work(*i) for i in inputs]
    torch.cuda.synchronize()
    got, errors, gate = [None, None], [], threading.Barrier(2)

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gate.wait(30)
                got[i] = work(*inputs[i])
            stream.synchronize()
        except Exception as e:      # for the test's own thread
            errors.append(e)

    for _ in range(3):
        threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not errors, errors
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_chunks_written_then_steps_over_int8_pages(P):  # noqa: F811
    """Prompts written in chunks into int8 pages, then steps, one of them captured and
    replayed, blocks behind the window freed as the sequences grow; against one 64-bit
    attention over what the pages stand for."""
    window, sinks, hkv, group, d, bs, rot, chunk = 48, 4, 2, 4, 64, 16, 32, 23
    hq, scale, prompt, steps = hkv * group, d ** -0.5, [70, 45, 20], 24
    n, total = len(prompt), [p + steps for p in prompt]
    gen = torch.Generator().manual_seed(45)
    qkv = [torch.randn((t, hq + 2 * hkv, d), generator=gen).to(torch.bfloat16) for t in total]
    width = max(-(-t // bs) for t in total)
    pools = [torch.full((n * width + 1, bs, hkv, d), 127, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.full((n * width + 1, bs, hkv), float("nan"), device="cuda") for _ in range(2)]
    tables = torch.randperm(n * width, generator=gen).to(torch.int32).view(n, width)
    whole = tables.clone()
    rope, st = P.Rope(rot), torch.zeros(1, dtype=torch.int32, device="cuda")
    for s in range(n):
        for c0 in range(0, prompt[s], chunk):
            x = qkv[s][None, c0:min(c0 + chunk, prompt[s])].cuda()
            q, k, v = x.split((hq, hkv, hkv), dim=2)
            P.paged_kv_write_rope(q, k, v, rope, *pools, tables[s:s + 1].cuda(), torch.tensor([c0], dtype=torch.int32, device="cuda"),
                                  k_scales=scales[0], v_scales=scales[1], dev_status=st)
    start = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    ctx, tab = start + 1, tables.cuda()
    lse = torch.zeros((n, hq), device="cuda")
    plan = P.WindowDecodePlan(*pools, tab, ctx, scale, hq, window, sinks, rope=rope, k_scales=scales[0], v_scales=scales[1],
                              lse_out=lse, dev_status=st)
    x = torch.zeros((n, 1, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split((hq, hkv, hkv), dim=2)
    graph, got = None, []
    for i in range(steps):
        for s in range(n):
            for b in range(width):
                if not any(t < sinks or t > prompt[s] + i - window for t in range(b * bs, (b + 1) * bs)):
                    tables[s, b] = GARBAGE_ID
        tab.copy_(tables)
        x.copy_(torch.stack([qkv[s][prompt[s] + i] for s in range(n)])[:, None])
        if i == steps // 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                plan.run(q[:, 0], k, v, start)
        if graph is None:
            plan.run(q[:, 0], k, v, start)
        else:
            graph.replay()
        got.append((plan.out.cpu(), lse.cpu()))
        start += 1
        ctx += 1
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    inv, mag = R.frequencies(rot)
    for s in range(n):
        t = torch.arange(total[s])
        rows = whole[s].long()[t // bs] * bs + t % bs
        held = [p.cpu().view(-1, hkv, d)[rows].double() * sc.cpu().view(-1, hkv)[rows].double()[..., None] for p, sc in zip(pools, scales)]
        # the pages: nearest codes of the turned keys and of the values
        kt, ksize = R.turn(qkv[s][:, hq:hq + hkv].double(), t, inv, mag, False)
        for x64, size, page, sc in ((kt, ksize, held[0], scales[0]), (qkv[s][:, hq + hkv:].double(), 0, held[1], scales[1])):
            step = sc.cpu().view(-1, hkv)[rows].double()[..., None]
            assert ((page - x64).abs() <= step * (0.5 + 2.0 ** -14) + R.TURN * size).all()
        for i in range(steps):
            p = prompt[s] + i
            qt, _ = R.turn(qkv[s][p:p + 1, :hq].double(), torch.tensor([p]), inv, mag, False)
            _check_decode(got[i][0][s:s + 1], got[i][1][s:s + 1], None, [[h[:p + 1] for h in held]], [p + 1], window, sinks, hkv,
                          scale, True, qt)
