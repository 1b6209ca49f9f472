"""The calls for ragged batches over values that are no numbers, that a sequence must not see, or
whose scales are far apart; head counts and alignments at their limits; the way that a call takes."""
import pytest
import torch

from batch_reference import Paged, check_rows
from test_gpu_batch import P, _ints, _shared_case, _status, rows_impl      # noqa: F401 - fixtures

pytestmark = pytest.mark.gpu


def _rows_of(table, first, stop, bs):
    t = torch.arange(first, stop)
    return table[t // bs].long() * bs + t % bs


# ---- tokens behind a sequence's end, within its group's prefix ---------------------------------

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,group", [(128, 4), (64, 8)])
@pytest.mark.parametrize("seen", [False, True])
def test_shared_tokens_behind_a_sequence_are_not_seen(P, int8, d, group, seen, rows_impl):     # noqa: F811
    """Tokens of a prefix that are not written yet (NaN, infinities, scales of any size) reach none of
    the sequences that end before them, whether another one of the group sees them or not."""
    hkv, bs, scale, end, prefix = 2, 16, d ** -0.5, 650, 700
    pages, tables, ctx, starts, ptables, values = _shared_case([9, 5], [prefix, 300], [20] * 14, 0, hkv, d, bs, int8, 4)
    ctx[:9] = [0, 1, 127, 128, 129, 640, end - 1, end, prefix + 20 if seen else 500]
    rows = _rows_of(ptables[0], end, prefix, bs)
    for which in range(2):
        if int8:
            s = pages.scales[which].view(-1, hkv)
            s[rows[:20]], s[rows[20:30]], s[rows[30:]] = 1e30, float("nan"), float("inf")
        else:
            v = pages.pools[which].view(-1, hkv, d)
            v[rows[:20]], v[rows[20:]] = float("inf"), float("nan")
    kp, vp, ks, vs = pages.cuda()
    q = torch.randn((14, hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    lse, st = torch.full((14, hkv * group), 7.0, device="cuda"), _status()
    out = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints([prefix, 300]),
                                          scale, k_scales=ks, v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s in range(14):
        if s == 8 and seen:
            assert out[s].isnan().all() and lse[s].isnan().all()
        else:
            check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *(v[:ctx[s]] for v in values[s]), scale, int8)


# ---- NaN that a row sees -------------------------------------------------------------------------

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("keys", [[40, 128, 100], [1000, 40, 3100]])       # runs of one tile, and runs that CTAs share
@pytest.mark.parametrize("where", ["query", "key", "value"])
def test_cross_passes_nan_on(P, int8, keys, where, rows_impl):     # noqa: F811
    """A NaN in a query, a key or a value makes NaN of what it reaches, and of nothing else."""
    hkv, group, d, bs, scale, n_q = 2, 3, 64, 16, 0.125, [50, 3, 90]
    pages = Paged(7, sum(-(-x // bs) for x in keys) + 1, hkv, d, bs, int8)
    added = [pages.add(0, x, max(-(-y // bs) for y in keys)) for x in keys]
    starts = [0, 50, 53, 143]
    q = torch.randn((143, hkv * group, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    bad = torch.zeros((143, hkv * group, d), dtype=torch.bool)          # outputs that are no numbers
    bad_lse = torch.zeros((143, hkv * group), dtype=torch.bool)
    if where == "query":
        for row, head in ((0, 0), (49, 5), (51, 2), (53, 3), (142, 4)):
            q[row, head, (row * 7) % d] = float("nan")
            bad[row, head] = bad_lse[row, head] = True
    else:
        # a key or value of each sequence's second kv head (int8: its scale), in the last token
        for s, x in enumerate(keys):
            at = _rows_of(added[s][0], x - 1, x, bs)
            if int8:
                pages.scales[where == "value"].view(-1, hkv)[at, 1] = float("nan")
            else:
                pages.pools[where == "value"].view(-1, hkv, d)[at, 1, 5] = float("nan")
        if where == "key":
            bad[:, group:] = bad_lse[:, group:] = True
        elif int8:
            bad[:, group:] = True
        else:
            bad[:, group:, 5] = True
    kp, vp, ks, vs = pages.cuda()
    lse, st = torch.full((143, hkv * group), 7.0, device="cuda"), _status()
    out = P.paged_cross_attention(q.cuda(), _ints(starts), kp, vp, torch.stack([t for t, _ in added]).cuda(), _ints(keys), scale,
                                  k_scales=ks, v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    assert torch.equal(out.cpu().isnan(), bad) and torch.equal(lse.cpu().isnan(), bad_lse)
    # the others are right: beside the NaN, whose places take the values without it
    clean = q.nan_to_num(0.0)
    for s in range(3):
        a, b = starts[s], starts[s + 1]
        o, ls = out[a:b].cpu().clone(), lse[a:b].cpu().clone()
        k, v = (x.nan_to_num(0.0) for x in added[s][1])
        sc = torch.einsum("mhgd,nhd->mhgn", clean[a:b].double().view(b - a, hkv, group, d), k) * scale
        ref = torch.einsum("mhgn,nhd->mhgd", torch.softmax(sc, -1), v).reshape(b - a, hkv * group, d)
        o = torch.where(bad[a:b], ref.to(torch.bfloat16), o)
        ls = torch.where(bad_lse[a:b], torch.logsumexp(sc, -1).reshape(b - a, -1).float(), ls)
        check_rows(o, ls, clean[a:b], k, v, scale, int8)


@pytest.mark.parametrize("int8", [False, True])
def test_shared_passes_nan_on(P, int8, rows_impl):     # noqa: F811
    """The same behind a prefix: a NaN query, in a sequence of a long and of a short group."""
    hkv, group, d, bs, scale = 2, 4, 128, 16, 0.09
    pages, tables, ctx, starts, ptables, values = _shared_case([20, 1], [2500, 60], [i % 5 for i in range(21)], 1, hkv, d, bs, int8, 6)
    kp, vp, ks, vs = pages.cuda()
    q = torch.randn((22, hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    bad = torch.zeros((22, hkv * group), dtype=torch.bool)
    for s, head in ((0, 1), (1, 0), (7, 7), (21, 3)):
        q[s, head, 9] = float("nan")
        bad[s, head] = True
    lse, st = torch.full((22, hkv * group), 7.0, device="cuda"), _status()
    out = P.paged_decode_attention_shared(q.cuda(), kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints([2500, 60]),
                                          scale, k_scales=ks, v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    assert torch.equal(out.cpu().isnan(), bad[..., None].expand(out.shape)) and torch.equal(lse.cpu().isnan(), bad)
    for s in range(22):
        if not bad[s].any():
            check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, int8)


# ---- scales far apart ------------------------------------------------------------------------------

def _most(impl, scales):
    """What check_rows adds for values far below the largest scale: nothing one by one."""
    return 0.0 if impl == "one" else float(scales.max())


@pytest.mark.parametrize("ramp", [(-6, 2), (2, -6), (-20, -14), (25, 30)])
@pytest.mark.parametrize("d", [64, 128])
def test_cross_over_scales_one_by_one(P, d, ramp, monkeypatch):     # noqa: F811
    """V scales over many orders of magnitude: one by one they join the weights, so that the bound has
    no term of the largest scale."""
    monkeypatch.setenv("PKV_ROWS_IMPL", "one")
    hkv, group, bs, scale, n = 2, 3, 16, d ** -0.5, 900
    pages = Paged(9, 60, hkv, d, bs, True)
    row, (k, _) = pages.add(0, n, 60)
    slots = _rows_of(row, 0, n, bs)
    flat = pages.scales[1].view(-1, hkv)
    flat[slots] = (flat[slots].double() * 10.0 ** torch.linspace(*ramp, n)[:, None]).float()
    v = pages.pools[1].view(-1, hkv, d)[slots].double() * flat[slots].double()[..., None]
    kp, vp, ks, vs = pages.cuda()
    q = torch.randn((40, hkv * group, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    lse = torch.empty((40, hkv * group), device="cuda")
    out = P.paged_cross_attention(q, _ints([0, 40]), kp, vp, row.view(1, -1).cuda(), _ints([n]), scale, k_scales=ks, v_scales=vs, lse_out=lse)
    check_rows(out, lse, q, k, v, scale, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("small_first", [False, True])
def test_cross_that_sees_the_small_scales_alone(P, d, small_first, rows_impl):     # noqa: F811
    """Queries whose weight lies on one key, of a V scale 2^-28 of the others': rows at once hold its
    values to 2^-24 of the largest scale, rows one by one to 2^-11 of themselves."""
    hkv, group, bs, scale, n = 2, 3, 16, d ** -0.5, 600
    pages = Paged(11, 40, hkv, d, bs, True)
    row, _ = pages.add(0, n, 40)
    slots = _rows_of(row, 0, n, bs)
    small = torch.arange(n) == (0 if small_first else n - 1)
    gen = torch.Generator().manual_seed(1)
    codes, sk, sv = pages.pools[0].view(-1, hkv, d), pages.scales[0].view(-1, hkv), pages.scales[1].view(-1, hkv)
    codes[slots] = torch.where(small[:, None, None], torch.randint(80, 128, (n, hkv, d), generator=gen),
                               torch.randint(-127, -79, (n, hkv, d), generator=gen)).to(torch.int8)
    sk[slots] = 0.02
    sv[slots] = torch.where(small[:, None], 0.01 * 2.0 ** -28, 0.01).expand(n, hkv).contiguous()
    k = codes[slots].double() * sk[slots].double()[..., None]
    v = pages.pools[1].view(-1, hkv, d)[slots].double() * sv[slots].double()[..., None]
    kp, vp, ks, vs = pages.cuda()
    q = (torch.rand((170, hkv * group, d), generator=gen) + 3).to(torch.bfloat16).cuda()     # scores 70 apart or more
    lse = torch.empty((170, hkv * group), device="cuda")
    out = P.paged_cross_attention(q, _ints([0, 170]), kp, vp, row.view(1, -1).cuda(), _ints([n]), scale, k_scales=ks, v_scales=vs, lse_out=lse)
    check_rows(out, lse, q, k, v, scale, True, _most(rows_impl, sv[slots]))


# ---- heads and alignment ---------------------------------------------------------------------------

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [9, 11, 13, 15, 16])
def test_cross_of_many_heads_and_outputs_of_16_bytes(P, group, d, int8):     # noqa: F811
    """9 to 16 query heads per kv head, which do not divide a product's 128 rows; whole and cut runs;
    outputs and queries aligned to 16 bytes and no more."""
    hkv, bs, scale, n_q, keys = 2, 16, d ** -0.5, [1, 40, 3], [700, 2300, 100]
    hq, total = hkv * group, 44
    pages = Paged(group, sum(-(-x // bs) for x in keys) + 1, hkv, d, bs, int8)
    added = [pages.add(0, x, 150) for x in keys]
    kp, vp, ks, vs = pages.cuda()
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(total * hq * d + 8, generator=gen).to(torch.bfloat16).cuda()[8:].view(total, hq, d)
    out = torch.zeros(total * hq * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(total, hq, d)
    assert q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    lse, st = torch.zeros((total, hq), device="cuda"), _status()
    starts, tables = _ints([0, 1, 41, 44]), torch.stack([t for t, _ in added]).cuda()
    P.paged_cross_attention(q, starts, kp, vp, tables, _ints(keys), scale, k_scales=ks, v_scales=vs, out=out, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s, (a, b) in enumerate(((0, 1), (1, 41), (41, 44))):
        check_rows(out[a:b], lse[a:b], q[a:b], *added[s][1], scale, int8)


@pytest.mark.parametrize("int8", [False, True])
def test_rows_into_outputs_of_16_bytes(P, int8, rows_impl):     # noqa: F811
    """Runs of one tile, which are whole, and outputs aligned to 16 bytes and no more, both calls."""
    hkv, group, d, bs, scale = 2, 4, 64, 16, 0.125
    pages, tables, ctx, starts, ptables, values = _shared_case([30, 5], [100, 128], [i % 20 for i in range(35)], 0, hkv, d, bs, int8, 8)
    kp, vp, ks, vs = pages.cuda()
    q = torch.randn((35, hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    out = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(q.shape)
    lse = torch.zeros((35, hkv * group), device="cuda")
    prefixes = _ints([100, 128])
    P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), prefixes, scale, k_scales=ks,
                                    v_scales=vs, out=out, lse_out=lse)
    for s in range(35):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, int8)
    P.paged_cross_attention(q, _ints(starts), kp, vp, ptables.cuda(), prefixes, scale, k_scales=ks, v_scales=vs, out=out, lse_out=lse)
    for (a, b), n in zip(((0, 30), (30, 35)), (100, 128)):
        check_rows(out[a:b], lse[a:b], q[a:b], *(x[:n] for x in values[a]), scale, int8)


# ---- the way that a call takes ---------------------------------------------------------------------

@pytest.mark.parametrize("int8", [False, True])
def test_as_many_groups_as_sequences_do_not_mean_one_each(P, int8, monkeypatch):     # noqa: F811
    """64 sequences and room for 64 groups, 58 sequences in one of them: those go at once, as with
    room for one group more."""
    hkv, group, d, bs, scale = 8, 4, 128, 16, 0.09
    sizes, prefixes = [1] * 6 + [58] + [0] * 57, [100] * 6 + [3000] + [16] * 57
    pages, tables, ctx, starts, ptables, values = _shared_case(sizes, prefixes, [i % 7 for i in range(64)], 0, hkv, d, bs, int8, 5)
    kp, vp, ks, vs = pages.cuda()
    wide = torch.zeros((64, 256), dtype=torch.int32)
    wide[:, :tables.shape[1]] = tables
    args = (kp, vp, wide.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints(prefixes), scale)
    q = torch.randn((64, hkv * group, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    outs = []
    for impl in (None, "both", "one"):
        if impl:
            monkeypatch.setenv("PKV_ROWS_IMPL", impl)
        else:
            monkeypatch.delenv("PKV_ROWS_IMPL", raising=False)
        lse = torch.empty((64, hkv * group), device="cuda")
        outs.append(P.paged_decode_attention_shared(q, *args, k_scales=ks, v_scales=vs, lse_out=lse))
        for s in range(64):
            check_rows(outs[-1][s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, int8)
    assert torch.equal(outs[0], outs[1])
    assert not torch.equal(outs[0], outs[2])       # (probabilities are rounded in other places)
