"""The calls for ragged batches where something is off or in the way: waits that run out,
random shapes, plans whose contents change between captured runs, workspaces that hold
another call's leftovers, calls that go through Python."""
import random

import pytest
import torch

from batch_reference import Paged, check_rows
from test_gpu_batch import P, _ints, _shared_case, _status, rows_impl      # noqa: F401 - fixtures

pytestmark = pytest.mark.gpu

TRIES = 5          # calls with the short limit; at least one of them must run out


def _fill(t, byte):
    return t.view(torch.uint8).fill_(byte)


@pytest.mark.parametrize("byte", [0, 0x7F, 0xFF])
@pytest.mark.parametrize("int8", [False, True])
def test_waits_run_out_then_recover(P, monkeypatch, int8, byte):     # noqa: F811
    """A limit of 1 ns: the kernels report PKV_DEV_TIMEOUT and end, whatever the workspace holds (the
    joins read it); the next calls are right.  Two key tiles at most per CTA, as every copy then
    fits the rings and a wind-down's waits complete."""
    monkeypatch.setenv("PKV_ROWS_IMPL", "all")
    hkv, group, d, bs, scale = 2, 4, 128, 16, 0.09
    pages, tables, ctx, starts, ptables, values = _shared_case([30], [250], [20] * 30, 0, hkv, d, bs, int8, 3)
    kp, vp, ks, vs = pages.cuda()
    hq = hkv * group
    q = torch.randn((30, hq, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    ws = torch.empty(P.rows_workspace_bytes(30, hq, d), dtype=torch.uint8, device="cuda")
    lse = torch.empty((30, hq), device="cuda")
    args = (tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints([250]))

    def shared(st):
        return P.paged_decode_attention_shared(q, kp, vp, *args, scale, k_scales=ks, v_scales=vs, lse_out=lse, workspace=ws, dev_status=st)

    def cross(st):
        return P.paged_cross_attention(q, args[2], kp, vp, args[3], args[4], scale, k_scales=ks, v_scales=vs, lse_out=lse, workspace=ws,
                                       dev_status=st)

    lib = P.load_library()
    for call, keys in ((shared, 270), (cross, 250)):
        seen = 0
        lib.pkv_set_pipeline_wait_ns(1)
        try:
            for _ in range(TRIES):
                _fill(ws, byte)
                st = _status()
                call(st)
                torch.cuda.synchronize()
                seen |= int(st.item())
        finally:
            lib.pkv_set_pipeline_wait_ns(0)
        assert seen & P.DEV_TIMEOUT
        _fill(ws, byte)
        st = _status()
        out = call(st)
        assert int(st.item()) == 0
        for s in range(30):
            check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *(x[:keys] for x in values[s]), scale, int8)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(P, rows_impl, seed):     # noqa: F811
    r = random.Random(seed)
    d, hkv, group, bs = r.choice([64, 128]), r.choice([1, 2, 3, 5]), r.choice([1, 2, 3, 4, 5, 6, 7, 8]), r.choice([16, 32, 48, 256])
    int8, scale, hq = r.random() < 0.4, d ** -0.5, hkv * group
    n = r.randint(1, 12)
    n_q, keys = [r.choice([0, 1, 1, 2, r.randint(1, 90)]) for _ in range(n)], [r.choice([0, 1, 15, 16, 128, r.randint(1, 700)]) for _ in range(n)]
    pages = Paged(seed, sum(-(-x // bs) for x in keys) + 1, hkv, d, bs, int8)
    added = [pages.add(0, x, max(max(-(-y // bs) for y in keys), 1)) for x in keys]
    kp, vp, ks, vs = pages.cuda()
    starts = [0]
    for x in n_q:
        starts.append(starts[-1] + x)
    rows = max(starts[-1], 1)
    q = torch.randn((rows, hq, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    lse, st = torch.empty((rows, hq), device="cuda"), _status()
    out = P.paged_cross_attention(q, _ints(starts), kp, vp, torch.stack([t for t, _ in added]).cuda(), _ints(keys), scale, k_scales=ks,
                                  v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s in range(n):
        a, b = starts[s], starts[s + 1]
        if a < b:
            check_rows(out[a:b], lse[a:b], q[a:b], *added[s][1], scale, int8)
    sizes = [r.randint(0, 40) for _ in range(r.randint(1, 6))]
    prefixes = [r.choice([0, 1, 16, 127, r.randint(1, 900)]) for _ in sizes]
    loose = r.randint(0, 3)
    if loose + sum(sizes) == 0:
        loose = 1
    behind = [r.choice([0, 1, 16, r.randint(0, 130)]) for _ in range(sum(sizes))]
    pages, tables, ctx, starts, ptables, values = _shared_case(sizes, prefixes, behind, loose, hkv, d, bs, int8, seed)
    kp, vp, ks, vs = pages.cuda()
    m = len(ctx)
    q = torch.randn((m, hq, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    lse, st = torch.empty((m, hq), device="cuda"), _status()
    out = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints(prefixes), scale,
                                          k_scales=ks, v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s in range(m):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, int8)


def test_graphs_that_share_a_workspace(P, rows_impl):     # noqa: F811
    """Two captured plans on one workspace, replayed in turn; the groups, lengths and tables that they
    read change in place between replays."""
    hkv, group, d, bs, scale, hq = 2, 4, 128, 16, 0.09, 8
    cases = [_shared_case([20, 7], [300, 140], [(i * 7) % 40 for i in range(27)], 0, hkv, d, bs, False, 1),
             _shared_case([5, 22], [140, 290], [(i * 5) % 33 for i in range(27)], 0, hkv, d, bs, False, 2)]
    width, pwidth = max(c[1].shape[1] for c in cases), max(c[4].shape[1] for c in cases)
    n_blocks = max(c[0].n_blocks for c in cases)
    ws = torch.empty(P.rows_workspace_bytes(27, hq, d), dtype=torch.uint8, device="cuda")
    state = []
    for _ in range(2):
        kp, vp = (torch.zeros((n_blocks + 1, bs, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        tab, ptab = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((27, width), (2, pwidth)))
        ctx, starts, plens = _ints([0] * 27), _ints([0, 0, 0]), _ints([0, 0])
        q, lse = torch.zeros((27, hq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((27, hq), device="cuda")
        plan = P.SharedDecodePlan(kp, vp, tab, ctx, starts, ptab, plens, scale, hq, lse_out=lse, workspace=ws)
        plan.run(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run(q)
        state.append((kp, vp, tab, ptab, ctx, starts, plens, q, lse, plan, graph))
    gen = torch.Generator().manual_seed(0)
    for turn in range(4):
        qs = []
        for i, (kp, vp, tab, ptab, ctx, starts, plens, q, lse, plan, graph) in enumerate(state):
            pages, tables, lens, first, ptables, values = cases[(turn + i) % 2]
            kp[:pages.n_blocks + 1].copy_(pages.pools[0])
            vp[:pages.n_blocks + 1].copy_(pages.pools[1])
            tab[:, :tables.shape[1]].copy_(tables)
            ptab[:, :ptables.shape[1]].copy_(ptables)
            ctx.copy_(torch.tensor(lens))
            starts.copy_(torch.tensor(first))
            plens.copy_(torch.tensor([300, 140] if (turn + i) % 2 == 0 else [140, 290]))
            q.copy_(torch.randn(q.shape, generator=gen).to(torch.bfloat16))
            qs.append(values)
        for s in state:
            s[10].replay()
        torch.cuda.synchronize()
        for values, (_, _, _, _, _, _, _, q, lse, plan, _) in zip(qs, state):
            for s in range(27):
                check_rows(plan.out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, False)


def test_native_and_python_marshalling_agree(P, monkeypatch):     # noqa: F811
    assert P._native is not None
    pages = Paged(5, 40, 2, 64, 16, True)
    added = [pages.add(0, x, 8) for x in (100, 40, 7)]
    kp, vp, ks, vs = pages.cuda()
    tables, lens, starts = torch.stack([t for t, _ in added]).cuda(), _ints([100, 40, 7]), _ints([0, 4, 5, 9])
    gen = torch.Generator().manual_seed(1)
    q = torch.randn((9, 8, 64), generator=gen).to(torch.bfloat16).cuda()
    k = torch.randn((9, 2, 64), generator=gen).to(torch.bfloat16).cuda()
    results = []
    for native in (P._native, None):
        monkeypatch.setattr(P, "_native", native)
        tab = torch.full((3, 8), 50, dtype=torch.int32, device="cuda")
        maps = P.StepMaps.empty(3, 12, "cuda")
        P.paged_step_maps(_ints([0, 3, 20]), _ints([4, 1, 4]), _ints(list(range(40))), tab, 16, 50, 12, out=maps)
        pools = [torch.zeros((51, 16, 2, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((51, 16, 2), device="cuda") for _ in range(2)]
        P.paged_kv_write_slots(k, k, *pools, maps.slots[:9], *scales)
        lse = torch.zeros((9, 8), device="cuda")
        out = P.paged_cross_attention(q, starts, kp, vp, tables, lens, 0.1, k_scales=ks, v_scales=vs, lse_out=lse)
        shared = P.paged_decode_attention_shared(q[:3], kp, vp, tables, lens, _ints([0, 3]), tables[:1], _ints([7]), 0.1, k_scales=ks,
                                                 v_scales=vs)
        results.append([tab, *maps, *pools, *scales, lse, out, shared])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_binding_refusals(P):     # noqa: F811
    """What does not fit is refused before anything is launched."""
    i2, pool = _ints([1, 1]), torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    tab, q = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    maps = P.StepMaps.empty(2, 4, "cuda")
    ok = dict(lens=i2, n_new=i2, free_blocks=i2, block_tables=tab, block_size=16, n_blocks=8, n_tokens=4, out=maps)
    for kw in (dict(lens=_ints([1])), dict(n_new=i2.long()), dict(free_blocks=tab), dict(n_tokens=5), dict(n_tokens=-1), dict(cursor=i2),
               dict(out=maps._replace(slots=maps.positions)), dict(lens=i2.cpu()), dict(dev_status=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            P.paged_step_maps(**dict(ok, **kw))
    for kw in (dict(out=maps._replace(ctx_lens=i2)), dict(cursor=maps.cursor), dict(block_size=24), dict(n_blocks=-1)):
        with pytest.raises(P.PagedKVError):
            P.paged_step_maps(**dict(ok, **kw))
    with pytest.raises(TypeError):
        P.paged_step_maps(**dict(ok, out=tuple(maps)))
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    for a in ((k, k, pool, pool, slots[:1]), (k, k, pool, pool, i2), (k, k[:1], pool, pool, slots), (k.float(), k, pool, pool, slots),
              (k[..., :32], k, pool, pool, slots), (k.transpose(0, 1), k, pool, pool, slots), (k, k, pool, pool[:5], slots)):
        with pytest.raises(ValueError):
            P.paged_kv_write_slots(*a)
    starts = _ints([0, 1, 2])
    good = dict(q=q, q_starts=starts, k_pool=pool, v_pool=pool, block_tables=tab, key_lens=i2, softmax_scale=0.1)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for kw in (dict(q_starts=i2), dict(key_lens=starts), dict(q=q[..., :32]), dict(out=q[:1].clone()), dict(lse_out=torch.zeros(2, device="cuda")),
               dict(workspace=q), dict(block_tables=tab.long())):
        with pytest.raises(ValueError):
            P.paged_cross_attention(**dict(good, **kw))
    for kw in (dict(out=q), dict(workspace=ws[:256]), dict(workspace=ws[16:]), dict(softmax_scale=0.0)):
        with pytest.raises(P.PagedKVError):
            P.paged_cross_attention(**dict(good, **kw))
    args = dict(q=q, k_pool=pool, v_pool=pool, block_tables=tab, ctx_lens=i2, group_starts=i2, prefix_tables=tab[:1], prefix_lens=_ints([3]),
                softmax_scale=0.1)
    for kw in (dict(group_starts=starts), dict(prefix_lens=i2), dict(ctx_lens=starts), dict(q=q[:1])):
        with pytest.raises(ValueError):
            P.paged_decode_attention_shared(**dict(args, **kw))
    with pytest.raises(P.PagedKVError):
        P.paged_decode_attention_shared(**dict(args, q=torch.zeros((2, 18, 64), dtype=torch.bfloat16, device="cuda")))
