"""Steps of the calls for ragged batches behind one another, whose inputs the kernel just before
them writes."""
import pytest
import torch

from batch_reference import Paged, check_rows
from test_gpu_batch import P, _ints, _status, rows_impl      # noqa: F401 - fixtures

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("d,group", [(64, 4), (128, 8)])
def test_steps_that_read_what_the_kernel_before_them_writes(P, int8, d, group, rows_impl):     # noqa: F811
    """Captured steps without a pause between them: the query stays at one address and is written by a
    kernel of the step, as are the new token's row and (int8) its scales, which with 2 kv heads share
    a sector with those of the tokens before.  Groups of many, of one and of two; an encoder's pages
    for the cross attention behind it."""
    hkv, bs, scale, steps, sizes, prefixes = 2, 16, d ** -0.5, 24, [9, 1, 2], [70, 48, 33]
    hq, n, width, n_blocks = hkv * group, sum(sizes), 12, 80
    pages = Paged(3, n_blocks, hkv, d, bs, int8)
    shared = [pages.add(0, x, 5) for x in prefixes]
    pools = pages.cuda()
    kp, vp, ks, vs = pools
    group_of = [g for g, m in enumerate(sizes) for _ in range(m)]
    tables = torch.full((n, width), n_blocks, dtype=torch.int32)
    free = pages.perm[pages.at:]
    for s, g in enumerate(group_of):
        if prefixes[g] % bs:                   # goes on in a block of its own, at the prefix's end
            tables[s, prefixes[g] // bs] = free.pop()
    tables, free = tables.cuda(), _ints(free)
    starts, plens, ptables = _ints([0, 9, 10, 12]), _ints(prefixes), torch.stack([r for r, _ in shared]).cuda()
    gen = torch.Generator().manual_seed(d)
    all_q = torch.randn((steps, n, hq, d), generator=gen).to(torch.bfloat16).cuda()
    # tokens of sizes that grow, so that no scale is the one before it
    all_kv = (torch.randn((steps, 2, n, hkv, d), generator=gen) * (1 + torch.arange(steps).view(-1, 1, 1, 1, 1))).to(torch.bfloat16).cuda()
    q, kv = torch.zeros_like(all_q[0]), torch.zeros_like(all_kv[0])
    lens, cursor, at = _ints([prefixes[g] for g in group_of]), _ints([0]), torch.zeros(1, dtype=torch.int64, device="cuda")
    m, st, one = P.StepMaps.empty(n, n, "cuda"), _status(), _ints([1] * n)
    lse, cross, cross_lse = (torch.zeros(x, dtype=t, device="cuda") for x, t in (((n, hq), torch.float32), ((n, hq, d), torch.bfloat16),
                                                                                 ((n, hq), torch.float32)))
    plan = P.SharedDecodePlan(kp, vp, tables, m.ctx_lens, starts, ptables, plens, scale, hq, k_scales=ks, v_scales=vs, lse_out=lse,
                              dev_status=st)
    ws = torch.empty(P.rows_workspace_bytes(n, hq, d), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros((steps, *x.shape), dtype=x.dtype, device="cuda") for x in (plan.out, lse, cross, cross_lse)]

    def step():
        P.paged_step_maps(lens, one, free, tables, bs, n_blocks, n, cursor=cursor, out=m, dev_status=st)
        torch.index_select(all_kv, 0, at, out=kv.unsqueeze(0))
        torch.index_select(all_q, 0, at, out=q.unsqueeze(0))
        P.paged_kv_write_slots(kv[0], kv[1], kp, vp, m.slots, ks, vs, dev_status=st)
        plan.run(q)
        P.paged_cross_attention(q, starts, kp, vp, ptables, plens, scale, k_scales=ks, v_scales=vs, out=cross, lse_out=cross_lse,
                                workspace=ws, dev_status=st)
        for all_of, x in zip(outs, (plan.out, lse, cross, cross_lse)):
            all_of.index_copy_(0, at, x.unsqueeze(0))
        lens.copy_(m.ctx_lens)
        cursor.copy_(m.cursor)
        at.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # what the pages hold in the end, which is what every step saw the beginning of
    cpu_tables, flat = tables.cpu(), [x.cpu() for x in pools[:2]]
    for s, g in enumerate(group_of):
        t = torch.arange(prefixes[g], prefixes[g] + steps)
        rows = cpu_tables[s][t // bs].long() * bs + t % bs
        own = [x.view(-1, hkv, d)[rows].double() for x in flat]
        if int8:
            own = [x * sc.cpu().view(-1, hkv)[rows].double()[..., None] for x, sc in zip(own, (ks, vs))]
        else:
            assert torch.equal(own[0], all_kv[:, 0, s].cpu().double())
        both = [torch.cat(x) for x in zip(shared[g][1], own)]
        for i in range(steps):
            check_rows(outs[0][i, s:s + 1], outs[1][i, s:s + 1], all_q[i, s:s + 1], *(x[:prefixes[g] + i + 1] for x in both), scale, int8)
            check_rows(outs[2][i, s:s + 1], outs[3][i, s:s + 1], all_q[i, s:s + 1], *shared[g][1], scale, int8)


def test_maps_of_a_step_behind_one_that_ran_out(P):     # noqa: F811
    """A sequence that found no block gets no slots in the step after that either, until it is given
    one; an inactive sequence, whose row is all scratch, writes to the scratch block."""
    bs, scratch = 16, 50
    tables = torch.full((5, 4), scratch, dtype=torch.int32)
    tables[:4, 0] = torch.tensor([7, 8, 9, 10])
    tables = tables.cuda()
    lens, free, cursor = _ints([16, 16, 16, 3, 5]), _ints([3]), _ints([0])

    def step(lens, cursor, new):
        st = _status()
        m = P.paged_step_maps(lens, _ints(new), free, tables, bs, scratch, sum(new), cursor=cursor, dev_status=st)
        return m, m.slots.tolist(), int(st.item())

    m, slots, status = step(lens, cursor, [3, 3, 20, 1, 1])     # the second and third sequence find no block
    assert slots == [48, 49, 50] + [-1] * 23 + [163, 805] and status == P.DEV_OUT_OF_BLOCKS
    assert tables.tolist() == [[7, 3, 50, 50], [8, 50, 50, 50], [9, 50, 50, 50], [10, 50, 50, 50], [50] * 4]
    m, slots, status = step(m.ctx_lens, m.cursor, [1] * 5)
    assert slots == [51, -1, -1, 164, 806] and status == P.DEV_OUT_OF_BLOCKS
    assert m.positions.tolist() == [19, 19, 36, 4, 6] and m.ctx_lens.tolist() == [20, 20, 37, 5, 7]
    tables[1, 1], tables[2, 1], tables[2, 2] = 20, 21, 22
    m, slots, status = step(m.ctx_lens, m.cursor, [1] * 5)
    assert slots == [52, 20 * 16 + 4, 22 * 16 + 5, 165, 807] and status == 0
    # the scratch block takes the rows of idle sequences, whatever they are
    k, v = (torch.randn((5, 2, 64), device="cuda").to(torch.bfloat16) for _ in range(2))
    pools = [torch.zeros((scratch + 1, bs, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    P.paged_kv_write_slots(k, v, *pools, m.slots)
    assert torch.equal(pools[0].view(-1, 2, 64)[m.slots], k)
