"""Decode steps behind one another without a pause, whose lengths change from step to step: the
launches of a step take its own plan, not the one of the step before."""
import pytest
import torch

from test_gpu_batch import P, _ints, _status      # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,longest", [(3, 6000), (70, 900)])
def test_captured_steps_of_other_lengths_give_the_eager_bits(P, n, longest, monkeypatch):     # noqa: F811
    monkeypatch.setenv("PKV_DECODE_IMPL", "split")
    hkv, group, d, bs, steps, scale = 4, 4, 128, 16, 20, 0.09
    gen = torch.Generator().manual_seed(n)
    width = -(-longest // bs)
    n_blocks = n * width
    kp, vp = (torch.randn((n_blocks + 1, bs, hkv, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    tables = torch.randperm(n_blocks, generator=gen).int().view(n, width).cuda()
    all_ctx = torch.randint(0, longest + 1, (steps, n), generator=gen)
    all_ctx[::3, ::2] = 20                      # steps whose work lies with every other sequence
    all_ctx = all_ctx.int().cuda()
    all_q = torch.randn((steps, n, hkv * group, d), generator=gen).to(torch.bfloat16).cuda()
    ctx, q, st = torch.zeros_like(all_ctx[0]), torch.zeros_like(all_q[0]), _status()
    lse = torch.zeros((n, hkv * group), device="cuda")
    plan = P.DecodePlan(kp, vp, tables, ctx, scale, hkv * group, lse_out=lse, dev_status=st)
    want = []
    for i in range(steps):
        ctx.copy_(all_ctx[i])
        q.copy_(all_q[i])
        torch.cuda.synchronize()
        plan.run(q)
        torch.cuda.synchronize()
        want.append((plan.out.clone(), lse.clone()))
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    outs = [torch.zeros((steps, *x.shape), dtype=x.dtype, device="cuda") for x in (plan.out, lse)]

    def step():
        torch.index_select(all_q, 0, at, out=q.unsqueeze(0))
        torch.index_select(all_ctx, 0, at, out=ctx.unsqueeze(0))
        plan.run(q)
        for all_of, x in zip(outs, (plan.out, lse)):
            all_of.index_copy_(0, at, x.unsqueeze(0))
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
    for i in range(steps):
        assert torch.equal(outs[0][i], want[i][0]) and torch.equal(outs[1][i], want[i][1]), i
