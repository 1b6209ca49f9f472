"""The windowed prefill's waits: those that run out over long windows, with rings of K and V that are
full of copies, and warps that fall behind one another."""
import time

import pytest
import torch

from test_gpu_window import P, _cuda, _paged      # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(64, 3), (128, 3), (64, 1), (128, 30)])
def test_waits_over_long_windows_run_out_at_once(P, d, n):     # noqa: F811
    """A limit below what a tile takes: the two warps that load K leave at different tiles, and none of
    them waits for copies that the other has not issued (4 s for each slot of the ring).  Whole
    units and halves; the call behind it gives the bits that it gives alone."""
    bs, hkv, group, chunk, window, sinks = 16, 4, 4, 300, 4000, 4
    lens = [3000 + 500 * (s % 3) for s in range(n)]
    pools, _, tables, _ = _paged(d + n, lens, window, sinks, 1, hkv, d, bs, False)
    q = torch.randn((n, chunk, hkv * group, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor([x - chunk for x in lens], dtype=torch.int32).cuda()
    call = lambda st, out: P.paged_prefill_attention_window(q, kp, vp, tab, pre, d ** -0.5, window, sinks, out=out, dev_status=st)
    good = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, got = call(good, torch.empty_like(q)).clone(), torch.empty_like(q)
    assert torch.isfinite(want.float()).all()
    torch.cuda.synchronize()
    lib, seen, longest = P.load_library(), 0, 0.0
    for ns in (1, 300, 1000, 2000, 3000, 1, 100, 3000, 5000, 4000, 1500):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t0 = time.monotonic()
        try:
            lib.pkv_set_pipeline_wait_ns(ns)
            call(st, got)
        finally:
            lib.pkv_set_pipeline_wait_ns(0)
        torch.cuda.synchronize()
        longest = max(longest, time.monotonic() - t0)
        seen |= int(st.item())
        got.zero_()
        call(good, got)
        assert int(good.item()) == 0 and torch.equal(got, want), ns
    assert seen == P.DEV_TIMEOUT and longest < 2.0


@pytest.mark.parametrize("d,n,chunk", [(64, 3, 300), (128, 3, 300), (64, 1, 300), (128, 1, 64), (64, 7, 90)])
def test_half_units_whose_warps_fall_behind(P, d, n, chunk):     # noqa: F811
    """Calls that find neither code nor data in the caches, so that the warps of a half unit are far
    apart: the bits of a warm call, and no wait that runs out."""
    bs, hkv, group, window, sinks = 16, 4, 4, 4000, 4
    lens = [3000 + 500 * (s % 3) for s in range(n)]
    pools, _, tables, _ = _paged(d + n, lens, window, sinks, 1, hkv, d, bs, False)
    q = torch.randn((n, chunk, hkv * group, d), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    kp, vp, tab = _cuda(*pools, tables)
    pre = torch.tensor([x - chunk for x in lens], dtype=torch.int32).cuda()
    st, got, flush = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty(96 << 20, device="cuda")
    want = None
    for i in range(60):
        got.zero_()
        if i % 4:                              # 384 MB through the L2, by kernels of other code
            flush.fill_(i).mul_(2).exp_().sum()
        P.paged_prefill_attention_window(q, kp, vp, tab, pre, d ** -0.5, window, sinks, out=got, dev_status=st)
        assert int(st.item()) == 0, i
        want = got.clone() if want is None else want
        assert torch.equal(got, want), i
