"""Waits of the kernels that run out over long runs: rings of K and V that are full of copies."""
import time

import pytest
import torch

from batch_reference import Paged, check_rows
from test_gpu_batch import P, _ints, _status      # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_waits_over_long_runs_run_out_at_once(P, monkeypatch, d, int8):     # noqa: F811
    """A limit below what a tile takes: the two warps that load K leave at different tiles, and none of
    them waits for copies that the other has not issued (4 s for each slot of the ring)."""
    monkeypatch.setenv("PKV_ROWS_IMPL", "all")
    hkv, group, bs, scale, n_q, keys = 4, 4, 16, d ** -0.5, [150, 70, 300], [6000, 9000, 5000]
    pages = Paged(d, sum(-(-x // bs) for x in keys) + 1, hkv, d, bs, int8)
    added = [pages.add(0, x, max(-(-y // bs) for y in keys)) for x in keys]
    kp, vp, ks, vs = pages.cuda()
    starts, total = [0, 150, 220, 520], 520
    q = torch.randn((total, hkv * group, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    args = (q, _ints(starts), kp, vp, torch.stack([t for t, _ in added]).cuda(), _ints(keys), scale)
    lse, ws = torch.empty((total, hkv * group), device="cuda"), torch.empty(P.rows_workspace_bytes(total, hkv * group, d),
                                                                          dtype=torch.uint8, device="cuda")
    more = dict(k_scales=ks, v_scales=vs, lse_out=lse, workspace=ws)
    P.paged_cross_attention(*args, **more)
    torch.cuda.synchronize()
    lib, seen, longest = P.load_library(), 0, 0.0
    try:
        for ns in (1, 300, 1000, 2000, 3000, 1, 100, 3000, 5000, 4000, 1500):
            st = _status()
            torch.cuda.synchronize()
            t0 = time.monotonic()
            lib.pkv_set_pipeline_wait_ns(ns)
            P.paged_cross_attention(*args, **more, dev_status=st)
            torch.cuda.synchronize()
            longest = max(longest, time.monotonic() - t0)
            seen |= int(st.item())
    finally:
        lib.pkv_set_pipeline_wait_ns(0)
    assert seen == P.DEV_TIMEOUT and longest < 2.0
    st = _status()
    out = P.paged_cross_attention(*args, **more, dev_status=st)
    assert int(st.item()) == 0
    for s in range(3):
        a, b = starts[s], starts[s + 1]
        check_rows(out[a:b], lse[a:b], q[a:b], *added[s][1], scale, int8)
