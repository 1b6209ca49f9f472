"""The calls for ragged batches on the GPU: step maps, slot writes, cross attention,
decode with shared prefixes, and a run of them together."""
import random
import threading

import pytest
import torch

from batch_reference import GARBAGE_ID, Paged, check_rows, maps

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


@pytest.fixture(params=["all", "one", "both", "auto"])
def rows_impl(request, monkeypatch):
    """Rows contracted all at once, one by one or each run its own way (PKV_ROWS_IMPL), and as the sizes say."""
    if request.param == "auto":
        monkeypatch.delenv("PKV_ROWS_IMPL", raising=False)
    else:
        monkeypatch.setenv("PKV_ROWS_IMPL", request.param)
    return request.param


def _ints(x, kind=torch.int32):
    return torch.tensor(x, dtype=kind, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- step maps ---------------------------------------------------------------------

def _maps_case(seed, n, bs, width, most_new, idle=0.2, fresh=0.3):
    r = random.Random(seed)
    new = [0 if r.random() < idle else r.randint(1, most_new) for _ in range(n)]
    lens = [0 if r.random() < fresh else r.randint(0, width * bs - m) for m in new]
    need = sum(-(-(h + m) // bs) - -(-h // bs) for h, m in zip(lens, new))
    held = [-(-h // bs) for h in lens]
    n_blocks = sum(held) + need + 5
    ids = list(range(n_blocks))
    r.shuffle(ids)
    tables = []
    for h in held:
        tables.append([ids.pop() for _ in range(h)] + [GARBAGE_ID] * (width - h))
    return lens, new, ids, tables, n_blocks


def _run_maps(P, lens, new, free, cursor, tables, bs, n_blocks, n_tokens, width):
    tab = torch.tensor(tables, dtype=torch.int32).view(len(lens), width).cuda()
    st = _status()
    m = P.paged_step_maps(_ints(lens), _ints(new), _ints(free), tab, bs, n_blocks, n_tokens,
                          cursor=None if cursor is None else _ints([cursor]), dev_status=st)
    want = maps(lens, new, free, cursor or 0, tables, bs, n_blocks, n_tokens)
    for name, got, ref in zip(m._fields, m, [want[0], want[1], want[2], want[3], want[4], [want[5]]]):
        assert got.tolist() == ref, name
    assert tab.tolist() == tables
    assert int(st.item()) == want[6]


@pytest.mark.parametrize("n,bs,width,most_new,pad", [
    (1, 16, 1, 1, 0), (3, 16, 4, 20, 7), (64, 16, 300, 1, 0), (64, 32, 9, 40, 1), (17, 256, 5, 700, 513), (513, 48, 40, 9, 100),
    (2048, 16, 6, 33, 0), (2049, 16, 3, 5, 31), (5000, 64, 17, 3, 2), (2, 16, 3000, 20000, 0)])
def test_maps(P, n, bs, width, most_new, pad):
    for seed in range(3):
        lens, new, free, tables, n_blocks = _maps_case(seed, n, bs, width, min(most_new, width * bs))
        cursor = seed * 2
        free = [GARBAGE_ID] * cursor + free
        _run_maps(P, lens, new, free, cursor if seed else None, tables, bs, n_blocks, sum(new) + pad, width)


def test_maps_of_nothing(P):
    _run_maps(P, [], [], [], 0, [], 16, 4, 0, 3)
    _run_maps(P, [], [], [1, 2], 1, [], 16, 4, 5, 3)
    _run_maps(P, [0, 17, 16], [0, 0, 0], [], 0, [[3, 2], [1, GARBAGE_ID], [0, GARBAGE_ID]], 16, 4, 0, 2)


def test_maps_with_bad_input(P):
    scratch = 50
    tables = [[GARBAGE_ID] * 4 for _ in range(9)]
    tables[1][:2], tables[6][:1], tables[8][:1] = [7, 51], [-1], [scratch]
    lens = [0, 20, -1, 0, 60, 0, 5, 0, 3]
    new = [3, 30, 4, -2, 5, 40, 4, 64, 2]      # bad: negative, negative, beyond the row; a bad held block (twice); scratch
    for free, cursor in (([9, 60, 11, 12], 0), ([9, -3, 11, 12, 13, 14, 15, 16, 17, 18, 19], 0), (list(range(40)), -1),
                         (list(range(40)), 38), ([], 0), (list(range(40)), 2 ** 31 - 3)):
        for n_tokens in (200, 50, 0):
            _run_maps(P, lens, new, free, cursor, [list(r) for r in tables], 16, scratch, n_tokens, 4)


def test_maps_of_the_widest_rows(P):
    """Rows of 2^31 - 16 tokens, full up to the last one; the step adds nothing, so none of it is touched."""
    width = 2 ** 27 - 1
    tab = torch.empty(1, dtype=torch.int32, device="cuda")
    lib, dev = P.load_library(), "cuda"
    m = P.StepMaps.empty(3, 4, dev)
    st = _status()
    lens = _ints([width * 16 - 1] * 3)
    new = _ints([0, 0, 0])
    rc = lib.paged_step_maps(lens.data_ptr(), new.data_ptr(), 3, None, 0, None, 8, 16, tab.data_ptr(), width, 4,
                             *(t.data_ptr() for t in m[:5]), m.cursor.data_ptr(), st.data_ptr(), None)
    torch.cuda.synchronize()
    assert rc == 0 and int(st.item()) == 0 and m.ctx_lens.tolist() == [width * 16 - 1] * 3
    assert m.token_seqs.tolist() == [-1] * 4 and m.cursor.tolist() == [0]


def test_maps_follow_the_block_manager(P):
    """Steps of the host manager and of the device, from the same free list."""
    bs, slots, width, n_blocks = 16, 5, 12, 60
    bm = P.BlockManager(n_blocks, bs, slots, width)
    prompts = [5, 16, 33, 1, 47]
    tab = torch.full((slots, width), n_blocks, dtype=torch.int32, device="cuda")
    free = _ints(list(range(n_blocks)))       # the manager hands out the lowest ids first
    zero = _ints([0])
    m = P.paged_step_maps(_ints([0] * slots), _ints(prompts), free, tab, bs, n_blocks, sum(prompts), cursor=zero)
    for s, x in enumerate(prompts):
        bm.admit(s, x)
    for _ in range(40):
        tables, lens, _ = bm.export()
        assert tab.cpu().tolist() == tables.tolist() and m.ctx_lens.tolist() == lens.tolist()
        assert bm.begin_step() == []
        m = P.paged_step_maps(m.ctx_lens, _ints([1] * slots), free, tab, bs, n_blocks, slots, cursor=m.cursor)
        bm.end_step()


# ---- slot writes ---------------------------------------------------------------------

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n,hkv,d,bs,strided", [(1, 1, 64, 16, False), (3, 1, 128, 16, True), (65, 3, 64, 32, True),
                                                (129, 8, 128, 16, True), (1000, 5, 64, 48, False)])
def test_write_slots(P, n, hkv, d, bs, strided, int8):
    """The same bits as paged_kv_write(_int8) writes; rows of no slot leave the pool alone."""
    gen = torch.Generator().manual_seed(n + hkv)
    n_blocks = -(-n // bs) * 2 + 3
    rows = torch.randperm(n_blocks * bs, generator=gen)[:n]
    if strided:
        qkv = torch.randn((n, 4 + 2 * hkv, d), generator=gen).to(torch.bfloat16).cuda()
        k, v = qkv[:, 4:4 + hkv], qkv[:, 4 + hkv:]
    else:
        k, v = (torch.randn((n, hkv, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    k[0, 0] = 0                                # a row of zeros
    if n > 2:
        v[1] = 1e-38                           # a scale below the normal range
        k[2, 0, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])    # ties
    skip = torch.rand(n, generator=gen) < 0.3
    slots = torch.where(skip, torch.where(torch.rand(n, generator=gen) < 0.5, -1, -2 ** 40), rows)
    shape = (n_blocks + 1, bs, hkv, d)
    kind = torch.int8 if int8 else torch.bfloat16
    fill = torch.randint(-100, 100, shape, generator=gen).to(kind)
    pools = [[fill.clone().cuda() for _ in range(2)] for _ in range(2)]
    scales = [[torch.full(shape[:3], 3.0, device="cuda") if int8 else None for _ in range(2)] for _ in range(2)]
    st = _status()
    P.paged_kv_write_slots(k, v, *pools[0], slots.cuda(), *scales[0], dev_status=st)
    # the reference: every row a sequence of one block, at its place in it
    there = ~skip
    tables, pos = (slots[there] // bs).int().cuda().view(-1, 1), (slots[there] % bs).int().cuda()
    if there.any():
        args = (k[there.cuda()].contiguous().unsqueeze(1), v[there.cuda()].contiguous().unsqueeze(1))
        if int8:
            P.paged_kv_write_int8(*args, *pools[1], *scales[1], tables, pos)
        else:
            P.paged_kv_write(*args, *pools[1], tables, pos)
    for a, b in zip(pools[0] + (scales[0] if int8 else []), pools[1] + (scales[1] if int8 else [])):
        assert torch.equal(a.view(torch.int8 if a.dtype is torch.int8 else torch.int16 if a.dtype is torch.bfloat16 else torch.int32),
                           b.view(torch.int8 if b.dtype is torch.int8 else torch.int16 if b.dtype is torch.bfloat16 else torch.int32))
    assert int(st.item()) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_write_slots_int8_codes(P, d):
    """Codes and scales bit for bit as paged_kv_write_int8 stores them, over rows of any size: halves
    and other simple fractions of the largest element (ties), subnormal scales, infinities, NaN."""
    gen = torch.Generator().manual_seed(d)
    hkv, bs, n = 4, 16, 4096
    x = torch.randn((2, n, hkv, d), generator=gen)
    top = x.abs().amax(-1, keepdim=True)
    share = torch.randint(-254, 255, x.shape, generator=gen) / 254.0           # multiples of half a step
    x = torch.where(torch.rand(x.shape, generator=gen) < 0.3, top * share, x)
    x = x * 2.0 ** torch.randint(-140, 120, (2, n, hkv, 1), generator=gen)
    odd = torch.rand((2, n, hkv, 1), generator=gen)
    at = torch.randint(0, d, (2, n, hkv, 1), generator=gen)
    for low, value in ((0.02, float("nan")), (0.04, float("inf")), (0.06, -float("inf")), (0.08, 0.0)):
        x = torch.where((odd < low) & (odd >= low - 0.02), x.scatter(-1, at, value) if value else torch.zeros_like(x), x)
    k, v = x.to(torch.bfloat16).cuda()
    pools = [[torch.zeros((n // bs + 1, bs, hkv, d), dtype=torch.int8, device="cuda") for _ in range(2)] for _ in range(2)]
    scales = [[torch.zeros((n // bs + 1, bs, hkv), device="cuda") for _ in range(2)] for _ in range(2)]
    P.paged_kv_write_slots(k, v, *pools[0], torch.arange(n, device="cuda"), *scales[0])
    P.paged_kv_write_int8(k.unsqueeze(0), v.unsqueeze(0), *pools[1], *scales[1], torch.arange(n // bs, dtype=torch.int32, device="cuda").view(1, -1),
                          _ints([0]))
    for a, b in zip(pools[0], pools[1]):
        assert torch.equal(a, b)
    for a, b in zip(scales[0], scales[1]):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("int8", [False, True])
def test_write_slots_outside_the_pool(P, int8):
    n_blocks, bs, hkv, d = 3, 16, 2, 64
    k, v = (torch.randn((5, hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    pools = [torch.zeros((n_blocks + 1, bs, hkv, d), dtype=torch.int8 if int8 else torch.bfloat16, device="cuda") for _ in range(2)]
    scales = [torch.zeros((n_blocks + 1, bs, hkv), device="cuda") if int8 else None for _ in range(2)]
    st = _status()
    P.paged_kv_write_slots(k, v, *pools, _ints([64, 2 ** 40, 63, -1, 2 ** 31], torch.int64), *scales, dev_status=st)
    assert int(st.item()) == P.DEV_BAD_POSITION
    written = pools[0].view(-1, hkv * d).float().abs().sum(1).nonzero().flatten().tolist()
    assert written == [63]                     # the last row of the scratch block
    st.zero_()
    P.paged_kv_write_slots(k, v, *pools, _ints([-1] * 5, torch.int64), *scales, dev_status=st)
    P.paged_kv_write_slots(k[:0], v[:0], *pools, _ints([], torch.int64), *scales, dev_status=st)
    assert int(st.item()) == 0


# ---- cross attention ---------------------------------------------------------------------

# queries per sequence, keys per sequence, hkv, group, d, bs
CROSS = [
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1, 1], [17, 0, 255, 16], 2, 4, 64, 16),
    ([1] * 9, [1, 2, 15, 127, 128, 129, 130, 256, 257], 2, 8, 128, 16),
    ([3, 0, 5, 1], [40, 77, 0, 128], 3, 3, 128, 48),
    ([33, 31, 64, 2], [129, 300, 1, 255], 1, 8, 64, 16),
    ([200, 1, 65], [333, 500, 64], 2, 5, 128, 32),
    ([130], [1000], 2, 1, 128, 256),
    ([7, 300], [260, 2000], 1, 16, 64, 16),
    ([19, 40], [700, 90], 2, 7, 128, 64),
    ([64], [5000], 1, 4, 128, 16),
    ([1] * 40, [100 + 37 * i for i in range(40)], 4, 4, 128, 16),
    ([0, 0], [5, 6], 1, 4, 64, 16),
    ([11, 13, 17], [600, 601, 602], 1, 6, 64, 16),
    ([257, 255], [256, 384], 8, 2, 64, 32),
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_q,keys,hkv,group,d,bs", CROSS)
def test_cross(P, n_q, keys, hkv, group, d, bs, int8, rows_impl):
    n, hq, scale = len(n_q), hkv * group, d ** -0.5
    pages = Paged(sum(n_q) + d, sum(-(-x // bs) for x in keys) + 1, hkv, d, bs, int8)
    width = max(-(-x // bs) for x in keys) + 2
    added = [pages.add(0, x, width) for x in keys]
    kp, vp, ks, vs = pages.cuda()
    tables = torch.stack([row for row, _ in added]).cuda()
    # two rows before the first sequence and three behind the last; queries a stride apart
    starts, total = [2], sum(n_q) + 5
    for x in n_q:
        starts.append(starts[-1] + x)
    gen = torch.Generator().manual_seed(5)
    q = torch.randn((total, hq + 3, d), generator=gen).to(torch.bfloat16).cuda()[:, 1:1 + hq]
    out = torch.full((total, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, hq), 7.0, device="cuda")
    st = _status()
    got = P.paged_cross_attention(q, _ints(starts), kp, vp, tables, _ints(keys), scale, k_scales=ks, v_scales=vs, out=out,
                                  lse_out=lse, dev_status=st)
    assert got is out and int(st.item()) == 0
    for rows in (slice(0, 2), slice(total - 3, total)):
        assert (out[rows] == 7).all() and (lse[rows] == 7).all()
    for s in range(n):
        a, b = starts[s], starts[s + 1]
        if a < b:
            check_rows(out[a:b], lse[a:b], q[a:b], *added[s][1], scale, int8)
    again = P.paged_cross_attention(q.contiguous(), _ints(starts), kp, vp, tables, _ints(keys), scale, k_scales=ks, v_scales=vs)
    assert torch.equal(again[2:total - 3], out[2:total - 3])


@pytest.mark.parametrize("n", [33, 64, 65, 1030])
def test_cross_of_many_sequences(P, n, rows_impl):
    """Sequences whose rows are looked up in several steps, some of them without rows or keys."""
    r = random.Random(n)
    n_q = [r.choice([0, 0, 1, 1, 2, 3]) for _ in range(n)]
    n_q[:3], n_q[-2:] = [0, 0, 1], [2, 0]
    keys = [r.choice([0, 1, 16, 17, 40, 130]) for _ in range(n)]
    hkv, group, d, bs, scale = 1, 2, 64, 16, 0.125
    pages = Paged(n, sum(-(-x // bs) for x in keys) + 1, hkv, d, bs, False)
    added = [pages.add(0, x, 9) for x in keys]
    kp, vp, _, _ = pages.cuda()
    tables = torch.stack([row for row, _ in added]).cuda()
    starts = [5]
    for x in n_q:
        starts.append(starts[-1] + x)
    total = starts[-1] + 40
    q = torch.randn((total, hkv * group, d), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    st = _status()
    P.paged_cross_attention(q, _ints(starts), kp, vp, tables, _ints(keys), scale, out=out, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for rows in (slice(0, 5), slice(total - 40, total)):
        assert (out[rows] == 7).all() and (lse[rows] == 7).all()
    for s in range(n):
        a, b = starts[s], starts[s + 1]
        if a < b:
            check_rows(out[a:b], lse[a:b], q[a:b], *added[s][1], scale, False)


@pytest.mark.parametrize("ramp", [(-6, 2), (2, -6), (-37, -30), (25, 30)])
@pytest.mark.parametrize("d", [64, 128])
def test_cross_over_scales_of_any_size(P, d, ramp, rows_impl):
    """int8 pages whose V scales grow or shrink over a sequence by many orders of magnitude, or are
    all tiny or huge."""
    hkv, group, bs, scale, n = 2, 3, 16, d ** -0.5, 900
    pages = Paged(9, 60, hkv, d, bs, True)
    row, (k, v) = pages.add(0, n, 60)
    slots = row[torch.arange(n) // bs].long() * bs + torch.arange(n) % bs
    factor = 10.0 ** torch.linspace(*ramp, n)[:, None].expand(n, hkv)
    flat = pages.scales[1].view(-1, hkv)
    flat[slots] = (flat[slots].double() * factor).float()
    v = pages.pools[1].view(-1, hkv, d)[slots].double() * flat[slots].double()[..., None]
    kp, vp, ks, vs = pages.cuda()
    q = torch.randn((170, hkv * group, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    lse = torch.empty((170, hkv * group), device="cuda")
    out = P.paged_cross_attention(q, _ints([0, 170]), kp, vp, row.view(1, -1).cuda(), _ints([n]), scale, k_scales=ks, v_scales=vs, lse_out=lse)
    check_rows(out, lse, q, k, v, scale, True, float(flat[slots].max()))


def test_cross_with_bad_input(P, rows_impl):
    hkv, group, d, bs, scale = 2, 2, 64, 16, 0.125
    pages = Paged(3, 20, hkv, d, bs, False)
    added = [pages.add(0, 64, 4) for _ in range(4)]
    kp, vp, _, _ = pages.cuda()
    tables = torch.stack([row for row, _ in added]).cuda()
    q = torch.randn((8, hkv * group, d), device="cuda").to(torch.bfloat16)
    starts = _ints([0, 2, 4, 6, 8])
    for lens, bad in (([64, -1, 65, 30], (1, 2)), ([2 ** 31 - 1, 64, 64, -2 ** 31], (0, 3))):
        lse = torch.full((8, hkv * group), 7.0, device="cuda")
        st = _status()
        out = P.paged_cross_attention(q, starts, kp, vp, tables, _ints(lens), scale, lse_out=lse, dev_status=st)
        assert int(st.item()) == P.DEV_BAD_LENGTH
        for s, x in enumerate(lens):
            n = 0 if s in bad else x
            check_rows(out[2 * s:2 * s + 2], lse[2 * s:2 * s + 2], q[2 * s:2 * s + 2], *(x[:n] for x in added[s][1]), scale, False)
    # a bad block: its tokens are rows of zeros
    for bad_id in (-1, 21, 2 ** 31 - 1):
        other = tables.clone()
        other[1, 2] = bad_id
        lse = torch.full((8, hkv * group), 7.0, device="cuda")
        st = _status()
        out = P.paged_cross_attention(q, starts, kp, vp, other, _ints([64] * 4), scale, lse_out=lse, dev_status=st)
        assert int(st.item()) == P.DEV_BAD_BLOCK_ID
        k, v = (x.clone() for x in added[1][1])
        k[32:48] = v[32:48] = 0
        check_rows(out[2:4], lse[2:4], q[2:4], k, v, scale, False)
        check_rows(out[4:6], lse[4:6], q[4:6], *added[2][1], scale, False)
    # starts that decrease or pass the rows: reported, and nothing outside the outputs is touched
    for bad_starts in ([0, 4, 2, 6, 8], [0, 2, 4, 6, 9], [-3, 2, 4, 6, 8], [0, 2, 2 ** 31 - 1, 6, 8]):
        st = _status()
        P.paged_cross_attention(q, _ints(bad_starts), kp, vp, tables, _ints([64] * 4), scale, dev_status=st)
        assert int(st.item()) & P.DEV_BAD_LENGTH


# ---- shared prefixes ---------------------------------------------------------------------

# sequences of each group, prefix of each, tokens behind it, sequences of no group, hkv, group, d, bs
SHARED = [
    ([1], [1], [1], 0, 1, 1, 64, 16),
    ([4], [100], [1, 40, 0, 17], 0, 2, 4, 64, 16),
    ([3, 2], [128, 0], [5, 0, 16, 3, 300], 2, 2, 8, 128, 16),
    ([1, 5, 1], [129, 257, 16], [1, 2, 3, 200, 5, 6, 7], 1, 1, 3, 128, 48),
    ([40], [1000], [i % 37 for i in range(40)], 0, 2, 7, 64, 32),
    ([70], [517], [(i * 13) % 90 for i in range(70)], 0, 8, 4, 128, 16),
    ([0, 6, 0], [64, 4000, 5], [700, 1, 20, 3, 90, 33], 0, 3, 5, 128, 64),
    ([33, 31], [2500, 300], [(i * 7) % 120 for i in range(64)], 3, 4, 1, 64, 256),
    ([10] * 12, [90 + 50 * i for i in range(12)], [i % 11 for i in range(120)], 0, 2, 2, 128, 16),
    ([1] * 20, [16 * i for i in range(20)], [3] * 20, 0, 8, 8, 64, 16),
    ([90], [300], [2] * 90, 0, 1, 6, 128, 16),
]


def _shared_case(sizes, prefixes, behind, loose, hkv, d, bs, int8, seed):
    """Pools, tables, lengths, starts and per sequence its K and V; `loose` sequences of 50 + i
    tokens that belong to no group come first."""
    n = loose + sum(sizes)
    per = [50 + i for i in range(loose)] + behind
    group = [-1] * loose + [g for g, m in enumerate(sizes) for _ in range(m)]
    pre = [0 if g < 0 else prefixes[g] for g in group]
    blocks = sum(-(-(p + x) // bs) - p // bs for p, x in zip(pre, per)) + sum(-(-p // bs) for p in prefixes)
    pages = Paged(seed, blocks + 2, hkv, d, bs, int8)
    wide_p, wide = max(max(-(-p // bs) for p in prefixes), 1), max(-(-(p + x) // bs) for p, x in zip(pre, per)) + 2
    shared = [pages.add(0, p, wide_p) for p in prefixes]
    own = [pages.add(p, p + x, wide) for p, x in zip(pre, per)]
    starts = [loose]
    for m in sizes:
        starts.append(starts[-1] + m)
    values = []
    for s in range(n):
        both = own[s][1] if group[s] < 0 else [torch.cat(x) for x in zip(shared[group[s]][1], own[s][1])]
        values.append(both)
    return (pages, torch.stack([r for r, _ in own]), [p + x for p, x in zip(pre, per)], starts,
            torch.stack([r for r, _ in shared]), values)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("sizes,prefixes,behind,loose,hkv,group,d,bs", SHARED)
def test_shared(P, sizes, prefixes, behind, loose, hkv, group, d, bs, int8, rows_impl):
    hq, scale = hkv * group, d ** -0.5
    pages, tables, ctx, starts, ptables, values = _shared_case(sizes, prefixes, behind, loose, hkv, d, bs, int8, len(behind))
    kp, vp, ks, vs = pages.cuda()
    n = len(ctx)
    gen = torch.Generator().manual_seed(3)
    q = torch.randn((n, hq + 2, d), generator=gen).to(torch.bfloat16).cuda()[:, 2:]
    lse = torch.full((n, hq), 7.0, device="cuda")
    st = _status()
    out = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(),
                                          _ints(prefixes), scale, k_scales=ks, v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s in range(n):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, int8)
    again = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(),
                                            _ints(prefixes), scale, k_scales=ks, v_scales=vs)
    assert torch.equal(again, out)


@pytest.mark.parametrize("groups", [33, 200])
def test_shared_of_many_groups(P, groups, rows_impl):
    r = random.Random(groups)
    sizes = [r.choice([0, 1, 2, 5]) for _ in range(groups)]
    prefixes = [r.choice([0, 1, 16, 100, 129]) for _ in range(groups)]
    behind = [r.choice([0, 1, 20]) for _ in range(sum(sizes))]
    hkv, group, d, bs, scale = 2, 2, 64, 16, 0.125
    pages, tables, ctx, starts, ptables, values = _shared_case(sizes, prefixes, behind, 3, hkv, d, bs, False, groups)
    kp, vp, _, _ = pages.cuda()
    q = torch.randn((len(ctx), hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    lse = torch.full((len(ctx), hkv * group), 7.0, device="cuda")
    st = _status()
    out = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(),
                                          _ints(prefixes), scale, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s in range(len(ctx)):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, False)


@pytest.mark.parametrize("int8", [False, True])
def test_shared_sequences_that_end_within_the_prefix(P, int8, rows_impl):
    """A sequence sees no more of its group's tokens than ctx_lens says; 0: an idle slot."""
    hkv, group, d, bs, scale = 2, 4, 128, 16, 0.09
    pages, tables, ctx, starts, ptables, values = _shared_case([9], [700], [3] * 9, 0, hkv, d, bs, int8, 4)
    ctx = [0, 1, 127, 128, 129, 699, 700, 701, 0]
    kp, vp, ks, vs = pages.cuda()
    q = torch.randn((9, hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    lse = torch.full((9, hkv * group), 7.0, device="cuda")
    st = _status()
    out = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints([700]),
                                          scale, k_scales=ks, v_scales=vs, lse_out=lse, dev_status=st)
    assert int(st.item()) == 0
    for s, x in enumerate(ctx):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *(v[:x] for v in values[s]), scale, int8)


def test_shared_equals_plain_decode_without_groups(P, rows_impl):
    """No group at all: the outputs of paged_decode_attention, within the bounds of both."""
    hkv, group, d, bs, scale = 2, 4, 64, 16, 0.125
    pages = Paged(8, 60, hkv, d, bs, False)
    added = [pages.add(0, x, 20) for x in (300, 1, 0, 90)]
    kp, vp, _, _ = pages.cuda()
    tables = torch.stack([r for r, _ in added]).cuda()
    q = torch.randn((4, hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    lse = torch.empty((4, hkv * group), device="cuda")
    none = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    out = P.paged_decode_attention_shared(q, kp, vp, tables, _ints([300, 1, 0, 90]), _ints([0]), none, _ints([]), scale, lse_out=lse)
    for s, x in enumerate(added):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *x[1], scale, False)


def test_shared_with_bad_input(P, rows_impl):
    hkv, group, d, bs, scale = 2, 2, 64, 16, 0.125
    sizes, prefixes = [3, 2, 2], [40, 64, 30]
    pages, tables, ctx, starts, ptables, values = _shared_case(sizes, prefixes, [9] * 7, 0, hkv, d, bs, False, 4)
    kp, vp, _, _ = pages.cuda()
    q = torch.randn((7, hkv * group, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()

    def run(ctx, starts, ptables, prefixes, tables=tables):
        lse, st = torch.full((7, hkv * group), 7.0, device="cuda"), _status()
        out = P.paged_decode_attention_shared(q, kp, vp, tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(),
                                              _ints(prefixes), scale, lse_out=lse, dev_status=st)
        return out, lse, int(st.item())

    def check(got, s, k, v):
        check_rows(got[0][s:s + 1], got[1][s:s + 1], q[s:s + 1], k, v, scale, False)

    # bad lengths of a sequence and of a group: their rows are empty, the others right
    bad_ctx = list(ctx)
    bad_ctx[1], bad_ctx[4] = -1, tables.shape[1] * bs + 1
    for wrong in (-5, 65, 2 ** 31 - 1):
        got = run(bad_ctx, starts, ptables, [40, 64, wrong])
        assert got[2] == P.DEV_BAD_LENGTH
        for s in range(7):
            n = 0 if s in (1, 4, 5, 6) else ctx[s]
            check(got, s, *(x[:n] for x in values[s]))
    # bad blocks, of a prefix and of a sequence: rows of zeros
    other, own = ptables.clone(), tables.clone()
    other[1, 1] = kp.shape[0]
    own[0, 3] = -7                              # tokens 48 .. 63: the last of the sequence's 49
    got = run(ctx, starts, other, prefixes, own)
    assert got[2] == P.DEV_BAD_BLOCK_ID
    for s in range(7):
        k, v = (x.clone() for x in values[s])
        if s in (3, 4):
            k[16:32] = v[16:32] = 0
        if s == 0:
            k[48:] = v[48:] = 0
        check(got, s, k, v)
    for bad_starts in ([0, 5, 3, 7], [0, 3, 5, 8], [-1, 3, 5, 7], [0, 3, 5, 2 ** 31 - 1]):
        assert run(ctx, bad_starts, ptables, prefixes)[2] & P.DEV_BAD_LENGTH


# ---- any call: streams, graphs, threads, large pools ---------------------------------------------

def test_rows_of_a_large_pool(P, rows_impl):
    """Pool offsets that pass 2^32 bytes and 2^31 elements."""
    hkv, group, d, bs, scale = 8, 1, 128, 16, 0.1
    n_blocks = 2 ** 31 // (bs * hkv * d) + 40
    pools = [torch.empty((n_blocks + 1, bs, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids = [n_blocks - 1, 3, n_blocks - 7, n_blocks - 20, 9]
    gen = torch.Generator().manual_seed(0)
    k, v = (torch.randn((80, hkv, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    slots = torch.tensor([ids[t // bs] * bs + t % bs for t in range(80)])
    P.paged_kv_write_slots(k.cuda(), v.cuda(), *pools, slots.cuda())
    assert torch.equal(pools[0].view(-1, hkv, d)[slots.cuda()].cpu(), k)
    q = torch.randn((3, hkv * group, d), generator=gen).to(torch.bfloat16).cuda()
    lse = torch.empty((3, hkv * group), device="cuda")
    table = _ints([ids])
    out = P.paged_cross_attention(q, _ints([0, 3]), *pools, table, _ints([80]), scale, lse_out=lse)
    check_rows(out, lse, q, k.double(), v.double(), scale, False)
    rows = table.expand(3, 5).contiguous()
    out = P.paged_decode_attention_shared(q, *pools, rows, _ints([80] * 3), _ints([0, 3]), table, _ints([37]), scale, lse_out=lse)
    check_rows(out, lse, q, k.double(), v.double(), scale, False)


def _step_state(P, seed, n=6, prefix=70, hkv=2, group=4, d=64, bs=16):
    """A batch behind one prompt: its prefix in the pool, the tables with the prefix's blocks."""
    gen = torch.Generator().manual_seed(seed)
    width, n_blocks = 16, 120
    pools = [torch.full((n_blocks + 1, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    whole = prefix // bs
    ptable = torch.arange(-(-prefix // bs), dtype=torch.int32).view(1, -1)
    kv = [torch.randn((prefix, hkv, d), generator=gen).to(torch.bfloat16) for _ in range(2)]
    slots = torch.arange(prefix)
    P.paged_kv_write_slots(kv[0].cuda(), kv[1].cuda(), *pools, slots.cuda())
    tables = torch.full((n, width), n_blocks, dtype=torch.int32)
    tables[:, :whole] = ptable[:, :whole]
    free = torch.randperm(n_blocks - 10, generator=gen).int() + 10
    if prefix % bs:                            # each sequence goes on in a block of its own, at the prefix's end
        tables[:, whole] = free[:n]
        free = free[n:]
    return dict(pools=pools, ptable=ptable.cuda(), tables=tables.cuda(), free=free.cuda(), kv=kv, gen=gen, n=n, prefix=prefix,
                hkv=hkv, hq=hkv * group, d=d, bs=bs, n_blocks=n_blocks)


def test_steps_together_in_a_graph(P, rows_impl):
    """Maps, slot writes and shared decode as a step of a layer, captured once and replayed with
    other tokens: every step against the 64-bit values of all tokens so far."""
    w = _step_state(P, 1)
    n, hkv, hq, d, scale, steps = w["n"], w["hkv"], w["hq"], w["d"], 0.125, 5
    lens, cursor = _ints([w["prefix"]] * n), _ints([0])
    new = _ints([1, 2, 1, 0, 1, 3][:n])
    total, rows = sum(new.tolist()), 10        # two rows of padding
    qkv = torch.zeros((rows, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    q1 = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
    m, st = P.StepMaps.empty(n, rows, "cuda"), _status()
    lse = torch.empty((n, hq), device="cuda")
    plan = P.SharedDecodePlan(*w["pools"], w["tables"], m.ctx_lens, _ints([0, n]), w["ptable"], _ints([w["prefix"]]), scale, hq,
                              lse_out=lse, dev_status=st)

    def step():
        P.paged_step_maps(lens, new, w["free"], w["tables"], w["bs"], w["n_blocks"], rows, cursor=cursor, out=m, dev_status=st)
        P.paged_kv_write_slots(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *w["pools"], m.slots, dev_status=st)
        plan.run(q1)
        lens.copy_(m.ctx_lens)
        cursor.copy_(m.cursor)

    def fill(i):
        gen = torch.Generator().manual_seed(100 + i)
        qkv.copy_(torch.randn(qkv.shape, generator=gen).to(torch.bfloat16))
        q1.copy_(torch.randn(q1.shape, generator=gen).to(torch.bfloat16))

    seen = [[x.double() for x in w["kv"]] for _ in range(n)]

    def check():
        rows_of = m.token_starts.tolist()
        for s in range(n):
            a, b = rows_of[s], rows_of[s + 1]
            seen[s] = [torch.cat([old, x[a:b].cpu().double()]) for old, x in zip(seen[s], (qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]))]
            check_rows(plan.out[s:s + 1], lse[s:s + 1], q1[s:s + 1], *seen[s], scale, False)
        assert int(st.item()) == 0 and m.token_starts.tolist()[-1] == total

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):              # one step outside the graph
        step()
    torch.cuda.current_stream().wait_stream(side)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, steps):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        check()


def test_maps_feed_cross_attention(P, rows_impl):
    """A packed batch from step maps: its queries against an encoder's pages."""
    new, keys, hkv, group, d, bs = [3, 0, 9, 1], [50, 7, 333, 16], 2, 4, 64, 16
    pages = Paged(6, 40, hkv, d, bs, False)
    added = [pages.add(0, x, 24) for x in keys]
    kp, vp, _, _ = pages.cuda()
    tab = torch.full((4, 8), 99, dtype=torch.int32, device="cuda")
    m = P.paged_step_maps(_ints([5, 6, 0, 15]), _ints(new), _ints(list(range(20))), tab, bs, 99, 16)
    q = torch.randn((16, hkv * group, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    lse = torch.empty((16, hkv * group), device="cuda")
    out = P.paged_cross_attention(q, m.token_starts, kp, vp, torch.stack([r for r, _ in added]).cuda(), _ints(keys), 0.1, lse_out=lse)
    for s, x in enumerate(added):
        a, b = m.token_starts.tolist()[s:s + 2]
        if a < b:
            check_rows(out[a:b], lse[a:b], q[a:b], *x[1], 0.1, False)


def test_calls_on_other_streams_and_threads(P, rows_impl):
    """Two threads, each on a stream of its own with tensors of its own."""
    hkv, group, d, bs, scale = 4, 4, 128, 16, 0.09
    results, errors = {}, []

    def work(i):
        try:
            pages, tables, ctx, starts, ptables, values = _shared_case([20], [600 + i], [(j * 5) % 30 for j in range(20)], 0, hkv, d, bs,
                                                                       bool(i & 1), i)
            kp, vp, ks, vs = pages.cuda()
            stream = torch.cuda.Stream()
            q = torch.randn((20, hkv * group, d), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
            lse = torch.empty((20, hkv * group), device="cuda")
            args = (tables.cuda(), _ints(ctx), _ints(starts), ptables.cuda(), _ints([600 + i]))
            torch.cuda.synchronize()
            for _ in range(20):
                out = P.paged_decode_attention_shared(q, kp, vp, *args, scale, k_scales=ks, v_scales=vs, lse_out=lse, stream=stream)
                cross = P.paged_cross_attention(q, args[2], kp, vp, args[3], args[4], scale, k_scales=ks, v_scales=vs, stream=stream)
            stream.synchronize()
            results[i] = (out, lse, cross, q, values, i)
        except Exception as e:      # noqa: BLE001 - shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for out, lse, cross, q, values, i in results.values():
        for s in range(20):
            check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1], *values[s], scale, bool(i & 1))
        assert torch.isfinite(cross).all()
