"""The calls for ragged batches on the CPU: refusals of the C calls before anything is
launched, refusals of the binding, workspace sizes, and the references."""
import pytest
import torch

from batch_reference import maps

FAKE, OTHER, MISALIGNED = 0x1000, 0x2000, 0x1008      # never dereferenced


@pytest.fixture(scope="module")
def P():
    from paged_kv_cache_212_gb300 import build as B
    try:
        B.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    B.build()
    import paged_kv_cache_212_gb300 as P
    P.load_library()
    return P


MAPS = ["lens", "n_new", "n_seqs", "free", "n_free", "cursor", "n_blocks", "bs", "tables", "width", "n_tokens", "ctx", "starts",
        "seqs", "positions", "slots", "cursor_out", "status", "stream"]


def _call(fn, names, base, **kw):
    args = dict(base, **kw)
    return fn(*(args[n] for n in names))


def test_maps_refusals(P):
    base = dict(lens=FAKE, n_new=FAKE, n_seqs=2, free=FAKE, n_free=4, cursor=FAKE, n_blocks=8, bs=16, tables=FAKE, width=4,
                n_tokens=3, ctx=OTHER, starts=FAKE, seqs=FAKE, positions=FAKE, slots=FAKE, cursor_out=OTHER, status=None, stream=None)
    f = P.load_library().paged_step_maps
    for kw, want in ((dict(bs=24), 2), (dict(bs=0), 1), (dict(bs=512), 2), (dict(n_blocks=-1), 1), (dict(n_seqs=-1), 1),
                     (dict(n_free=-1), 1), (dict(width=0), 1), (dict(n_tokens=-1), 1), (dict(width=2 ** 30), 3),
                     (dict(n_blocks=2 ** 28), 3), (dict(starts=None), 1), (dict(cursor_out=None), 1), (dict(cursor_out=FAKE), 1),
                     (dict(ctx=FAKE), 1), (dict(lens=None), 1), (dict(n_new=None), 1), (dict(tables=None), 1), (dict(ctx=None), 1),
                     (dict(free=None), 1), (dict(seqs=None), 1), (dict(positions=None), 1), (dict(slots=None), 1),
                     (dict(slots=0x1004), 1), (dict(lens=0x1002), 1), (dict(tables=0x1001), 1)):
        assert _call(f, MAPS, base, **kw) == want, kw


SLOTS = ["k", "ks", "v", "vs", "kp", "vp", "ksc", "vsc", "dt", "dims", "slots", "n", "status", "stream"]


def test_write_slots_refusals(P):
    base = dict(k=FAKE, ks=128, v=FAKE, vs=128, kp=FAKE, vp=FAKE, ksc=None, vsc=None, dt=0, dims=P.Dims(8, 16, 2, 64), slots=FAKE,
                n=3, status=None, stream=None)
    f = P.load_library().paged_kv_write_slots
    assert _call(f, SLOTS, base, n=0, k=None, v=None, kp=None, vp=None, slots=None) == 0
    for kw, want in ((dict(n=-1), 1), (dict(k=None), 1), (dict(v=MISALIGNED), 1), (dict(kp=None), 1), (dict(vp=MISALIGNED), 1),
                     (dict(slots=None), 1), (dict(slots=0x1004), 1), (dict(ks=120), 1), (dict(vs=132), 1), (dict(ks=-128), 1),
                     (dict(dt=2), 2), (dict(dt=1), 1), (dict(dt=1, ksc=FAKE, vsc=0x1002), 1), (dict(dims=P.Dims(8, 16, 2, 96)), 2),
                     (dict(dims=P.Dims(8, 24, 2, 64)), 2), (dict(dims=P.Dims(8, 16, 0, 64)), 1),
                     (dict(dims=P.Dims(2 ** 28, 16, 2, 64)), 3)):
        assert _call(f, SLOTS, base, **kw) == want, kw


CROSS = ["q", "qs", "hq", "starts", "n_rows", "kp", "vp", "ksc", "vsc", "dt", "dims", "tables", "width", "keys", "n_seqs", "scale", "out",
         "lse", "ws", "wsb", "status", "stream"]
SHARED = ["q", "qs", "hq", "kp", "vp", "ksc", "vsc", "dt", "dims", "tables", "width", "ctx", "n_seqs", "starts", "n_groups", "ptables",
          "pwidth", "plens", "scale", "out", "lse", "ws", "wsb", "status", "stream"]


def _rows_base(P):
    return dict(q=FAKE, qs=512, hq=8, kp=FAKE, vp=FAKE, ksc=None, vsc=None, dt=0, dims=P.Dims(8, 16, 2, 64), tables=FAKE, width=4,
                scale=0.125, out=OTHER, lse=None, ws=FAKE, wsb=1 << 30, status=None, stream=None, n_seqs=3, starts=FAKE,
                n_rows=5, keys=FAKE, ctx=FAKE, n_groups=2, ptables=FAKE, pwidth=3, plens=FAKE)


COMMON = ((dict(q=None), 1), (dict(q=MISALIGNED), 1), (dict(out=FAKE), 1), (dict(out=None), 1), (dict(kp=None), 1),
          (dict(vp=MISALIGNED), 1), (dict(lse=0x1002), 1), (dict(qs=504), 1), (dict(qs=516), 1), (dict(hq=7), 1), (dict(hq=0), 1),
          (dict(dt=2), 2), (dict(dt=1), 1), (dict(dt=1, ksc=FAKE, vsc=0x1002), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
          (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ws=None), 4), (dict(ws=0x1080), 4), (dict(wsb=1000), 4),
          (dict(tables=None), 1), (dict(starts=None), 1), (dict(width=0), 1), (dict(width=2 ** 27), 3))


def test_cross_refusals(P):
    f, base = P.load_library().paged_cross_attention, _rows_base(P)
    for kw, want in COMMON + ((dict(hq=34, qs=2176), 2), (dict(n_rows=-1), 1), (dict(n_seqs=-1), 1), (dict(keys=None), 1),
                              (dict(n_rows=2 ** 29), 3), (dict(dims=P.Dims(8, 16, 2, 96)), 2)):
        assert _call(f, CROSS, base, **kw) == want, kw
    assert _call(f, CROSS, base, n_rows=0, q=None, out=None, ws=None) == 0
    assert _call(f, CROSS, base, n_seqs=0, tables=None, keys=None) == 0


def test_shared_refusals(P):
    f, base = P.load_library().paged_decode_attention_shared, _rows_base(P)
    for kw, want in COMMON + ((dict(hq=18, qs=1152), 2), (dict(n_seqs=-1), 1), (dict(n_groups=-1), 1), (dict(ctx=None), 1),
                              (dict(ptables=None), 1), (dict(plens=None), 1), (dict(pwidth=0), 1), (dict(pwidth=-1), 1),
                              (dict(pwidth=2 ** 27), 3), (dict(n_seqs=2 ** 29), 3)):
        assert _call(f, SHARED, base, **kw) == want, kw
    assert _call(f, SHARED, base, n_seqs=0, q=None, out=None, ws=None, tables=None, ctx=None) == 0


def test_workspace_sizes(P):
    f = P.load_library().pkv_rows_workspace_bytes
    assert f(-1, 8, 64) == 0 and f(4, 0, 64) == 0 and f(4, 8, 96) == 0
    assert f(100, 8, 64) - f(0, 8, 64) == 100 * 8 * (2 * 64 + 8) * 4
    with pytest.raises(ValueError):
        P.rows_workspace_bytes(1, 8, 100)


def test_binding_refuses_cpu_tensors(P):
    t = torch.zeros((2, 2), dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    pool = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        P.paged_step_maps(one, one, one, t, 16, 8, 2)
    with pytest.raises(ValueError):
        P.paged_kv_write_slots(x, x, pool, pool, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        P.paged_cross_attention(x, torch.zeros(3, dtype=torch.int32), pool, pool, t, one, 0.1)
    with pytest.raises(ValueError):
        P.paged_decode_attention_shared(x, pool, pool, t, one, one, t, one, 0.1)
    with pytest.raises(TypeError):
        P.paged_cross_attention(None, one, pool, pool, t, one, 0.1)


def test_maps_reference():
    """The plain maps on a batch worked out by hand: blocks of 16, free list 7, 5, 3."""
    tables = [[9, 4, -1], [-1, -1, -1], [2, -1, -1]]
    got = maps([20, 0, 16], [13, 2, 1], [7, 5, 3], 0, tables, 16, 10, 18)
    assert tables == [[9, 4, 7], [5, 10, 10], [2, 3, -1]]
    assert got[0] == [33, 2, 17] and got[1] == [0, 13, 15, 16] and got[5] == 3 and got[6] == 0
    assert got[2] == [0] * 13 + [1] * 2 + [2] + [-1] * 2
    assert got[3] == list(range(20, 33)) + [0, 1, 16, 0, 0]
    assert got[4] == [4 * 16 + i for i in range(4, 16)] + [7 * 16, 80, 81, 48, -1, -1]
