"""Rotary page writes and sliding-window attention over a paged KV cache: inputs,
plain forms and 64-bit values for measuring them.

Four operators, each over pools [n_blocks + 1, block_size, Hkv, D] reached through
int32 block tables (token t of a sequence: row table[t // bs] * bs + t % bs):

* "rope_write": q and k of n_new tokens per sequence are turned by the angle of
  their positions (half or interleaved pairs, rot_dim of the D elements, scaled
  frequencies), k and v go into the pages (bf16, or int8 codes with one fp32
  absmax / 127 scale per row), the turned q is returned.
* "decode": one query per sequence at position ctx - 1 sees the first `sinks`
  tokens and the last `window` ones.
* "prefill": query i of a chunk sits at prefix + i and sees the tokens t <= prefix + i
  with t < sinks or t > prefix + i - window.
* "step": rope_write of one token per sequence, then decode, as one layer's step.

With ``own`` false, run() computes in torch in 32 bits; with ``own`` true it calls
paged_kv_cache_212_gb300.
"""
import math
import random

import torch

own = False


# ----------------------------------------------------------------------------- cases

def _case(name, op, lens, n, lo, hi, hq, hkv, d, bs, **more):
    c = {"name": name, "op": op, "lens": lens, "n": n, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d, "bs": bs,
         "int8": False, "n_new": 1, "window": 0, "sinks": 0, "rot": 0, "base": 10000.0, "inter": False,
         "scaling": "none", "factor": 1.0, "orig": 4096}
    c.update(more)
    return c


def listed():
    return [
        # a prefill chunk's q, k, v straight from the fused projection, frequencies scaled in bands
        _case("rope write chunk", "rope_write", 1, 8, 0, 8191, 32, 8, 128, 16, n_new=512, rot=128, base=500000.0,
              scaling="bands", factor=8.0, orig=8192),
        # one decode token for each of 64 sequences, half of the head turned, interleaved pairs
        _case("rope write tokens", "rope_write", 2, 64, 512, 4096, 32, 8, 128, 16, rot=64, inter=True,
              scaling="linear", factor=4.0),
        # fresh ragged-size prompts into int8 pages
        _case("rope write int8", "rope_write", 3, 5, 0, 40, 32, 8, 128, 16, n_new=301, rot=128, int8=True,
              scaling="yarn", factor=4.0),
        # the smallest decode: four short sequences
        _case("decode tiny", "decode", 4, 4, 17, 255, 8, 2, 64, 16, window=64, sinks=4),
        # a serving batch, most contexts longer than the window
        _case("decode batch", "decode", 5, 64, 512, 4096, 32, 8, 128, 16, window=1024, sinks=4),
        # the same over int8 pages with eight query heads per kv head
        _case("decode batch int8", "decode", 6, 64, 512, 4096, 64, 8, 128, 16, window=1024, sinks=4, int8=True),
        # few long sequences: the window has to be split over the machine
        _case("decode long", "decode", 7, 2, 20011, 32768, 64, 8, 128, 32, window=16384, sinks=64),
        # a small odd chunk
        _case("prefill small", "prefill", 8, 2, 5, 300, 8, 2, 64, 16, n_new=37, window=100, sinks=3),
        # chunked prefill behind resident prefixes
        _case("prefill chunk", "prefill", 9, 8, 0, 8191, 32, 8, 128, 16, n_new=512, window=1024, sinks=4),
        # one long prompt at once
        _case("prefill prompt", "prefill", 10, 1, 0, 0, 32, 8, 128, 16, n_new=4095, window=1000, sinks=16),
        # one layer's step of the smallest batch, and of the serving batch
        _case("step tiny", "step", 11, 4, 17, 255, 8, 2, 64, 16, window=64, sinks=4, rot=64),
        _case("step batch", "step", 12, 64, 512, 4096, 32, 8, 128, 16, window=1024, sinks=4, rot=128,
              base=500000.0, scaling="ntk", factor=4.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_write", "decode", "prefill", "step"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32, 64])
    more = {}
    if op in ("rope_write", "step"):
        more["rot"] = rng.choice([d, d, d // 2])
        more["base"] = rng.choice([10000.0, 500000.0])
        more["inter"] = rng.random() < 0.4
        more["scaling"] = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
        more["factor"] = 1.0 if more["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
    if op in ("decode", "prefill", "step"):
        more["sinks"] = rng.choice([0, 1, 4, 16, 33])
    if op == "rope_write":
        n = _log(rng, 1, 64)
        more["n_new"] = _log(rng, 1, max(1, 4096 // n))
        more["int8"] = rng.random() < 0.4
        lo, hi = 0, _log(rng, 16, 2048)
    elif op == "prefill":
        n = _log(rng, 1, 8)
        more["n_new"] = _log(rng, 2, 4095 * 32 // max(32, hkv * g) // n)
        more["window"] = _log(rng, 32, 1024)
        lo, hi = 0, _log(rng, 16, 8191)
    else:
        n = _log(rng, 1, 64)
        more["window"] = _log(rng, 32, 1024 if n > 4 else 8192)
        more["int8"] = op == "decode" and rng.random() < 0.5
        hi = _log(rng, 64, 4096 if n > 4 else 16384)
        lo = hi // 8
    c = _case("", op, rng.randrange(1 << 30), n, lo, hi, hkv * g, hkv, d, bs, **more)
    del c["name"]
    return c


def _stored(case):
    """Tokens resident before the step, per sequence (the same for every seed)."""
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def _visible(length, window, sinks):
    a = min(sinks, length)
    return a + length - max(a, length - window)


def work(case):
    n, n_new, hq, hkv, d = (case[k] for k in ("n", "n_new", "hq", "hkv", "d"))
    stored, row = _stored(case), hkv * d
    kv = row * (1 if case["int8"] else 2) + (hkv * 4 if case["int8"] else 0)      # one stored row of K or of V
    new = n * n_new * (hq * d + 2 * row) * 2                                       # q, k, v as they come
    if case["op"] == "rope_write":
        return {"bytes": new + n * n_new * (hq * d * 2 + 2 * kv), "flops": n * n_new * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "prefill":
        keys = sum(min(case["sinks"], p + n_new) + p + n_new - max(min(case["sinks"], p + n_new), p - case["window"] + 1, 0)
                   for p in stored)
        pairs = sum(_visible(p + i + 1, case["window"], case["sinks"]) for p in stored for i in range(n_new))
        return {"bytes": keys * 2 * kv + 2 * n * n_new * hq * d * 2, "flops": 4 * pairs * hq * d}
    seen = sum(_visible(p + 1, case["window"], case["sinks"]) for p in stored)
    b = seen * 2 * kv + n * hq * d * 2 * 2
    if case["op"] == "step":      # the new row is written, and attended without being read back
        b += n * 2 * row * 2
    return {"bytes": b, "flops": 4 * seen * hq * d}


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    n, n_new, hq, hkv, d, bs = (case[k] for k in ("n", "n_new", "hq", "hkv", "d", "bs"))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    stored = _stored(case)
    blocks = [-(-(p + n_new) // bs) for p in stored]
    n_blocks, width = sum(blocks) + 3, max(blocks)
    perm = torch.randperm(n_blocks, generator=gen, device=dev).to(torch.int32).cpu()
    tables = torch.full((n, width), n_blocks, dtype=torch.int32)
    at = 0
    for s, b in enumerate(blocks):
        tables[s, :b] = perm[at:at + b]
        at += b
    st = {"case": case, "scale": 1.0 / math.sqrt(d), "tables": tables.to(dev),
          "stored": torch.tensor(stored, dtype=torch.int32, device=dev)}
    st["ctx"] = st["stored"] + n_new
    shape = (n_blocks + 1, bs, hkv, d)
    for x in ("k", "v"):
        if case["int8"]:
            st[x + "p"] = torch.randint(-127, 128, shape, generator=gen, device=dev, dtype=torch.int8)
            st[x + "s"] = torch.rand(shape[:3], generator=gen, device=dev) * 0.015 + 0.015
        else:
            st[x + "p"] = torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)
            st[x + "s"] = None
    # the most tokens that one sequence's query (or chunk) sees, known to the host that scheduled them
    st["span"] = max(min(case["sinks"] + case["window"] + n_new - 1, p + n_new) for p in stored)
    if case["op"] in ("rope_write", "step"):
        # the fused projection's rows: q heads, k heads, v heads of each token side by side
        qkv = torch.randn((n, n_new, hq + 2 * hkv, d), generator=gen, device=dev).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv.split((hq, hkv, hkv), dim=2)
        st["inv_freq"], st["magnitude"] = _frequencies(case)
        st["inv_freq"] = st["inv_freq"].to(dev)
        if case["op"] == "step":
            st["q"] = st["q"][:, 0]
        if own:
            import paged_kv_cache_212_gb300 as P
            st["rope"] = P.Rope(case["rot"], base=case["base"], interleaved=case["inter"], scaling=case["scaling"],
                                factor=case["factor"], original_context=case["orig"], device=dev)
    else:
        q_shape = (n, hq, d) if case["op"] == "decode" else (n, n_new, hq, d)
        st["q"] = torch.randn(q_shape, generator=gen, device=dev).to(torch.bfloat16)
    if own and case["op"] in ("decode", "step"):
        import paged_kv_cache_212_gb300 as P
        st["plan"] = P.WindowDecodePlan(st["kp"], st["vp"], st["tables"], st["ctx"], st["scale"], hq,
                                        case["window"], sinks=case["sinks"], rope=st.get("rope"), k_scales=st["ks"],
                                        v_scales=st["vs"])
    return st


def _frequencies(case):
    """Radians per position of each pair (64 bits), and the factor on the turned elements."""
    rot, base, factor, orig = case["rot"], case["base"], case["factor"], case["orig"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        inv = inv / factor
    elif case["scaling"] == "bands":        # kept above orig / 4 turns, divided below orig / 1, blended between
        turns = orig * inv / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        inv = inv * keep + inv / factor * (1 - keep)
    elif case["scaling"] == "yarn":         # a ramp over the pairs between those of 32 turns and of 1 turn in orig
        lo, hi = (rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        divide = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        inv = inv * (1 - divide) + inv / factor * divide
        return inv, 0.1 * math.log(factor) + 1.0
    return inv, 1.0


# ----------------------------------------------------------------------------- plain forms

def _rows(st, pos):
    """Pool rows of positions [n, m]."""
    bs = st["case"]["bs"]
    return torch.gather(st["tables"].long(), 1, pos // bs) * bs + pos % bs


def _turned(st, x, pos):
    """x [n, m, heads, D] in 32 bits, turned by its positions [n, m]; the angles in 64 bits."""
    rot = st["case"]["rot"]
    angle = pos.double().unsqueeze(-1) * st["inv_freq"]
    cos = (torch.cos(angle) * st["magnitude"]).float().unsqueeze(2)
    sin = (torch.sin(angle) * st["magnitude"]).float().unsqueeze(2)
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if st["case"]["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _store(st, x, rows, pool, scales):
    c = st["case"]
    flat = pool.view(-1, c["hkv"], c["d"])
    if c["int8"]:
        scale = x.abs().amax(dim=-1) / 127.0
        code = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)).clamp(-127, 127)
        flat[rows] = code.to(torch.int8)
        scales.view(-1, c["hkv"])[rows] = scale
    else:
        flat[rows] = x.to(torch.bfloat16)


def _loaded(st, rows, pool, scales):
    c = st["case"]
    x = pool.view(-1, c["hkv"], c["d"])[rows].float()
    return x * scales.view(-1, c["hkv"])[rows].unsqueeze(-1) if c["int8"] else x


def _values(st, pool, scales):
    """What the pages stand for."""
    if not st["case"]["int8"]:
        return pool
    return torch.mul(pool, scales.unsqueeze(-1), out=torch.empty_like(pool, dtype=torch.bfloat16))


def _write_plain(st, q):
    c = st["case"]
    pos = st["stored"].long().unsqueeze(1) + torch.arange(c["n_new"], device=q.device)
    rows = _rows(st, pos)
    _store(st, _turned(st, st["k"], pos), rows, st["kp"], st["ks"])
    _store(st, st["v"].float(), rows, st["vp"], st["vs"])
    return _turned(st, q, pos)


def _attend_plain(st, q):
    """q [n, m, Hq, D] in 32 bits, query i at position ctx - m + i."""
    c = st["case"]
    n, m, hq, d = q.shape
    hkv, window, sinks = c["hkv"], c["window"], c["sinks"]
    last = st["ctx"].long().unsqueeze(1)                                      # one past the last query
    slot = torch.arange(st["span"], device=q.device).unsqueeze(0)
    first = torch.clamp(last, max=sinks)                                      # tokens seen as first ones
    low = torch.maximum(first, last - m + 1 - window)                         # and from here on
    tok = torch.where(slot < first, slot, low + slot - first)
    there = tok < last
    rows = _rows(st, torch.minimum(tok, last - 1))
    k, v = _loaded(st, rows, st["kp"], st["ks"]), _loaded(st, rows, st["vp"], st["vs"])
    qpos = (last - m + torch.arange(m, device=q.device)).unsqueeze(2)         # [n, m, 1]
    tok, there = tok.unsqueeze(1), there.unsqueeze(1)
    seen = there & (tok <= qpos) & ((tok < sinks) | (tok > qpos - window))    # [n, m, span]
    qg = q.view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)).mul_(st["scale"]).view(n, hkv, hq // hkv, m, -1)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    p = torch.exp_(s.sub_(s.amax(dim=-1, keepdim=True)))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, -1, p.shape[-1]), v.transpose(1, 2)).view(n, hkv, hq // hkv, m, d) / total
    return o.permute(0, 3, 1, 2, 4).reshape(n, m, hq, d).to(torch.bfloat16)


def _run_plain(st):
    op = st["case"]["op"]
    if op == "rope_write":
        q = _write_plain(st, st["q"]).to(torch.bfloat16)
        return {"q": q, "k_pool": _values(st, st["kp"], st["ks"]), "v_pool": _values(st, st["vp"], st["vs"])}
    if op == "prefill":
        return {"out": _attend_plain(st, st["q"].float())}
    if op == "decode":
        return {"out": _attend_plain(st, st["q"].float().unsqueeze(1)).squeeze(1)}
    q = _write_plain(st, st["q"].unsqueeze(1))
    return {"out": _attend_plain(st, q).squeeze(1), "k_pool": st["kp"], "v_pool": st["vp"]}


# ----------------------------------------------------------------------------- the framework's calls

def _run_own(st):
    import paged_kv_cache_212_gb300 as P
    c = st["case"]
    if c["op"] == "rope_write":
        q = P.paged_kv_write_rope(st["q"], st["k"], st["v"], st["rope"], st["kp"], st["vp"], st["tables"], st["stored"],
                                  k_scales=st["ks"], v_scales=st["vs"])
        return {"q": q, "k_pool": _values(st, st["kp"], st["ks"]), "v_pool": _values(st, st["vp"], st["vs"])}
    if c["op"] == "prefill":
        return {"out": P.paged_prefill_attention_window(st["q"], st["kp"], st["vp"], st["tables"], st["stored"], st["scale"],
                                                        c["window"], sinks=c["sinks"])}
    if c["op"] == "decode":
        return {"out": st["plan"].run(st["q"])}
    return {"out": st["plan"].run(st["q"], st["k"], st["v"], st["stored"]), "k_pool": st["kp"], "v_pool": st["vp"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- 64 bits

def _exact_turn(x, inv, magnitude, first, rot, inter):
    """x [m, heads, D] (64 bits) as complex pairs times magnitude * exp(i position inv)."""
    pos = torch.arange(first, first + x.shape[0], device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.full_like(pos, magnitude)[:, None].expand(-1, inv.numel()).contiguous(),
                       pos[:, None] * inv[None, :])[:, None, :]
    y = x.clone()
    if inter:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        h = rot // 2
        z = torch.complex(x[..., :h].contiguous(), x[..., h:rot].contiguous()) * turn
        y[..., :h], y[..., h:rot] = z.real, z.imag
    return y


def _exact_page(x, int8):
    """The values that rows x [m, Hkv, D] are stored as: nearest bf16, or nearest of 255 steps of absmax / 127."""
    if not int8:
        return x.to(torch.bfloat16).double()
    step = x.abs().amax(dim=-1, keepdim=True) / 127
    return torch.where(step > 0, torch.round(x / step.clamp(min=1e-300)) * step, torch.zeros_like(x))


def exact(case, seed):
    st = prepare(case, seed)
    n, n_new, hq, hkv, d, bs = (case[k] for k in ("n", "n_new", "hq", "hkv", "d", "bs"))
    stored, tables = _stored(case), st["tables"].cpu().tolist()

    def pages(pool, scales):
        x = pool.double().view(-1, hkv, d)
        return x * scales.double().view(-1, hkv, 1) if scales is not None else x

    kp, vp = pages(st["kp"], st["ks"]), pages(st["vp"], st["vs"])
    rows = [torch.tensor([tables[s][t // bs] * bs + t % bs for t in range(p + n_new)], device=kp.device)
            for s, p in enumerate(stored)]
    q = st["q"].double().view(n, n_new, hq, d) if case["op"] != "step" else st["q"].double().unsqueeze(1)
    if case["op"] in ("rope_write", "step"):
        inv = st["inv_freq"].double()
        turned = torch.empty(n, n_new, hq, d, dtype=torch.float64, device=kp.device)
        for s, p in enumerate(stored):
            turned[s] = _exact_turn(q[s], inv, st["magnitude"], p, case["rot"], case["inter"])
            k = _exact_turn(st["k"][s].double(), inv, st["magnitude"], p, case["rot"], case["inter"])
            kp[rows[s][p:]] = _exact_page(k, case["int8"])
            vp[rows[s][p:]] = _exact_page(st["v"][s].double(), case["int8"])
        q = turned
    pools = {"k_pool": kp.view(st["kp"].shape), "v_pool": vp.view(st["vp"].shape)}
    if case["op"] == "rope_write":
        return {"q": q, **pools}
    out = torch.empty(n, n_new, hq, d, dtype=torch.float64, device=kp.device)
    for s, p in enumerate(stored):
        t = torch.arange(p + n_new, device=kp.device)
        here = torch.arange(p, p + n_new, device=kp.device)[:, None]
        hidden = (t > here) | ((t >= case["sinks"]) & (t <= here - case["window"]))
        for h in range(hkv):
            k, v = kp[rows[s], h], vp[rows[s], h]
            qs = q[s, :, h * (hq // hkv):(h + 1) * (hq // hkv)].transpose(0, 1)                    # [G, m, D]
            w = torch.softmax((qs @ k.T * st["scale"]).masked_fill(hidden, -math.inf), dim=-1)
            out[s, :, h * (hq // hkv):(h + 1) * (hq // hkv)] = (w @ v).transpose(0, 1)
    if case["op"] == "prefill":
        return {"out": out}
    return {"out": out[:, 0]} if case["op"] == "decode" else {"out": out[:, 0], **pools}
