"""Calls for batches of requests of any lengths over a paged KV cache: inputs, plain
forms and 64-bit values for measuring them.

Four operators, over pools [n_blocks + 1, block_size, Hkv, D] reached through int32
block tables (token t of a sequence: row table[t // bs] * bs + t % bs):

* "maps": from the tokens that each request holds and adds, the blocks it takes from a
  free list (written into its table row), and for every new token of the packed batch
  its sequence, position and pool row.
* "write": packed k and v rows go to their pool rows (bf16, or int8 codes with one fp32
  absmax / 127 scale per row).
* "cross": packed queries, some per sequence, see all of their sequence's keys.
* "shared": one query per sequence; the sequences of a group share their first tokens,
  which lie in the group's own pages, and each goes on in pages of its own.

With ``own`` false, run() computes in torch in 32 bits; with ``own`` true it calls
paged_kv_cache_212_gb300.
"""
import math
import random

import torch

own = False


# ----------------------------------------------------------------------------- cases

def _case(name, op, lens, n, lo, hi, hq, hkv, d, bs, **more):
    """n sequences that hold lo .. hi tokens (of keys; "shared": behind the prefix)."""
    c = {"name": name, "op": op, "lens": lens, "n": n, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d, "bs": bs,
         "int8": False, "new_lo": 1, "new_hi": 1, "pad": 0, "fresh": 0.0, "groups": 1, "pre_lo": 0, "pre_hi": 0}
    c.update(more)
    return c


def listed():
    return [
        # one decode step of a serving batch: a token each, a block now and then
        _case("maps step", "maps", 1, 64, 1, 4096, 32, 8, 128, 16),
        # a mixed batch padded to a fixed size: prompts that start, chunks that go on, single tokens, idle slots
        _case("maps mixed", "maps", 2, 500, 0, 4096, 32, 8, 128, 16, new_lo=0, new_hi=260, pad=1000, fresh=0.4),
        # ragged chunks of a mixed batch, k and v parts of the fused projection's rows
        _case("write chunks", "write", 3, 24, 0, 2048, 32, 8, 128, 16, new_lo=1, new_hi=700, pad=130),
        # a token each into int8 pages
        _case("write tokens int8", "write", 4, 64, 1, 4096, 32, 8, 128, 16, int8=True),
        # the smallest decode against encoder states
        _case("cross tiny", "cross", 5, 4, 17, 255, 8, 2, 64, 16),
        # one token per sequence against encoder states of ragged lengths
        _case("cross step", "cross", 6, 64, 512, 4096, 32, 8, 128, 16),
        # packed ragged targets against encoder states, int8 pages
        _case("cross ragged int8", "cross", 7, 12, 0, 1500, 24, 8, 64, 32, new_lo=1, new_hi=333, int8=True),
        # whole targets at once against long sources
        _case("cross targets", "cross", 8, 8, 1000, 8191, 32, 8, 128, 16, new_lo=200, new_hi=800),
        # four short continuations of one short prompt
        _case("shared tiny", "shared", 9, 4, 1, 40, 8, 2, 64, 16, pre_lo=100, pre_hi=100),
        # a serving batch behind one system prompt
        _case("shared batch", "shared", 10, 64, 16, 512, 32, 8, 128, 16, pre_lo=4096, pre_hi=4096),
        # several long prompts, each sampled many times, eight query heads per kv head
        _case("shared groups", "shared", 11, 256, 1, 700, 64, 8, 128, 16, groups=6, pre_lo=2000, pre_hi=16384),
        # the same kind of batch over int8 pages
        _case("shared batch int8", "shared", 12, 96, 16, 512, 32, 8, 128, 16, groups=2, pre_lo=3000, pre_hi=8000,
              int8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["maps", "write", "cross", "shared"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    bs = rng.choice([16, 32, 64, 128])
    more = {}
    if op != "maps":
        more["int8"] = rng.random() < 0.4
    if op in ("maps", "write"):
        n = _log(rng, 1, 512)
        hi = _log(rng, 1, 4096)
        lo = rng.choice([0, hi // 8])
        if rng.random() < 0.6:
            more["new_lo"] = 0
            more["new_hi"] = _log(rng, 1, max(1, (120000 if op == "maps" else 16000) // n))
        more["pad"] = rng.choice([0, _log(rng, 1, 500)])
        more["fresh"] = rng.choice([0.0, 0.3])
    elif op == "cross":
        n = _log(rng, 1, 64)
        hi = _log(rng, 16, 8191)
        lo = rng.choice([0, hi // 8])
        if rng.random() < 0.6:
            more["new_lo"] = 1
            more["new_hi"] = _log(rng, 2, max(2, min(1000, 4096 // n * 32 // max(32, hkv * g))))
    else:
        n = _log(rng, 1, 256)
        hi = _log(rng, 1, 700)
        lo = rng.choice([1, 1 + hi // 8])
        hi = max(hi, lo)
        more["groups"] = min(n, _log(rng, 1, max(1, n)))
        more["pre_hi"] = _log(rng, 16, max(16, 16384 // more["groups"]))
        more["pre_lo"] = rng.choice([0, more["pre_hi"] // 2, more["pre_hi"]])
    c = _case("", op, rng.randrange(1 << 30), n, lo, hi, hkv * g, hkv, d, bs, **more)
    del c["name"]
    return c


def _lengths(case):
    """Tokens that each sequence holds, tokens that it adds (or queries with), and the groups'
    first sequences and prefix lengths (the same for every seed)."""
    r = random.Random(case["lens"])
    held = [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n"])]
    if sum(new) == 0:
        new[0] = 1
    held = [0 if r.random() < case["fresh"] else h for h in held]
    cuts = sorted(r.sample(range(1, case["n"]), case["groups"] - 1))
    return held, new, [0] + cuts + [case["n"]], [r.randint(case["pre_lo"], case["pre_hi"]) for _ in range(case["groups"])]


def work(case):
    held, new, starts, prefix = _lengths(case)
    hq, hkv, d, bs, n = (case[k] for k in ("hq", "hkv", "d", "bs", "n"))
    kv = hkv * d * (1 if case["int8"] else 2) + (hkv * 4 if case["int8"] else 0)      # one stored row of K or of V
    tokens = sum(new)
    if case["op"] == "maps":
        added = sum(-(-(h + m) // bs) - -(-h // bs) for h, m in zip(held, new))
        tail = sum(_width(case) - -(-m // bs) for h, m in zip(held, new) if h == 0)
        last = sum(1 for h, m in zip(held, new) if m and h % bs)
        return {"bytes": 16 * n + 16 * (tokens + case["pad"]) + 8 * added + 4 * (tail + last), "flops": tokens}
    if case["op"] == "write":
        return {"bytes": tokens * (2 * hkv * d * 2 + 2 * kv + 8), "flops": tokens * 2 * hkv * d * (2 if case["int8"] else 0)}
    if case["op"] == "cross":
        return {"bytes": tokens * hq * d * 4 + sum(held) * 2 * kv, "flops": 4 * hq * d * sum(h * m for h, m in zip(held, new))}
    seen = sum(prefix[g] * (starts[g + 1] - starts[g]) for g in range(case["groups"])) + sum(held)
    return {"bytes": n * hq * d * 4 + (sum(prefix) + sum(held)) * 2 * kv, "flops": 4 * hq * d * seen}


def _width(case):
    """Blocks that a table row has room for."""
    held, new, _, _ = _lengths(case)
    if case["op"] in ("maps", "write"):
        return max(-(-(h + m) // case["bs"]) for h, m in zip(held, new)) + 8
    return -(-max(max(held), 1) // case["bs"])


# ----------------------------------------------------------------------------- inputs

def _tables(counts, width, perm, at, scratch):
    """Rows of `width` block ids, the first counts[s] of them taken from perm[at:]."""
    rows = torch.full((len(counts), width), scratch, dtype=torch.int32)
    for s, b in enumerate(counts):
        rows[s, :b] = perm[at:at + b]
        at += b
    return rows, at


def prepare(case, seed):
    n, hq, hkv, d, bs = (case[k] for k in ("n", "hq", "hkv", "d", "bs"))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    held, new, starts, prefix = _lengths(case)
    st = {"case": case, "scale": 1.0 / math.sqrt(d)}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def up(x):
        return -(-x // bs)

    tokens = sum(new)
    if case["op"] == "maps":
        need = sum(up(h + m) - up(h) for h, m in zip(held, new))
        used = sum(up(h) for h in held)
        st["n_blocks"] = used + need + 40
        perm = torch.randperm(st["n_blocks"], generator=gen, device=dev).to(torch.int32).cpu()
        rows, at = _tables([up(h) for h in held], _width(case), perm, 0, st["n_blocks"])
        # the free list, of which earlier steps have taken some
        st["free"], st["cursor"] = perm[max(at - 7, 0):].to(dev), ints([min(at, 7)])
        st["tables"], st["n_tokens"] = rows.to(dev), tokens + case["pad"]
        st["held"], st["new"] = ints(held), ints(new)
        if own:      # the outputs, which a program keeps from step to step
            import paged_kv_cache_212_gb300 as P
            st["maps"] = P.StepMaps.empty(n, st["n_tokens"], dev)
        return st
    counts = [up(h + m) for h, m in zip(held, new)] if case["op"] == "write" else [up(h) for h in held]
    shared = [up(p) for p in prefix]
    if case["op"] == "shared":
        counts = [up(prefix[g] + held[s]) - prefix[g] // bs for g in range(case["groups"])
                  for s in range(starts[g], starts[g + 1])]
    n_blocks = sum(counts) + (sum(shared) if case["op"] == "shared" else 0) + 3
    perm = torch.randperm(n_blocks, generator=gen, device=dev).to(torch.int32).cpu()
    shape = (n_blocks + 1, bs, hkv, d)
    for x in ("k", "v"):
        if case["int8"]:
            st[x + "p"] = torch.randint(-127, 128, shape, generator=gen, device=dev, dtype=torch.int8)
            st[x + "s"] = torch.rand(shape[:3], generator=gen, device=dev) * 0.015 + 0.015
        else:
            st[x + "p"] = torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)
            st[x + "s"] = None
    if case["op"] == "write":
        rows, _ = _tables(counts, max(counts), perm, 0, n_blocks)
        at = [(rows[s, t // bs].long() * bs + t % bs) for s in range(n)
              for t in [torch.arange(held[s], held[s] + new[s])]]
        # a batch of a fixed size: the rows behind the last token go nowhere
        st["slots"] = torch.cat(at + [torch.full((case["pad"],), -1)]).to(dev)
        st["tokens"] = tokens
        qkv = torch.randn((tokens + case["pad"], hq + 2 * hkv, d), generator=gen, device=dev).to(torch.bfloat16)
        _, st["k"], st["v"] = qkv.split((hq, hkv, hkv), dim=1)
        return st
    if case["op"] == "cross":
        rows, _ = _tables(counts, _width(case), perm, 0, n_blocks)
        st["keys"] = ints(held)
        st["starts"] = torch.cat([ints([0]), torch.cumsum(ints(new), 0, dtype=torch.int32)])
        st["span"], st["most"] = max(max(held), 1), max(new)
        st["q"] = torch.randn((tokens, hq, d), generator=gen, device=dev).to(torch.bfloat16)
        st["tables"] = rows.to(dev)
        if own:
            import paged_kv_cache_212_gb300 as P
            st["ws"] = torch.empty(P.rows_workspace_bytes(tokens, hq, d), dtype=torch.uint8, device=dev)
        return st
    # "shared": a sequence's row has the blocks wholly inside the prefix from the group's row, then its own
    pre, at = _tables(shared, max(max(shared), 1), perm, 0, n_blocks)
    group = [g for g in range(case["groups"]) for _ in range(starts[g], starts[g + 1])]
    width = max(up(prefix[group[s]] + held[s]) for s in range(n))
    rows = torch.full((n, width), n_blocks, dtype=torch.int32)
    for s in range(n):
        whole = prefix[group[s]] // bs
        rows[s, :whole] = pre[group[s], :whole]
        rows[s, whole:whole + counts[s]] = perm[at:at + counts[s]]
        at += counts[s]
    st["tables"], st["prefix_tables"] = rows.to(dev), pre.to(dev)
    st["starts"], st["prefix"] = ints(starts), ints(prefix)
    st["group"] = ints(group)
    st["ctx"] = st["prefix"][st["group"].long()] + ints(held)
    st["bounds"], st["lengths"] = starts, prefix
    st["q"] = torch.randn((n, hq, d), generator=gen, device=dev).to(torch.bfloat16)
    st["span"] = max(held)
    if own:
        import paged_kv_cache_212_gb300 as P
        st["plan"] = P.SharedDecodePlan(st["kp"], st["vp"], st["tables"], st["ctx"], st["starts"], st["prefix_tables"],
                                        st["prefix"], st["scale"], hq, k_scales=st["ks"], v_scales=st["vs"])
    return st


# ----------------------------------------------------------------------------- plain forms

def _maps_plain(st):
    bs, scratch = st["case"]["bs"], st["n_blocks"]
    held, new, tables, free = st["held"].long(), st["new"].long(), st["tables"], st["free"]
    dev, width = tables.device, tables.shape[1]
    ctx = held + new
    old, want = (held + bs - 1) // bs, (ctx + bs - 1) // bs
    need = want - old
    first = torch.cumsum(need, 0) - need + st["cursor"].long()
    ends = torch.cumsum(new, 0)
    col = torch.arange(width, device=dev).unsqueeze(0)
    place = (first.unsqueeze(1) + col - old.unsqueeze(1)).clamp(0, free.numel() - 1)
    added = (col >= old.unsqueeze(1)) & (col < want.unsqueeze(1))
    tables.copy_(torch.where(added, free[place], torch.where((col >= want.unsqueeze(1)) & (held == 0).unsqueeze(1),
                                                             torch.full_like(tables, scratch), tables)))
    i = torch.arange(st["n_tokens"], device=dev)
    seq = torch.searchsorted(ends, i, right=True)
    real = seq < held.numel()
    s = seq.clamp(max=held.numel() - 1)
    pos = i - (ends - new)[s] + held[s]
    block = tables[s, (pos // bs).clamp(0, width - 1)].long()
    return {"tables": tables, "ctx": ctx.int(), "starts": torch.cat([ends[:1] * 0, ends]).int(),
            "seqs": torch.where(real, seq, -1).int(), "positions": torch.where(real, pos, 0).int(),
            "slots": torch.where(real, block * bs + pos % bs, -1), "cursor": (st["cursor"] + need.sum()).int()}


def _store(st, x, pool, scales):
    c = st["case"]
    rows, flat = st["slots"][:st["tokens"]], pool.view(-1, c["hkv"], c["d"])
    x = x[:st["tokens"]].float()
    if c["int8"]:
        scale = x.abs().amax(dim=-1) / 127.0
        code = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)).clamp(-127, 127)
        flat[rows] = code.to(torch.int8)
        scales.view(-1, c["hkv"])[rows] = scale
    else:
        flat[rows] = x.to(torch.bfloat16)


def _values(st, pool, scales):
    """What the pages stand for."""
    if not st["case"]["int8"]:
        return pool
    return torch.mul(pool, scales.unsqueeze(-1), out=torch.empty_like(pool, dtype=torch.bfloat16))


def _loaded(st, tables, pos, pool, scales):
    """Rows of positions [n, m] in 32 bits: [n, m, Hkv, D]."""
    c = st["case"]
    bs = c["bs"]
    rows = torch.gather(tables.long(), 1, pos // bs) * bs + pos % bs
    x = pool.view(-1, c["hkv"], c["d"])[rows].float()
    return x * scales.view(-1, c["hkv"])[rows].unsqueeze(-1) if c["int8"] else x


def _scores(st, q, k, seen):
    """q [n, m, Hq, D] against k [n, t, Hkv, D], keys not seen [n, 1 or m, t] at -inf: [n, Hkv, G, m, t]."""
    n, m, hq, d = q.shape
    hkv = k.shape[2]
    qg = q.float().view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)).mul_(st["scale"]).view(n, hkv, hq // hkv, m, -1)
    return s.masked_fill_(~seen[:, None, None], float("-inf"))


def _weighted(p, v):
    """p [n, Hkv, G, m, t] times v [n, t, Hkv, D]: [n, m, Hkv, G, D]."""
    n, hkv, g, m, t = p.shape
    o = torch.matmul(p.view(n, hkv, -1, t), v.transpose(1, 2)).view(n, hkv, g, m, -1)
    return o.permute(0, 3, 1, 2, 4)


def _cross_plain(st):
    keys, starts, span, most = st["keys"].long(), st["starts"].long(), st["span"], st["most"]
    dev = keys.device
    slot = torch.arange(span, device=dev).unsqueeze(0)
    pos = torch.minimum(slot, (keys - 1).clamp(min=0).unsqueeze(1))
    k = _loaded(st, st["tables"], pos, st["kp"], st["ks"])
    v = _loaded(st, st["tables"], pos, st["vp"], st["vs"])
    # the packed queries, padded to the longest, and back
    i = torch.arange(most, device=dev).unsqueeze(0)
    row = torch.minimum(starts[:-1].unsqueeze(1) + i, (starts[1:] - 1).clamp(min=0).unsqueeze(1))
    s = _scores(st, st["q"][row], k, (slot < keys.unsqueeze(1)).unsqueeze(1))
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp_(s.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)))
    total = p.sum(dim=-1).permute(0, 3, 1, 2).unsqueeze(-1)
    o = _weighted(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    t = torch.arange(st["q"].shape[0], device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return o[seq, t - starts[seq]].reshape(st["q"].shape).to(torch.bfloat16)


def _shared_plain(st):
    """The prefix's scores of a group at once, each sequence's own behind them."""
    c, q = st["case"], st["q"]
    n, hq, d = q.shape
    hkv, dev = c["hkv"], q.device
    prefix = st["prefix"].long()[st["group"].long()]
    own_len = st["ctx"].long() - prefix
    slot = torch.arange(st["span"], device=dev).unsqueeze(0)
    pos = prefix.unsqueeze(1) + torch.minimum(slot, (own_len - 1).clamp(min=0).unsqueeze(1))
    s = _scores(st, q.unsqueeze(1), _loaded(st, st["tables"], pos, st["kp"], st["ks"]),
                (slot < own_len.unsqueeze(1)).unsqueeze(1))
    top = s.amax(dim=-1)                                                       # [n, Hkv, G, 1]
    p = torch.exp_(s.sub_(top.unsqueeze(-1)))
    o = _weighted(p, _loaded(st, st["tables"], pos, st["vp"], st["vs"]))[:, 0]    # [n, Hkv, G, D]
    top, total = top[..., 0], p.sum(dim=-1)[..., 0]
    out = torch.empty_like(q)
    for g, length in enumerate(st["lengths"]):
        a, b = st["bounds"][g], st["bounds"][g + 1]
        og, tg, mg = o[a:b], total[a:b], top[a:b]
        if length:
            at = torch.arange(length, device=dev).unsqueeze(0)
            k = _loaded(st, st["prefix_tables"][g:g + 1], at, st["kp"], st["ks"])
            v = _loaded(st, st["prefix_tables"][g:g + 1], at, st["vp"], st["vs"])
            s = _scores(st, q[a:b].unsqueeze(0), k, torch.ones(1, 1, length, dtype=torch.bool, device=dev))
            m = s.amax(dim=-1)                                                 # [1, Hkv, G, rows]
            p = torch.exp_(s.sub_(m.unsqueeze(-1)))
            po, pt, m = _weighted(p, v)[0], p.sum(dim=-1)[0].permute(2, 0, 1), m[0].permute(2, 0, 1)
            both = torch.maximum(m, mg)
            x, y = torch.exp(mg - both), torch.exp(m - both)
            og = og * x.unsqueeze(-1) + po * y.unsqueeze(-1)
            tg = tg * x + pt * y
        out[a:b] = (og / tg.unsqueeze(-1)).reshape(b - a, hq, d).to(torch.bfloat16)
    return out


def _run_plain(st):
    op = st["case"]["op"]
    if op == "maps":
        return _maps_plain(st)
    if op == "write":
        _store(st, st["k"], st["kp"], st["ks"])
        _store(st, st["v"], st["vp"], st["vs"])
        return {"k_pool": _values(st, st["kp"], st["ks"]), "v_pool": _values(st, st["vp"], st["vs"])}
    return {"out": _cross_plain(st) if op == "cross" else _shared_plain(st)}


# ----------------------------------------------------------------------------- the framework's calls

def _run_own(st):
    import paged_kv_cache_212_gb300 as P
    op = st["case"]["op"]
    if op == "maps":
        m = P.paged_step_maps(st["held"], st["new"], st["free"], st["tables"], st["case"]["bs"], st["n_blocks"],
                              st["n_tokens"], cursor=st["cursor"], out=st["maps"])
        return {"tables": st["tables"], "ctx": m.ctx_lens, "starts": m.token_starts, "seqs": m.token_seqs,
                "positions": m.positions, "slots": m.slots, "cursor": m.cursor}
    if op == "write":
        P.paged_kv_write_slots(st["k"], st["v"], st["kp"], st["vp"], st["slots"], k_scales=st["ks"], v_scales=st["vs"])
        return {"k_pool": _values(st, st["kp"], st["ks"]), "v_pool": _values(st, st["vp"], st["vs"])}
    if op == "cross":
        return {"out": P.paged_cross_attention(st["q"], st["starts"], st["kp"], st["vp"], st["tables"], st["keys"],
                                               st["scale"], k_scales=st["ks"], v_scales=st["vs"], workspace=st["ws"])}
    return {"out": st["plan"].run(st["q"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- 64 bits

def _exact_attention(q, k, v, scale):
    """q [m, Hq, D] over k, v [t, Hkv, D], all in 64 bits; no key: zeros."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    out, g = torch.empty_like(q), q.shape[1] // k.shape[1]
    for h in range(k.shape[1]):
        x = q[:, h * g:(h + 1) * g].transpose(0, 1)                            # [G, m, D]
        out[:, h * g:(h + 1) * g] = (torch.softmax(x @ k[:, h].T * scale, dim=-1) @ v[:, h]).transpose(0, 1)
    return out


def _exact_maps(case, st):
    held, new, _, _ = _lengths(case)
    bs, free, cursor = case["bs"], st["free"].tolist(), st["cursor"].item()
    tables = st["tables"].cpu()
    seqs, positions, slots, starts = [], [], [], [0]
    for s, (h, m) in enumerate(zip(held, new)):
        row = tables[s].tolist()
        for b in range(-(-h // bs), -(-(h + m) // bs)):
            row[b] = free[cursor]
            cursor += 1
        if h == 0:
            row[-(-m // bs):] = [st["n_blocks"]] * (len(row) - -(-m // bs))
        tables[s] = torch.tensor(row, dtype=torch.int32)
        seqs += [s] * m
        positions += range(h, h + m)
        slots += [row[t // bs] * bs + t % bs for t in range(h, h + m)]
        starts.append(starts[-1] + m)
    pad = case["pad"]

    def ints(x, kind=torch.int32):
        return torch.tensor(x, dtype=kind, device="cuda")

    return {"tables": tables.cuda(), "ctx": ints([h + m for h, m in zip(held, new)]), "starts": ints(starts),
            "seqs": ints(seqs + [-1] * pad), "positions": ints(positions + [0] * pad),
            "slots": ints(slots + [-1] * pad, torch.int64), "cursor": ints([cursor])}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "maps":
        return _exact_maps(case, st)
    held, new, starts, prefix = _lengths(case)
    hq, hkv, d, bs = (case[k] for k in ("hq", "hkv", "d", "bs"))

    def pages(pool, scales):
        x = pool.double().view(-1, hkv, d)
        return x * scales.double().view(-1, hkv, 1) if scales is not None else x

    kp, vp = pages(st["kp"], st["ks"]), pages(st["vp"], st["vs"])
    if case["op"] == "write":
        for flat, x in ((kp, st["k"]), (vp, st["v"])):
            for i, row in enumerate(st["slots"].tolist()):
                if row < 0:
                    continue
                y = x[i].double()
                if case["int8"]:      # the nearest of 255 steps of absmax / 127
                    step = (y.abs().amax(dim=-1, keepdim=True) / 127).clamp(min=1e-300)
                    y = torch.round(y / step) * step
                flat[row] = y
        return {"k_pool": kp.view(st["kp"].shape), "v_pool": vp.view(st["vp"].shape)}
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=kp.device)
    q = st["q"].double()

    def rows(table, first, stop):
        t = torch.arange(first, stop, device=kp.device)
        return table[t // bs].long() * bs + t % bs

    if case["op"] == "cross":
        at = 0
        for s in range(case["n"]):
            r = rows(st["tables"][s], 0, held[s])
            out[at:at + new[s]] = _exact_attention(q[at:at + new[s]], kp[r], vp[r], st["scale"])
            at += new[s]
        return {"out": out}
    for g in range(case["groups"]):
        p = rows(st["prefix_tables"][g], 0, prefix[g])
        for s in range(starts[g], starts[g + 1]):
            r = torch.cat([p, rows(st["tables"][s], prefix[g], prefix[g] + held[s])])
            out[s:s + 1] = _exact_attention(q[s:s + 1], kp[r], vp[r], st["scale"])
    return {"out": out}
