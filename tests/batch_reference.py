"""Pools, 64-bit references and error bounds of the calls for ragged batches.

A pool holds NaN (int8: code 127 under a NaN scale) in every row that no query sees,
and table entries of blocks without such a row hold an id outside the pool."""
import torch

import window_reference as R

GARBAGE_ID = -12345


class Paged:
    """Pools of `n_blocks` shuffled blocks, handed out in order by add()."""

    def __init__(self, seed, n_blocks, hkv, d, bs, int8):
        self.gen = torch.Generator().manual_seed(seed)
        self.hkv, self.d, self.bs, self.int8, self.n_blocks = hkv, d, bs, int8, n_blocks
        self.perm, self.at = torch.randperm(n_blocks, generator=self.gen).tolist(), 0
        shape = (n_blocks + 1, bs, hkv, d)
        if int8:
            self.pools = [torch.full(shape, 127, dtype=torch.int8) for _ in range(2)]
            self.scales = [torch.full(shape[:3], float("nan")) for _ in range(2)]
        else:
            self.pools = [torch.full(shape, float("nan"), dtype=torch.bfloat16) for _ in range(2)]
            self.scales = [None, None]

    def add(self, first, stop, width):
        """Tokens first .. stop - 1 of a sequence: its table row, and K and V [stop - first, Hkv, D] in 64 bits."""
        row = torch.full((width,), GARBAGE_ID, dtype=torch.int32)
        for b in range(first // self.bs, -(-stop // self.bs)):
            row[b] = self.perm[self.at]
            self.at += 1
        t = torch.arange(first, stop)
        rows = row[t // self.bs].long() * self.bs + t % self.bs
        pair = []
        for which in range(2):
            if self.int8:
                code = torch.randint(-127, 128, (len(t), self.hkv, self.d), generator=self.gen, dtype=torch.int8)
                code[..., 3] = 127                # a quantised row's largest code
                # scales spread over three powers of ten, some rows of zeros
                sc = 10.0 ** (torch.rand((len(t), self.hkv), generator=self.gen) * 3 - 4.5)
                sc[torch.rand((len(t), self.hkv), generator=self.gen) < 0.03] = 0
                self.pools[which].view(-1, self.hkv, self.d)[rows] = code
                self.scales[which].view(-1, self.hkv)[rows] = sc
                pair.append(code.double() * sc.double()[..., None])
            else:
                val = torch.randn((len(t), self.hkv, self.d), generator=self.gen).to(torch.bfloat16)
                self.pools[which].view(-1, self.hkv, self.d)[rows] = val
                pair.append(val.double())
        return row, pair

    def cuda(self):
        return [None if t is None else t.cuda() for t in self.pools + self.scales]


def check_rows(out, lse, q, k, v, scale, int8, most=0.0):
    """out [m, Hq, D] and lse [m, Hq] of queries q [m, Hq, D] that all see k, v [n, Hkv, D] (64 bits).

    The error: roundings of a prefill (probabilities to bf16 once) or, for a sequence's own
    tokens, those of a decode; keys may be in up to 192 pieces, whose joins round a sum 4
    times each.  int8 pages that many rows read: probabilities and values are rounded to fp16
    (2^-11, less than U16 together), values to 2^-25 of a power of two at most twice the largest
    scale at least, which `most` is (0: scales within 2^13 of one another, whose values are all
    in fp16's normal range), and probabilities to 2^-32 of one at least, of n keys."""
    m, hq, d = out.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    out, lse, q = out.cpu().double(), lse.cpu().double(), q.cpu().double()
    if n == 0:
        assert not out.any() and (lse == -torch.inf).all()
        return
    seen = torch.ones((m, n), dtype=torch.bool)
    for h in range(hkv):
        o, ls, absum, size, top = R.attend(q[:, h * g:(h + 1) * g], k[:, h], v[:, h], seen, scale)
        tol = R.prefill_tolerance(o, absum, size, d, n) + absum * (192 * 4 * R.U32)
        if int8:
            tol = tol + R.decode_tolerance(o, absum, size, d, n, top) + 2.0 ** -24 * most
        got = out[:, h * g:(h + 1) * g]
        assert torch.isfinite(got).all(), h
        over = (got - o).abs() - tol
        assert (over <= 0).all(), (h, float(over.max()))
        over = (lse[:, h * g:(h + 1) * g] - ls).abs() - R.lse_tolerance(ls, size, d, n, int8) - 192 * 4 * R.U32
        assert (over <= 0).all(), (h, float(over.max()))


def maps(lens, new, free, cursor, tables, bs, n_blocks, n_tokens):
    """paged_step_maps in plain Python; tables (a list of lists) is written.  Returns
    ctx, starts, seqs, positions, slots, cursor and the status bits."""
    width = len(tables[0]) if tables else 0
    top = 2 ** 31 - 1
    status, ctx, starts, seqs, positions, slots, place = 0, [], [0], [], [], [], cursor
    total = 0
    for s, (h, n) in enumerate(zip(lens, new)):
        if h < 0 or n < 0 or h + n > width * bs:
            status |= 4
            ctx.append(0)
            starts.append(min(total, top))
            continue
        row, held, want = tables[s], -(-h // bs), -(-(h + n) // bs)
        usable = {}
        if n and h % bs:
            usable[held - 1] = 0 <= row[held - 1] <= n_blocks
            if not usable[held - 1] and total < n_tokens:
                status |= 1
        for b in range(held, want):
            ok = 0 <= place < len(free) and cursor >= 0
            if not ok:
                status |= 32
            elif not 0 <= free[place] < n_blocks:
                status |= 1
                ok = False
            row[b] = free[place] if ok else n_blocks
            usable[b] = ok
            place += 1
        if h == 0:
            row[want:] = [n_blocks] * (width - want)
        for t in range(h, h + n):
            if total + t - h >= n_tokens:
                break
            seqs.append(s)
            positions.append(t)
            slots.append(row[t // bs] * bs + t % bs if usable[t // bs] else -1)
        total += n
        ctx.append(h + n)
        starts.append(min(total, top))
    if total > n_tokens:
        status |= 2
    pad = n_tokens - len(seqs)
    return ctx, starts, seqs + [-1] * pad, positions + [0] * pad, slots + [-1] * pad, min(place, top), status
