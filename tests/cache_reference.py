"""The 8-bit cache's operators in float64 on the host, one sequence and head at
a time, and the cases that the tests run.  Written from the definitions in
include/spec_verify.h; shares no code with the package."""
import math

import torch

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}  # significand bits after the point, smallest normal exponent


def round8(x, code):
    """float64 values to the nearest code's value, ties to even, within the largest code; NaN for what is not finite."""
    bits, low = BITS[code]
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=low)
    step = torch.exp2(e - bits)
    y = (torch.round(x / step) * step).clamp(-TOP[code], TOP[code])
    return torch.where(torch.isfinite(x), y, torch.nan)


def scale_for(x, code):
    """The smallest power of two s with |x| <= s * top for the finite x, 2^-100 at least."""
    x = x[torch.isfinite(x)]
    amax = float(x.abs().max()) if x.numel() else 0.0
    s = 2.0 ** -100
    while s * TOP[code] < amax:
        s *= 2
    return s


class Pool:
    """A cache on the host: codes as float64 values, scales, tables."""

    def __init__(self, pages, heads, block, dim, code="e4m3", positions=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.code, self.block, self.heads, self.dim = code, block, heads, dim
        x = torch.randn(2, pages, heads, block, dim, generator=g, dtype=torch.float64)
        x *= torch.exp(0.5 * torch.randn(2, pages, heads, 1, 1, generator=g, dtype=torch.float64))
        self.scale = torch.tensor([[[scale_for(x[s, p, h], code) for h in range(heads)] for p in range(pages)]
                                   for s in range(2)], dtype=torch.float64)
        self.codes = round8(x / self.scale[..., None, None], code)
        self.positions = None
        if positions:
            self.positions = torch.randint(0, 4, (pages, heads, block), generator=g).int()
        self.gen = g

    def spread_positions(self, table):
        """Increasing positions with gaps along each sequence and head."""
        for b in range(table.shape[0]):
            pos = torch.randint(1, 4, (self.heads, table.shape[1] * self.block), generator=self.gen).cumsum(1)
            for j in range(table.shape[1]):
                if 0 <= table[b, j] < len(self.positions):
                    self.positions[table[b, j]] = pos[:, j * self.block:(j + 1) * self.block].int()

    def to(self, sv, device="cuda", nhd=False):
        """The package's cache with these contents; nhd: pools laid out [page, token, head, dim]."""
        t = []
        for side in range(2):
            c = self.codes[side].float().to(F8[self.code])
            if nhd:
                c = c.view(torch.uint8).transpose(1, 2).contiguous().view(F8[self.code]).to(device)
                t.append(c.view(torch.uint8).transpose(1, 2).view(F8[self.code]))
            else:
                t.append(c.contiguous().to(device))
        pos = None if self.positions is None else self.positions.to(device)
        return sv.KVCache(t[0], t[1], self.scale[0].float().to(device), self.scale[1].float().to(device), pos)

    def tokens(self, side, table, h, n):
        """Values of the first n tokens of one sequence and head, and which of them are cached."""
        pages = table[torch.arange(n) // self.block].long()
        ok = (pages >= 0) & (pages < self.codes.shape[1])
        pages = pages.clamp(0, self.codes.shape[1] - 1)
        rows = torch.arange(n) % self.block
        return self.codes[side][pages, h, rows] * self.scale[side][pages, h][:, None], ok

    def position(self, table, h, n):
        if self.positions is None:
            return torch.arange(n, dtype=torch.float64)
        pages = table[torch.arange(n) // self.block].long().clamp(0, self.codes.shape[1] - 1)
        return self.positions[pages, h, torch.arange(n) % self.block].double()


def mask(length, new, i, window=0, prefix=0, parent=None):
    """Which of the tokens 0..length-1 query i (of `new`) sees."""
    j = torch.arange(length)
    at = length - new + i
    if parent is None:
        see = j <= at
    else:
        see = j < length - new
        k = i
        while k >= 0:
            see[length - new + k] = True
            up = int(parent[k]) if k > 0 else -1
            k = up if 0 <= up < k else -1
    if window:
        see = see & (j > at - window)
    return see | (j < prefix)


def attend(pool, table, lengths, q, scale, num_new=None, softcap=0.0, slopes=None, window=0, prefix=None,
           parent=None):
    """dict: out, lse, and error bounds' ingredients (float64): `mean` = sum p |v|, `dx` = how far 32-bit scores
    of queries split into two 4-bit significands may be off, `p` = per (b, kv head): [rows of i, g][tokens]."""
    B, n, H, D = q.shape
    G = H // pool.heads
    q = q.double()
    out = torch.zeros(B, n, H, D, dtype=torch.float64)
    mean, dx = torch.zeros_like(out), torch.zeros(B, n, H, dtype=torch.float64)
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64)
    xs = {}
    for b in range(B):
        L = int(lengths[b])
        m = n if num_new is None else int(num_new[b])
        for h in range(pool.heads):
            k, ok = pool.tokens(0, table[b], h, L)
            v, _ = pool.tokens(1, table[b], h, L)
            pos = pool.position(table[b], h, L)
            for i in range(m):
                see = mask(L, m, i, window, int(prefix[b]) if prefix is not None else 0,
                           parent[b] if parent is not None else None) & ok
                if not see.any():
                    continue
                for g in range(G):
                    H1 = h * G + g
                    qq = q[b, i, H1]
                    kk = k[see]
                    x = kk @ qq * scale
                    err = scale * 2.0 ** -17 * (float(qq.abs().max()) * kk.abs().sum(1) + kk.abs() @ qq.abs())
                    if softcap:
                        x = softcap * torch.tanh(x / softcap)
                        err = err + 2.0 ** -20 * softcap
                    if slopes is not None:
                        bias = float(slopes[H1]) * (pos[L - m + i] - pos[see]).abs()
                        x = x - bias
                        err = err + 2.0 ** -22 * (bias + x.abs())
                    z = torch.logsumexp(x, 0)
                    p = torch.exp(x - z)
                    lse[b, i, H1] = z
                    out[b, i, H1] = p @ v[see]
                    mean[b, i, H1] = p @ v[see].abs()
                    # how far lse may be off: the weighted mean of the scores' errors, and 32-bit sums
                    dx[b, i, H1] = float((p * err).nan_to_num().sum()) + 2.0 ** -20 * (1 + float(z.abs().nan_to_num()))
                    xs[b, i, H1] = (see, x, err)
    return dict(out=out, lse=lse, mean=mean, dx=dx, xs=xs)


def weigh(pool, table, lengths, ref, lse, weights):
    """(weights in float64 after the call, bound of their error) for the scores of attend()."""
    w, off = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    for (b, i, H1), (see, x, err) in ref["xs"].items():
        G = lse.shape[2] // pool.heads
        h = H1 // G
        j = see.nonzero()[:, 0]
        p = torch.exp(x - float(lse[b, i, H1]))
        page, row = table[b][j // pool.block].long(), j % pool.block
        w[page, h, row] += p
        off[page, h, row] += p * (1.5 * err + 2.0 ** -20 * (1 + x.abs()))
    return w, off + 2.0 ** -21 * w.abs()


def append(pool, table, lengths, k, v, num_new=None, positions=None):
    """pool after the call."""
    B, n = k.shape[:2]
    for b in range(B):
        L = int(lengths[b])
        m = n if num_new is None else int(num_new[b])
        for blk in range(L // pool.block, -(-(L + m) // pool.block)):
            page = int(table[b, blk])
            lo, hi = max(L, blk * pool.block), min(L + m, (blk + 1) * pool.block)
            old = lo - blk * pool.block
            if lo >= hi:
                continue
            for h in range(pool.heads):
                for side, x in enumerate((k, v)):
                    new = x[b, lo - L:hi - L, h].double()
                    s = scale_for(new, pool.code)
                    if old:
                        had = float(pool.scale[side, page, h])
                        s = max(s, had)
                        pool.codes[side, page, h, :old] = round8(pool.codes[side, page, h, :old] * (had / s), pool.code)
                    pool.scale[side, page, h] = s
                    pool.codes[side, page, h, old:old + hi - lo] = round8(new / s, pool.code)
                if pool.positions is not None:
                    pos = torch.arange(lo, hi).int() if positions is None else positions[b, lo - L:hi - L]
                    pool.positions[page, h, old:old + hi - lo] = pos
    return pool


def evict(pool, table, lengths, weights, keep, recent, out_table):
    """(lengths, index) after the call; pool and weights (both changed)."""
    B = table.shape[0]
    kept = torch.tensor([min(int(x), keep) for x in lengths], dtype=torch.int32)
    index = torch.full((B, pool.heads, keep), -1, dtype=torch.int32)
    codes, scale, was = pool.codes.clone(), pool.scale.clone(), weights.clone()
    pos = None if pool.positions is None else pool.positions.clone()
    for b in range(B):
        L = int(lengths[b])
        for h in range(pool.heads):
            def at(j):
                return int(table[b, j // pool.block]), h, j % pool.block
            if L <= keep:
                take = list(range(L))
            else:
                def rank(j):
                    w = float(was[at(j)])
                    return (-w if w == w else math.inf, w != w, j)
                take = sorted(sorted(range(L - recent), key=rank)[:keep - recent]) + list(range(L - recent, L))
            index[b, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
            for blk in range(-(-len(take) // pool.block)):
                part = take[blk * pool.block:(blk + 1) * pool.block]
                page = int(out_table[b, blk])
                for side in range(2):
                    had = [float(scale[side][at(j)[:2]]) for j in part]
                    s = max(had)
                    pool.scale[side, page, h] = s
                    for t, j in enumerate(part):
                        pool.codes[side, page, h, t] = round8(codes[side][at(j)] * (had[t] / s), pool.code)
                for t, j in enumerate(part):
                    weights[page, h, t] = was[at(j)]
                    if pos is not None:
                        pool.positions[page, h, t] = pos[at(j)]
    return kept, index
