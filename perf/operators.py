"""The operators of the 8-bit key/value cache, as cases that can be timed and compared.

A target model that scores gamma + 1 drafted tokens per round reads its keys and
values from a paged cache held in 8 bits, with one scale for each block of tokens
and head.  Four operators work on that cache:

  append  writes new tokens (8-bit codes and the block's scale)
  attend  attention of the newest tokens over the cache (capped scores, a bias
          by distance, window, prefix and candidate-tree masks)
  weigh   adds the attention weight that each cached token received
  evict   keeps the tokens with the most weight and the most recent ones

Every case is a dict of plain values.  `run` computes a pass in plain torch
operations, or, where `own` is true, with the package's calls.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BASE = dict(kind="attend", batch=1, new=1, ragged=False, heads=8, kv_heads=2, dim=64, block=16, length=64,
            code="e4m3", softcap=0.0, slopes=False, window=0, prefix=0, tree=False, keep=0, recent=0)


def listed():
    def case(name, **kw):
        return dict(BASE, name=name, **kw)

    return [
        # a first step after a short prompt: one sequence, one token, latency alone
        case("attend first token", length=37),
        # the benchmark's batch: 256 sequences, 4 drafted tokens and the last emitted one
        case("attend round of 256", batch=256, new=5, heads=32, kv_heads=8, dim=128, block=64, length=2048),
        # one token for each of 64 sequences, every head with its own keys, a window and four kept first tokens
        case("attend window", batch=64, new=1, heads=16, kv_heads=16, dim=128, block=16, length=3001, window=1024,
             prefix=4),
        # few sequences and long documents: the work has to be split along the cache
        case("attend long", batch=4, new=5, heads=64, kv_heads=8, dim=128, block=128, length=100001, slopes=True),
        # a tree of 64 candidates in one forward, scores capped by a tanh
        case("attend tree", batch=16, new=64, ragged=True, heads=32, kv_heads=8, dim=128, block=32, length=3001,
             softcap=30.0, tree=True),
        # a chunk of a prompt with a prefix that every token sees, codes with the wider exponent
        case("attend prompt", batch=2, new=1000, heads=16, kv_heads=4, dim=64, block=64, length=8190, prefix=2500,
             code="e5m2"),
        # weights of a short sequence, and of a serving batch
        case("weigh short", kind="weigh", length=300),
        case("weigh round", kind="weigh", batch=32, new=5, heads=32, kv_heads=8, dim=128, block=64, length=8192),
        # the tokens of one round, and of a prompt
        case("append round", kind="append", batch=256, new=5, ragged=True, kv_heads=8, dim=128, block=64, length=150),
        case("append prompt", kind="append", batch=8, new=2047, kv_heads=8, dim=128, block=64, length=30),
        # a short sequence, and a batch of long ones cut to a quarter
        case("evict short", kind="evict", batch=2, length=700, keep=256, recent=32),
        case("evict batch", kind="evict", batch=16, kv_heads=8, dim=128, block=64, length=16384, keep=4096,
             recent=256),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "weigh", "append", "evict"])
    dim, block = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    c = dict(BASE, kind=kind, dim=dim, block=block, kv_heads=kv_heads, heads=kv_heads * group,
             code=rng.choice(["e4m3", "e4m3", "e5m2"]), batch=_log(rng, 1, 64), ragged=rng.random() < 0.5)
    if kind in ("attend", "weigh"):
        c["tree"] = rng.random() < 0.25
        c["new"] = _log(rng, 1, 64) if c["tree"] else rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 500)])
        most = min(60000, int(2e8 / (c["batch"] * kv_heads * dim)), int(6e7 / (c["batch"] * c["heads"] * c["new"])))
        c["length"] = _log(rng, c["new"], max(c["new"] + 1, most))
        c["softcap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        c["slopes"] = rng.random() < 0.3
        if not c["tree"] and rng.random() < 0.4:
            c["window"] = _log(rng, 1, c["length"])
        if rng.random() < 0.3:
            c["prefix"] = _log(rng, 1, c["length"])
    elif kind == "append":
        c["new"] = rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 2000)])
        c["batch"] = min(c["batch"], max(1, int(2e7 / (c["new"] * kv_heads * dim))))
        c["length"] = rng.randrange(0, 300)
    else:
        c["length"] = _log(rng, 2, min(40000, int(2e8 / (c["batch"] * kv_heads * dim))))
        c["keep"] = _log(rng, 1, c["length"])
        c["recent"] = rng.randrange(0, c["keep"] + 1)
        c["slopes"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# sizes that follow from the case alone
# ---------------------------------------------------------------------------
def _lengths(c):
    """Tokens of each sequence: the longest first, the others down to half of it.
    For append: tokens before the call; else with the new ones among them."""
    low = 0 if c["kind"] == "append" else c["new"]
    return [max(low, c["length"] - (b * 977) % (c["length"] // 2 + 1)) for b in range(c["batch"])]


def _news(c):
    """New tokens of each sequence: `new`, or anything from one to that."""
    return [c["new"] - (b * 7) % c["new"] if c["ragged"] else c["new"] for b in range(c["batch"])]


def _pages_per_sequence(c):
    most = c["length"] + (c["new"] if c["kind"] == "append" else 0)
    return max(1, -(-most // c["block"]))


def _seen(c):
    """Per sequence: (cached tokens that some query reads, (query, token) pairs)."""
    got = []
    for length, new in zip(_lengths(c), _news(c)):
        first = length - new
        p = min(c["prefix"], length)
        w = c["window"] or length + 1
        low = max(0, first - w + 1)
        pairs = 0
        for i in range(new):
            q = first + i
            a, e = max(0, q - w + 1), q + 1
            pairs += (e - a) + (p if p <= a else max(0, a) + max(0, p - e))
        got.append((length - max(0, low - p), pairs))
    return got


def work(c):
    B, H, KH, D, P, n = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["block"], c["new"]
    if c["kind"] in ("attend", "weigh"):
        seen = _seen(c)
        tokens, pairs = sum(s[0] for s in seen), sum(s[1] for s in seen)
        sides = 2 if c["kind"] == "attend" else 1
        scales = sides * 4 * KH * tokens / P
        rows = sum(_news(c)) * H
        b = sides * tokens * KH * D + scales + rows * D * 2 + rows * 4 + 4 * tokens / P
        b += (rows * D * 2) if c["kind"] == "attend" else 8 * tokens * KH
        b += 4 * tokens * KH if c["slopes"] else 0
        return {"bytes": b, "flops": 2 * sides * pairs * H * D}
    if c["kind"] == "append":
        tokens = sum(_news(c)) * KH
        return {"bytes": 2 * tokens * D * 3 + 2 * 4 * KH * sum(_news(c)) / P, "flops": 4 * tokens * D}
    tokens = sum(_lengths(c)) * KH
    kept = sum(min(c["keep"], x) for x in _lengths(c)) * KH
    b = 4 * tokens + kept * (4 * D + 4 + 4) + 4 * 4 * kept / P + (8 * kept if c["slopes"] else 0)
    return {"bytes": b, "flops": tokens + 2 * kept * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pow2_scale(amax, code):
    """The smallest power of two s with amax <= s * (largest code), 2^-100 at least."""
    top = torch.finfo(F8[code]).max  # 1.75 * 2^8 for both forms of the significand: 448 and 57344
    m, e = torch.frexp(amax)
    mt, et = math.frexp(top)
    e = e - et + (m > mt).to(e.dtype)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100))


def _filled(shape, code, gen, spread):
    """A pool of blocks as a run of appends leaves it: codes and scales."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= spread
    s = _pow2_scale(x.abs().amax(dim=(2, 3)), code)
    return (x / s[:, :, None, None]).to(F8[code]), s


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    B, H, KH, D, P, n = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["block"], c["new"]
    per = _pages_per_sequence(c)
    spare = B * -(-c["keep"] // P) if c["kind"] == "evict" else 0
    pages = B * per + spare
    # keys have a few strong channels, values are even; blocks differ in size
    strong = 1 + 3 * (torch.rand(D, generator=gen, device="cuda") < 0.06).float()
    block = torch.exp(0.3 * torch.randn(pages, KH, 1, 1, generator=gen, device="cuda"))
    s = dict(case=c)
    s["k"], s["k_scale"] = _filled((pages, KH, P, D), c["code"], gen, strong * block)
    s["v"], s["v_scale"] = _filled((pages, KH, P, D), c["code"], gen, block)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    s["block_table"] = order[: B * per].reshape(B, per).contiguous()
    s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    s["num_new"] = torch.tensor(_news(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
    s["positions"] = None
    if c["slopes"]:  # each head kept its own tokens of a longer text: positions with gaps
        gaps = torch.randint(1, 4, (B, KH, per * P), generator=gen, device="cuda")
        pos = gaps.cumsum(2).to(torch.int32)
        s["positions"] = torch.zeros(pages, KH, P, dtype=torch.int32, device="cuda")
        s["positions"][s["block_table"].reshape(-1).long()] = (
            pos.reshape(B, KH, per, P).permute(0, 2, 1, 3).reshape(B * per, KH, P))
    if c["kind"] in ("attend", "weigh"):
        s["q"] = torch.randn(B, n, H, D, generator=gen, device="cuda").to(torch.bfloat16)
        s["scale"] = 1 / math.sqrt(D)
        s["slopes"] = None
        if c["slopes"]:
            s["slopes"] = torch.exp2(-8 * torch.arange(1, H + 1, device="cuda").float() / H)
        s["prefix"] = None
        if c["prefix"]:
            s["prefix"] = torch.full((B,), c["prefix"], dtype=torch.int32, device="cuda")
        s["parent"] = None
        if c["tree"]:
            u = torch.rand(B, n, generator=gen, device="cuda")
            s["parent"] = (u * torch.arange(n, device="cuda")).to(torch.int32)
    if c["kind"] == "weigh":
        s["lse"] = _attend(s)[1]
        s["weights"] = torch.rand(pages, KH, P, generator=gen, device="cuda")
    if c["kind"] == "append":
        # what a projection hands over: keys and values side by side in one tensor
        kv = torch.randn(B, n, 2, KH, D, generator=gen, device="cuda")
        kv[:, :, 0] *= strong
        kv = kv.to(torch.bfloat16)
        s["new_k"], s["new_v"] = kv[:, :, 0], kv[:, :, 1]
    if c["kind"] == "evict":
        # few tokens hold most of the weight; many of the others have none at all
        w = torch.randn(pages, KH, P, generator=gen, device="cuda").mul_(2).exp_()
        s["weights"] = w * (torch.rand(pages, KH, P, generator=gen, device="cuda") < 0.8)
        s["out_table"] = order[B * per:].reshape(B, -(-c["keep"] // P)).contiguous()
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _tokens(pool, table):
    """[pages, heads, block, ...] and [batch, pages] -> [batch, heads, tokens, ...]"""
    x = pool[table.long()]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], x.shape[2] * x.shape[3], *x.shape[4:])


def _values(codes, scale, table):
    x = _tokens(codes.view(torch.uint8), table).view(codes.dtype).float()
    return x * scale[table.long()].transpose(1, 2).repeat_interleave(codes.shape[2], dim=2)[..., None]


def _scores(s):
    """Scores [batch, kv heads, new, group, tokens] in float32, -inf where a query does not see a token."""
    c = s["case"]
    q, table = s["q"].float(), s["block_table"]
    B, n, H, D = q.shape
    KH = s["k"].shape[1]
    L = table.shape[1] * c["block"]
    dev = q.device
    q = q.reshape(B, n, KH, H // KH, D).permute(0, 2, 1, 3, 4)
    x = q.reshape(B, KH, -1, D) @ _values(s["k"], s["k_scale"], table).transpose(2, 3)
    x = x.reshape(B, KH, n, H // KH, L) * s["scale"]
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    length = s["lengths"].long()[:, None, None]
    new = (s["num_new"].long() if s["num_new"] is not None else torch.full((B,), n, device=dev))[:, None, None]
    i, j = torch.arange(n, device=dev)[None, :, None], torch.arange(L, device=dev)[None, None, :]
    at = length - new + i
    if s["slopes"] is not None:
        pos = _tokens(s["positions"], table)
        pq = pos.gather(2, at[:, None, :, 0].clamp(0, L - 1).expand(B, KH, n))
        far = (pq[..., None] - pos[:, :, None, :]).abs().float()
        x = x - s["slopes"].reshape(KH, 1, H // KH, 1) * far[:, :, :, None, :]
    if s["parent"] is None:
        see = j <= at
    else:
        eye = torch.eye(n, device=dev)
        up = torch.zeros(B, n, n, device=dev).scatter_(2, s["parent"].long()[..., None], 1.0).tril(-1)
        kin = torch.linalg.solve_triangular(eye - up, eye.expand(B, n, n), upper=False, unitriangular=True) > 0.5
        node = (j - (length - new)).expand(B, n, L)
        see = (node < 0) | (kin.gather(2, node.clamp(0, n - 1)) & (node < n))
    if c["window"]:
        see = see & (j > at - c["window"])
    if s["prefix"] is not None:
        see = see | (j < s["prefix"].long()[:, None, None])
    see = see & (j < length) & (i < new)
    return x.masked_fill(~see[:, None, :, None, :], -math.inf)


def _attend(s):
    c = s["case"]
    x = _scores(s)
    B, KH, n, G, L = x.shape
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = torch.where(total > 0, m + torch.log(total), torch.full_like(m, -math.inf))
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    j = torch.arange(L, device=x.device)
    v = _values(s["v"], s["v_scale"], s["block_table"])
    v = v.masked_fill((j >= s["lengths"][:, None])[:, None, :, None], 0.0)
    o = p.reshape(B, KH, n * G, L) @ v
    out = o.reshape(B, KH, n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, KH * G, -1)
    return out.to(torch.bfloat16), lse[..., 0].permute(0, 2, 1, 3).reshape(B, n, KH * G)


def _weigh(s):
    c = s["case"]
    x = _scores(s)
    B, KH, n, G, L = x.shape
    lse = s["lse"].reshape(B, n, KH, G).permute(0, 2, 1, 3)[..., None]
    p = torch.where(x == -math.inf, torch.zeros_like(x), torch.exp(x - lse))
    add = p.sum(dim=(2, 3)).reshape(B, KH, -1, c["block"]).transpose(1, 2)
    s["weights"][s["block_table"].reshape(-1).long()] += add.reshape(-1, KH, c["block"])
    return s["weights"]


def _append_one(s, codes, scale, x):
    c = s["case"]
    P = c["block"]
    B, n, KH, D = x.shape
    dev = x.device
    length = s["lengths"].long()
    new = s["num_new"].long() if s["num_new"] is not None else torch.full((B,), n, device=dev)
    first = length // P
    blocks = first[:, None] + torch.arange((n + P - 2) // P + 1, device=dev)  # [B, blocks that may be touched]
    touched = (blocks * P < (length + new)[:, None]) & (new > 0)[:, None]
    b, t = touched.nonzero(as_tuple=True)
    blk = blocks[b, t]
    page = s["block_table"][b, blk].long()
    j = blk[:, None] * P + torch.arange(P, device=dev)
    old = j < length[b][:, None]
    put = ~old & (j < (length + new)[b][:, None])
    rows = x.float()[b[:, None], (j - length[b][:, None]).clamp(0, n - 1)].transpose(1, 2)  # [M, KH, P, D]
    amax = (rows.abs() * put[:, None, :, None]).amax(dim=(2, 3))
    had = torch.where(old.any(1)[:, None], scale[page], torch.zeros_like(amax))
    now = torch.maximum(_pow2_scale(amax, c["code"]), had)
    there = codes.view(torch.uint8)[page].view(codes.dtype)
    again = (there.float() * (had / now)[..., None, None]).to(codes.dtype).view(torch.uint8)
    fresh = (rows / now[..., None, None]).to(codes.dtype).view(torch.uint8)
    both = torch.where(put[:, None, :, None], fresh, torch.where(old[:, None, :, None], again, there.view(torch.uint8)))
    codes.view(torch.uint8)[page] = both
    scale[page] = now


def _append(s):
    _append_one(s, s["k"], s["k_scale"], s["new_k"])
    _append_one(s, s["v"], s["v_scale"], s["new_v"])
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _evict(s):
    c = s["case"]
    P, keep, recent = c["block"], c["keep"], c["recent"]
    w = _tokens(s["weights"], s["block_table"])
    B, KH, L = w.shape
    dev = w.device
    j = torch.arange(L, device=dev)
    length = s["lengths"].long()[:, None, None]
    rank = torch.where(j >= length, -2.0, torch.where(j >= length - recent, math.inf, w))
    order = torch.sort(rank, dim=2, descending=True, stable=True)[1][:, :, :keep]
    kept = torch.minimum(length, torch.tensor(keep, device=dev))
    order = torch.where(torch.arange(order.shape[2], device=dev) < kept, order, L)
    index = torch.sort(order, dim=2)[0]  # [B, KH, keep] cached index, L where there is none
    index = torch.nn.functional.pad(index, (0, -(-keep // P) * P - index.shape[2]), value=L)
    none = index >= L
    at = index.clamp(max=L - 1)
    page = s["block_table"].long().gather(1, (at // P).reshape(B, -1)).reshape(at.shape)
    h = torch.arange(KH, device=dev)[None, :, None]
    row = at % P
    dst = s["out_table"].long()
    nb = dst.shape[1]
    has = ~none.reshape(B, KH, nb, P)

    def put(pool, x):  # x: [B, KH, tokens, ...] into the pages of `out_table`, where there is a token
        x = x.reshape(B, KH, nb, P, *x.shape[3:]).transpose(1, 2)
        m = has.transpose(1, 2).reshape(has.shape[0], nb, KH, P, *([1] * (x.dim() - 4)))
        pool[dst] = torch.where(m, x, pool[dst])

    for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        had = torch.where(none, torch.zeros_like(scale[page, h]), scale[page, h])
        now = had.reshape(B, KH, nb, P).amax(3)
        x = codes.view(torch.uint8)[page, h, row].view(codes.dtype).float()
        x = x * (had / now.clamp(min=2.0 ** -126).repeat_interleave(P, dim=2))[..., None]
        put(codes.view(torch.uint8), x.to(codes.dtype).view(torch.uint8))
        scale[dst] = torch.where(has.any(3).transpose(1, 2), now.transpose(1, 2), scale[dst])
    put(s["weights"], s["weights"][page, h, row])
    if s["positions"] is not None:
        put(s["positions"], s["positions"][page, h, row])
    index = torch.where(none, -1, index)[:, :, :keep].to(torch.int32)
    return s["k"], s["v"], s["k_scale"], s["v_scale"], s["weights"], kept[:, 0, 0].to(torch.int32), index, s["positions"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verification_45_gb300 as sv

        cache = sv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["positions"])
        if c["kind"] == "append":
            sv.cache_append(cache, s["block_table"], s["lengths"], s["new_k"], s["new_v"], num_new=s["num_new"])
            return s["k"], s["v"], s["k_scale"], s["v_scale"]
        if c["kind"] == "evict":
            kept, index = sv.cache_evict(cache, s["block_table"], s["lengths"], s["weights"], c["keep"], c["recent"],
                                         s["out_table"])
            return s["k"], s["v"], s["k_scale"], s["v_scale"], s["weights"], kept, index, s["positions"]
        form = dict(num_new=s["num_new"], scale=s["scale"], softcap=c["softcap"], slopes=s["slopes"],
                    window=c["window"], prefix=s["prefix"], parent=s["parent"])
        if c["kind"] == "attend":
            return sv.cache_attend(s["q"], cache, s["block_table"], s["lengths"], **form)
        return sv.cache_weigh(s["q"], cache, s["block_table"], s["lengths"], s["lse"], s["weights"], **form)
    return {"attend": _attend, "weigh": _weigh, "append": _append, "evict": _evict}[c["kind"]](s)


# ---------------------------------------------------------------------------
# the definition, in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------
def _round8(x, code):
    """x (float64) to the nearest value of the 8-bit form, ties to even; the largest one bounds it."""
    bits, low, top = (3, -6, 448.0) if code == "e4m3" else (2, -14, 57344.0)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=low)
    step = torch.exp2(e - bits)
    return (torch.round(x / step) * step).clamp(-top, top)


def _fit(amax, code):
    top = 448.0 if code == "e4m3" else 57344.0
    s = 2.0 ** -100
    if amax > 0:
        s = max(s, 2.0 ** (math.floor(math.log2(amax)) - int(math.log2(top)) - 1))
        while s * top < amax:
            s *= 2
    return s


def _seq(pool, table, h, n, scale=None):
    """Tokens 0..n-1 of one sequence and head, in 64 bits."""
    x = pool[table.long(), h].double()
    if scale is not None:
        x = x * scale[table.long(), h].double()[:, None, None]
    return x.reshape(-1, *x.shape[2:])[:n]


def exact(c, seed):
    s = prepare(c, seed)
    B, KH, D, P = c["batch"], c["kv_heads"], c["dim"], c["block"]
    lengths, news = _lengths(c), _news(c)
    if c["kind"] in ("attend", "weigh"):
        G, n = c["heads"] // KH, c["new"]
        out = torch.zeros(B, n, KH * G, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, n, KH * G), -math.inf, dtype=torch.float64, device="cuda")
        weights = s["weights"].double() if c["kind"] == "weigh" else None
        for b in range(B):
            L, nn = lengths[b], news[b]
            base = L - nn
            j = torch.arange(L, device="cuda")
            i = torch.arange(nn, device="cuda")[:, None]
            see = j[None] <= base + i
            if c["tree"]:
                up = s["parent"][b].tolist()
                see = (j[None] < base).expand(nn, L).clone()
                for k in range(nn):
                    at = k
                    line = [k]
                    while at > 0:
                        at = up[at]
                        line.append(at)
                    see[k, [base + x for x in line]] = True
            if c["window"]:
                see = see & (base + i - j[None] < c["window"])
            if c["prefix"]:
                see = see | (j[None] < c["prefix"])
            table = s["block_table"][b]
            for h in range(KH):
                x = torch.einsum("igd,jd->gij", s["q"][b, :nn, h * G:(h + 1) * G].double(),
                                 _seq(s["k"], table, h, L, s["k_scale"])) * s["scale"]
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                if c["slopes"]:
                    pos = _seq(s["positions"], table, h, L)
                    x = x - (s["slopes"][h * G:(h + 1) * G].double()[:, None, None]
                             * (pos[base:, None] - pos[None]).abs())
                x = torch.where(see[None], x, -math.inf)
                if c["kind"] == "attend":
                    z = torch.logsumexp(x, -1)
                    lse[b, :nn, h * G:(h + 1) * G] = z.t()
                    p = torch.nan_to_num(torch.exp(x - z[..., None]), nan=0.0)
                    out[b, :nn, h * G:(h + 1) * G] = (p @ _seq(s["v"], table, h, L, s["v_scale"])).transpose(0, 1)
                else:
                    z = s["lse"][b, :nn, h * G:(h + 1) * G].double().t()
                    p = torch.where(see[None], torch.exp(x - z[..., None]), 0.0).sum((0, 1))
                    weights[table[j // P].long(), h, j % P] += p
        return (out, lse) if c["kind"] == "attend" else weights
    k, v, ks, vs = (s[x].double() for x in ("k", "v", "k_scale", "v_scale"))
    if c["kind"] == "append":
        if B * KH * (c["new"] // P + 2) > 20000:
            return None
        for b in range(B):
            L, nn = lengths[b], news[b]
            for blk in range(L // P, (L + nn - 1) // P + 1):
                page = int(s["block_table"][b, blk])
                lo, hi = max(blk * P, L), min(blk * P + P, L + nn)
                for codes, scale, x in ((k, ks, s["new_k"]), (v, vs, s["new_v"])):
                    x = x[b, lo - L:hi - L].double()  # [tokens, KH, D]
                    most = x.abs().amax(dim=(0, 2)).tolist()
                    now = torch.tensor([_fit(a, c["code"]) for a in most], dtype=torch.float64, device="cuda")
                    if lo > blk * P:
                        had = scale[page]
                        now = torch.maximum(now, had)
                        part = codes[page, :, :lo - blk * P]
                        codes[page, :, :lo - blk * P] = _round8(part * (had / now)[:, None, None], c["code"])
                    codes[page, :, lo - blk * P:hi - blk * P] = _round8(x.transpose(0, 1) / now[:, None, None], c["code"])
                    scale[page] = now
        return k, v, ks, vs
    keep, recent = c["keep"], c["recent"]
    index = torch.full((B, KH, keep), -1, dtype=torch.int32, device="cuda")
    weights, pos = s["weights"].double(), s["positions"]
    for b in range(B):
        L = lengths[b]
        m = min(L, keep)
        to = s["out_table"][b].long()
        for h in range(KH):
            w = _seq(s["weights"], s["block_table"][b], h, L)
            take = torch.arange(L, device="cuda")
            if L > keep:
                old = w[:L - recent].cpu().numpy()
                best = torch.from_numpy((-old).argsort(kind="stable")[:keep - recent].copy()).to("cuda")
                take = torch.cat([best, take[L - recent:]]).sort()[0]
            index[b, h, :m] = take.to(torch.int32)
            page = s["block_table"][b, take // P].long()
            t = torch.arange(m, device="cuda")
            dst = to[t // P]
            for codes, scale in ((k, ks), (v, vs)):
                had = scale[page, h]
                now = torch.zeros(len(to), dtype=torch.float64, device="cuda").scatter_reduce(0, t // P, had, "amax")
                x = codes[page, h, take % P] * (had / now[t // P])[:, None]
                codes[dst, h, t % P] = _round8(x, c["code"])
                used = -(-m // P)
                scale[to[:used], h] = now[:used]
            weights[dst, h, t % P] = weights[page, h, take % P]
            if pos is not None:
                pos[dst, h, t % P] = pos[page, h, take % P]
    kept = torch.tensor([min(x, keep) for x in lengths], dtype=torch.int32, device="cuda")
    return k, v, ks, vs, weights, kept, index, pos
