"""The operators around a target's 8-bit products, as cases that can be timed and compared.

Between the attention over the cache and the logits that are verified stand a
target's projections.  Their operands are held in 8 bits: a row (an activation)
has a power-of-two scale for each 128 of its elements, a weight one for each
128 x 128 block.  Four operators work on that form:

  norm      adds the residual, normalises by the root mean square, and quantises
  gate      act(gate) * up of a feed-forward layer, and quantises
  quantise  quantises what is there: rows, or a weight
  product   rows times a weight's rows, in bf16 or fp32: projections and logits

Every case is a dict of plain values.  `run` computes a pass in plain torch
operations, or, where `own` is true, with the package's calls.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128
EPS = 1e-6
BASE = dict(kind="product", rows=1, width=1024, out=0, dtype="bf16", code="e4m3", weight_code="e4m3", residual=True,
            stream="bf16", act="silu", tile=1)


def listed():
    def case(name, **kw):
        return dict(BASE, name=name, **kw)

    return [
        # the projection after the attention of 32 heads of 128, for one sequence and one token: latency
        case("product one token", rows=1, width=4096, out=4096),
        # the logits of a round for one sequence (4 drafts and the last token), in fp32: the weight is read once
        case("product logits of 5", rows=5, width=2048, out=32000, dtype="fp32"),
        # a projection to the second layer of a feed-forward for 32 sequences of 5 tokens
        case("product round of 32", rows=160, width=8192, out=8192),
        # the benchmark's logits: 256 sequences, 4 drafted tokens and the last one, 128,256 words
        case("product logits of 1280", rows=1280, width=4096, out=128256),
        # q, k and v (32 + 8 + 8 heads of 128) for eight prompts of 2,047 tokens
        case("product prompt", rows=16376, width=4096, out=6144),
        # sizes that no tile divides: a ragged batch, the last block of a row not whole, an odd number of outputs
        case("product odd", rows=333, width=2832, out=5001, code="e5m2"),
        # one token of one sequence, and a prompt, through the norm before a projection
        case("norm one token", kind="norm", rows=1, width=4096),
        case("norm prompt", kind="norm", rows=16376, width=8192),
        # a feed-forward of 4 times the width: a round of 32 sequences, and a chunk of a prompt
        case("gate round of 32", kind="gate", rows=160, width=16384),
        case("gate prompt", kind="gate", rows=4094, width=16384),
        # the attention's output for a round of 256, and a weight as it is loaded
        case("quantise round of 256", kind="quantise", rows=1280, width=4096),
        case("quantise weight", kind="quantise", rows=32000, width=4096, tile=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["product", "product", "product", "norm", "gate", "quantise"])
    c = dict(BASE, kind=kind, rows=rng.choice([_log(rng, 1, 16), _log(rng, 1, 300), _log(rng, 1, 16384)]),
             code=rng.choice(["e4m3", "e4m3", "e5m2"]))
    # whole blocks of 128, or any number that rows of 8-bit codes can have
    c["width"] = BLOCK * _log(rng, 1, 128) if rng.random() < 0.6 else 16 * _log(rng, 1, 1024)
    if kind == "product":
        most = min(152000, int(4e11 / (c["rows"] * c["width"])), int(5e8 / c["width"]), int(2e8 / c["rows"]))
        c["out"] = _log(rng, 1, max(1, most))
        c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        c["weight_code"] = rng.choice(["e4m3", "e4m3", "e5m2"])
    else:
        c["rows"] = min(c["rows"], max(1, int(1e8 / c["width"])))
        c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        c["residual"] = rng.random() < 0.75
        c["stream"] = rng.choice(["bf16", "bf16", "fp32"])
        c["act"] = rng.choice(["silu", "gelu_tanh"])
        c["tile"] = rng.choice([1, 128])
    return c


def _blocks(n):
    return -(-n // BLOCK)


def work(c):
    T, D, N = c["rows"], c["width"], c["out"]
    size = {"bf16": 2, "fp32": 4}
    if c["kind"] == "product":
        b = N * D + _blocks(N) * _blocks(D) + T * D + T * _blocks(D) + T * N * size[c["dtype"]]
        return {"bytes": b, "flops": 2 * T * N * D}
    coded = T * D + (_blocks(T) if c["kind"] == "quantise" and c["tile"] == 128 else T) * _blocks(D)
    if c["kind"] == "norm":
        stream = 2 * size[c["stream"]] * T * D if c["residual"] else 0
        return {"bytes": T * D * size[c["dtype"]] + stream + 4 * D + coded, "flops": 7 * T * D}
    if c["kind"] == "gate":
        return {"bytes": 2 * T * D * size[c["dtype"]] + coded, "flops": 8 * T * D}
    return {"bytes": T * D * size[c["dtype"]] + coded, "flops": 2 * T * D}


# ---------------------------------------------------------------------------
# the 8-bit form, in plain operations
# ---------------------------------------------------------------------------
def _exponent(amax, code):
    """e, 2^e the smallest power of two with amax <= 2^e * (largest code), -100 at least."""
    m, e = torch.frexp(amax)
    mt, et = math.frexp(torch.finfo(F8[code]).max)  # 1.75 * 2^8 and 1.75 * 2^15
    e = e - et + (m > mt).to(e.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)


def _tiles(x, tile):
    """[rows, width] -> [row blocks, tile, column blocks, 128], zeros behind the ends."""
    T, D = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(D) * BLOCK - D, 0, -(-T // tile) * tile - T))
    return x.reshape(-1, tile, _blocks(D), BLOCK)


def _code(x, code, tile=1):
    """Codes and scales of x (float32): what is not finite becomes NaN and counts for no scale."""
    t = _tiles(x, tile)
    fine = torch.isfinite(t)
    e = _exponent(torch.where(fine, t.abs(), torch.zeros_like(t)).amax((1, 3)), code)
    q = torch.ldexp(t, -e[:, None, :, None])
    q = torch.where(fine, q, torch.full_like(q, math.nan))
    q = q.reshape(t.shape[0] * tile, -1)[: x.shape[0], : x.shape[1]].contiguous()
    return q.to(F8[code]), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _value(codes, scale, tile=1):
    x = codes.float()
    e = scale.view(torch.uint8).to(torch.int32) - 127
    e = e.repeat_interleave(tile, 0)[: x.shape[0]].repeat_interleave(BLOCK, 1)[:, : x.shape[1]]
    return torch.ldexp(x, e)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(c, gen, spread=1.0):
    """Activations: a few strong channels, rows of different size."""
    T, D = c["rows"], c["width"]
    x = torch.randn(T, D, generator=gen, device="cuda")
    x *= 1 + 6 * (torch.rand(D, generator=gen, device="cuda") < 0.02).float()
    x *= torch.exp(spread * torch.randn(T, 1, generator=gen, device="cuda"))
    return x


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    T, D, N = c["rows"], c["width"], c["out"]
    s = dict(case=c)
    if c["kind"] == "product":
        s["rows"] = _code(_rows(c, gen), c["code"])
        w = torch.randn(N, D, generator=gen, device="cuda")
        w *= torch.exp(0.3 * torch.randn(N, 1, generator=gen, device="cuda")) / math.sqrt(D)
        s["weight"] = _code(w, c["weight_code"], BLOCK)
        return s
    dtype = TYPES[c["dtype"]]
    if c["kind"] == "norm":
        s["x"] = _rows(c, gen, 0.3).to(dtype)
        s["residual"] = (3 * _rows(c, gen)).to(TYPES[c["stream"]]) if c["residual"] else None
        s["factor"] = 1 + 0.2 * torch.randn(D, generator=gen, device="cuda")
    elif c["kind"] == "gate":
        # what a product of gate and up together hands over: the two side by side in one tensor
        both = torch.cat([_rows(c, gen, 0.3), _rows(c, gen, 0.3)], 1).to(dtype)
        s["gate"], s["up"] = both[:, :D], both[:, D:]
    else:
        s["x"] = _rows(c, gen).to(dtype)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _product(s):
    c = s["case"]
    return (_value(*s["rows"]) @ _value(*s["weight"], BLOCK).t()).to(TYPES[c["dtype"]])


def _norm(s):
    c = s["case"]
    h, total = s["x"].float(), None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        total = h.to(s["residual"].dtype)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["factor"]
    return (*_code(y, c["code"]), total)


def _gate(s):
    c = s["case"]
    g, u = s["gate"].float(), s["up"].float()
    # 0.5 * (1 + tanh(z)) is 1 / (1 + exp(-2 z)), which keeps its digits where tanh is near -1
    z = g if c["act"] == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
    return _code(g / (1 + torch.exp(-z)) * u, c["code"])


def _quantise(s):
    c = s["case"]
    return _code(s["x"].float(), c["code"], c["tile"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verification_45_gb300 as sv

        if c["kind"] == "product":
            return sv.rows_product(sv.Coded(*s["rows"]), sv.Coded(*s["weight"]), dtype=TYPES[c["dtype"]])
        code = F8[c["code"]]
        if c["kind"] == "norm":
            coded, total = sv.rows_norm(s["x"], s["factor"], residual=s["residual"], eps=EPS, code=code)
            return coded.codes, coded.scale, total
        if c["kind"] == "gate":
            return tuple(sv.rows_gate(s["gate"], s["up"], act=c["act"], code=code))
        return tuple((sv.rows_quantise if c["tile"] == 1 else sv.weight_quantise)(s["x"], code=code))
    return {"product": _product, "norm": _norm, "gate": _gate, "quantise": _quantise}[c["kind"]](s)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _fit(most, code):
    """The scales, as numbers, for the largest magnitudes `most` (float64) of the blocks."""
    top = 448.0 if code == "e4m3" else 57344.0
    s = torch.exp2(torch.ceil(torch.log2((most / top).clamp(min=2.0 ** -100))))
    s = torch.where(s * top < most, 2 * s, s)  # the logarithm is not exact next to a power of two
    return torch.where((s > 2.0 ** -100) & (0.5 * s * top >= most), 0.5 * s, s)


def _largest(x):
    """The largest magnitude of each 128 columns of each row of x."""
    return torch.stack([x[:, k:k + BLOCK].abs().amax(1) for k in range(0, x.shape[1], BLOCK)], 1)


def _grid(x, code, slack):
    """x (float64) to the nearest value of the 8-bit form, ties to even.  What lies within `slack` of itself from
    the middle between two values stays there: 32 bits may end on either side of it."""
    bits, low, top = (3, -6, 448.0) if code == "e4m3" else (2, -14, 57344.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=low) - bits)
    t = x / step
    off = (t - torch.floor(t) - 0.5).abs() * step
    return torch.where(off < slack * x.abs(), x, torch.round(t) * step).clamp(-top, top)


def _coded(y, code, slack=2.0 ** -20):
    """Codes and scales of y (float64).  A scale whose block lies within `slack` of a border, and its codes, are
    halfway between the two that 32 bits may choose."""
    spread = lambda t: t.repeat_interleave(BLOCK, 1)[:, : y.shape[1]]  # noqa: E731
    top = 448.0 if code == "e4m3" else 57344.0
    most = _largest(y)
    scale = _fit(most, code)
    part = most / (scale * top)  # in (1/2, 1], lower for the least scale
    up, down = part > 1 - slack, (part < 0.5 * (1 + slack)) & (scale > 2.0 ** -100)
    codes = _grid(y / spread(scale), code, slack)
    one = torch.ones_like(scale)
    codes = codes * spread(torch.where(up, 0.75 * one, torch.where(down, 1.5 * one, one)))
    return codes, scale * torch.where(up, 1.5 * one, torch.where(down, 0.75 * one, one))


def exact(c, seed):
    s = prepare(c, seed)
    D = c["width"]
    if c["kind"] == "product":
        a, sa = s["rows"]
        w, sw = s["weight"]
        out = torch.zeros(c["rows"], c["out"], dtype=torch.float64, device="cuda")
        for k in range(_blocks(D)):
            at = slice(k * BLOCK, (k + 1) * BLOCK)
            left = torch.exp2(sa.view(torch.uint8)[:, k].double() - 127)[:, None]
            right = torch.exp2(sw.view(torch.uint8)[:, k].double() - 127).repeat_interleave(BLOCK)[: c["out"], None]
            out.addmm_(a[:, at].double() * left, (w[:, at].double() * right).t())
        return out
    if c["kind"] == "quantise":
        x = s["x"].double()
        if c["tile"] == 1:
            scale = _fit(_largest(x), c["code"])
            each = scale
        else:
            scale = torch.stack([_fit(_largest(x[r:r + BLOCK]).amax(0), c["code"]) for r in range(0, len(x), BLOCK)])
            each = scale.repeat_interleave(BLOCK, 0)[: len(x)]
        return _grid(x / each.repeat_interleave(BLOCK, 1)[:, :D], c["code"], 0.0), scale
    if c["kind"] == "norm":
        h = s["x"].double()
        if c["residual"]:
            h = h + s["residual"].double()
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / D + EPS) * s["factor"].double()
        return (*_coded(y, c["code"]), h if c["residual"] else None)
    g, u = s["gate"].double(), s["up"].double()
    if c["act"] == "silu":
        return _coded(g * torch.sigmoid(g) * u, c["code"])
    return _coded(0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3)))) * u, c["code"])
