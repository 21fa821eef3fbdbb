"""The operators of 8-bit rows from their definitions, in 64 bits on the CPU (test infrastructure)."""
import math

import torch

BLOCK = 128
FORMS = {torch.float8_e4m3fn: (3, -6, 448.0), torch.float8_e5m2: (2, -14, 57344.0)}


def blocks(n):
    return -(-n // BLOCK)


def spread(scale, shape, block_rows=1):
    """Scales [row blocks, blocks] at every element of a [rows, dim] matrix."""
    return scale.repeat_interleave(block_rows, 0)[: shape[0]].repeat_interleave(BLOCK, 1)[:, : shape[1]]


def scale_values(scale):
    """e8m0 bytes as float64."""
    byte = scale.cpu().view(torch.uint8).double()
    return torch.where(byte == 255, math.nan, torch.exp2(byte - 127))


def values(coded, block_rows=1):
    codes = coded.codes.cpu().double()
    flat = codes.reshape(-1, codes.shape[-1])
    return flat * spread(scale_values(coded.scale).reshape(-1, blocks(codes.shape[-1])), flat.shape, block_rows)


def largest(x, block_rows):
    """The largest finite magnitude of each block."""
    x = torch.where(torch.isfinite(x), x.abs(), 0.0)
    rows, dim = x.shape
    x = torch.nn.functional.pad(x, (0, blocks(dim) * BLOCK - dim, 0, -(-rows // block_rows) * block_rows - rows))
    return x.reshape(-1, block_rows, blocks(dim), BLOCK).amax((1, 3))


def fit(most, code):
    """2^e, the smallest with most <= 2^e * top, e >= -100 (powers of two and their products with top are exact)."""
    top = FORMS[code][2]
    s = torch.full_like(most, 2.0 ** -100)
    for _ in range(260):
        s = torch.where(s * top < most, 2 * s, s)
    return s


def nearest(x, code):
    """x to the nearest value of the form, ties to even, up to the largest."""
    bits, low, top = FORMS[code]
    _, e = torch.frexp(x.abs())
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=low) - bits)
    return (torch.round(x / step) * step).clamp(-top, top)


def quantise(x, code, block_rows=1):
    """(codes, scales) of x [rows, dim], all float64; what is not finite becomes NaN."""
    s = fit(largest(x, block_rows), code)
    q = nearest(x / spread(s, x.shape, block_rows), code)
    return torch.where(torch.isfinite(x), q, math.nan), s


def check_coded(coded, y, code, slack):
    """Codes and scales are those of y [rows, dim] (float64), of which the kernel knows each element to `slack` of itself."""
    got, s = coded.codes.cpu().double().reshape(y.shape), scale_values(coded.scale).reshape(len(y), -1)
    slack = torch.as_tensor(slack, dtype=torch.float64).expand(y.shape)
    most, edge = largest(y, 1), largest(slack, 1)
    ok = (s == fit(most * (1 - edge), code)) | (s == fit(most * (1 + edge), code))
    assert ok.all(), f"{(~ok).sum()} scales are off"
    z = y / spread(s, y.shape)
    fine = torch.isfinite(y)
    assert torch.isnan(got[~fine]).all()
    # the nearest code, or one that is as near for a z within slack
    off = (got - z).abs() - (nearest(z, code) - z).abs()
    bad = fine & ~(off <= 2 * slack * z.abs())
    assert not bad.any(), f"{bad.sum()} codes are off, by {off[bad].max()}"


def norm(x, residual, weight, eps):
    """(y, h) in float64."""
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return (y if weight is None else y * weight.double()), h


def gate(g, u, act):
    """(y, z) in float64, y = g / (1 + exp(-z)) * u."""
    g, u = g.double(), u.double()
    if act == "silu":
        return g * torch.sigmoid(g) * u, g
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return 0.5 * g * (1 + torch.tanh(inner)) * u, 2 * inner


def product(rows, weight):
    """(out, the sum of magnitudes) in float64."""
    a, w = values(rows), values(weight, BLOCK)
    return a @ w.t(), a.abs() @ w.abs().t()


def random_coded(rows, dim, code, gen, sv, block_rows=1, spread_of=5):
    """Codes of every size and scales 2^-spread_of .. 2^spread_of, each block's its own."""
    x = torch.randn(rows, dim, generator=gen) * torch.exp(torch.randn(rows, dim, generator=gen))
    codes = (x * 16).clamp(-448, 448).to(code)
    byte = torch.randint(127 - spread_of, 128 + spread_of, (-(-rows // block_rows), blocks(dim)), generator=gen)
    return sv.Coded(codes, byte.to(torch.uint8).view(torch.float8_e8m0fnu))
