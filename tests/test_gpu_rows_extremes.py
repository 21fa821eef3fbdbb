"""Norm and gate at the ends of their types' ranges, against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import rows_reference as ref
from tests.test_gpu_rows import NORM_SLACK

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as sv

    return sv


# NORM_SLACK counts 74 + 6 roundings of 2^-24, the sum's halved by the root: 2^-18.5.  The factor of a row that is scaled has 21
# binary digits at least, which adds 2^-22: still below 2^-18.  The other steps of the scaling are by powers of two.
@pytest.mark.parametrize("rows,dim", [(3, 16), (5, 272), (9, 1024), (2, 1040), (700, 4096), (6, 4096), (3, 16400), (2, 32768)])
@pytest.mark.parametrize("x_type,r_type", [(F32, None), (BF16, None), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("exponent", [56, 60, 63, 64, 100, 123])
def test_rows_whose_squares_pass_32_bits(sv, rows, dim, x_type, r_type, exponent):
    """Finite rows are normalised whatever their size, beside small ones and a row of zeros."""
    g = torch.Generator().manual_seed(exponent)
    x = torch.randn(rows, dim, generator=g).clamp(-7, 7) * 2.0 ** exponent  # below 2^126: sums stay finite
    x[1] = torch.randn(dim, generator=g)
    x[-1, : dim // 2] *= 2.0 ** -exponent
    x = x.to(x_type)
    r = None if r_type is None else (torch.randn(rows, dim, generator=g).clamp(-7, 7) * 2.0 ** (exponent - 1)).to(r_type)
    w = (1 + 0.3 * torch.randn(dim, generator=g)).clamp(0.1)
    coded, total = sv.rows_norm(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=1e-5)
    y, _ = ref.norm(x.float() if r is None else x.float() + r.float(), None, w, 1e-5)  # of the 32-bit sum
    ref.check_coded(coded, y, E4, NORM_SLACK)
    if r is not None:
        assert torch.equal(total.cpu(), (x.float() + r.float()).to(r_type))


@pytest.mark.parametrize("dim", [16, 1024, 4096, 32768])
def test_both_sides_of_the_border(sv, dim):
    """Rows of one value, of which the squares' sum is below 2^128, at it and above: 1 everywhere, or 1 / rms."""
    at = 64 - math.log2(dim) / 2
    x = torch.tensor([[2.0 ** (at - 0.001)], [2.0 ** at], [2.0 ** (at + 0.001)], [2.0 ** (at + 1)], [-(2.0 ** 127)], [torch.finfo(F32).max]])
    x = x.expand(6, dim).contiguous()
    for eps in (1e-6, 2.0 ** -126, 3e38):
        coded, _ = sv.rows_norm(x.cuda(), eps=eps, code=E5)
        # eps is handed on in 32 bits
        y, _ = ref.norm(x, None, None, torch.tensor(eps).double().item())
        ref.check_coded(coded, y, E5, NORM_SLACK)


def test_a_sum_that_is_no_longer_finite(sv):
    """An element that overflows in x + residual is an infinity: zeros and NaN, as for one that was given; others are as ever."""
    x, r = torch.full((3, 256), 2.0 ** 100), torch.full((3, 256), 2.0 ** 100)
    x[0, 7] = r[0, 7] = torch.finfo(F32).max
    x[1, 9] = -math.inf
    coded, total = sv.rows_norm(x.cuda(), residual=r.cuda())
    codes = coded.codes.float().cpu()
    assert codes[0, 7].isnan() and codes[1, 9].isnan() and codes[:2].isnan().sum() == 2 and codes[:2].nan_to_num().eq(0).all()
    y, _ = ref.norm(x[2:] + r[2:], None, None, 1e-6)
    last = sv.Coded(coded.codes.cpu()[2:], coded.scale.cpu().view(torch.uint8)[2:].view(coded.scale.dtype))
    ref.check_coded(last, y, E4, NORM_SLACK)
    assert torch.equal(total.cpu(), x + r)


def gated(g, u, act):
    """y = g / (1 + exp(-z)) * u and z, in float64 (which holds 1 + exp(-z) for all z here)."""
    g, u = g.double(), u.double()
    z = g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(z) * u, z


@pytest.mark.parametrize("act,low,high", [("silu", -170.0, -70.0), ("silu", -95.0, -80.0), ("silu", -90.0, 5.0),
                                          ("gelu_tanh", -14.0, -9.0), ("gelu_tanh", -11.0, 3.0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("code", [E4, E5])
def test_strongly_negative_gates(sv, act, low, high, dtype, code):
    """1 + exp(-z) passes 32 bits, or its reciprocal does; with a large partner the product is a number like any other."""
    gen = torch.Generator().manual_seed(11)
    g = (low + (high - low) * torch.rand(41, 400, generator=gen)).to(dtype)
    u = (torch.randn(41, 400, generator=gen) * torch.exp2(torch.arange(41) * 3.0)[:, None]).to(dtype)  # up to 2^122
    coded = sv.rows_gate(g.cuda(), u.cuda(), act=act, code=code)
    y, z = gated(g, u, act)
    # as for other gates: the exponential's argument is off by 2^-22 of itself through up to four roundings; four
    # exponentials of a quarter of it are off by 2^-22 each, and five products by 2^-24 each
    ref.check_coded(coded, y, code, 2.0 ** -19 + z.abs() * 2.0 ** -22)


def test_gates_at_the_ends(sv):
    """Gates past every exponential: 0, the gate's own size, or NaN where the definition has none."""
    big = torch.finfo(F32).max
    g = torch.tensor([-big, -1e30, -1e4, -1000.0, -400.0, 0.0, 400.0, 1e30, big, -math.inf, math.inf, math.nan])
    for act in ("silu", "gelu_tanh"):
        for partner in (1.0, 2.0 ** -20, big):
            gate = g[:, None].expand(12, 128).contiguous()
            coded = sv.rows_gate(gate.cuda(), torch.full((12, 128), partner).cuda(), act=act)
            got = coded.codes.double().cpu() * ref.scale_values(coded.scale)
            assert (got[:6] == 0).all()
            assert got[9].isnan().all() and got[11].isnan().all() and got[10].isnan().all()
            for i in (6, 7, 8):
                want = g[i].double().item() * partner
                if want > big:
                    assert got[i].isnan().all()
                else:
                    assert ((got[i] - want).abs() <= 2.0 ** -4 * want).all()
