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
