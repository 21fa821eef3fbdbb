"""The product of 8-bit rows with 8-bit weights against its definition in 64 bits."""
import pytest
import torch

from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as sv

    return sv


def dev(coded, sv):
    return sv.Coded(coded.codes.cuda(), coded.scale.cuda())


def bound(out, total, dim, dtype):
    """A product of two codes is exact in 32 bits.  A sum of `dim` of them in any order that adds 32 at a time, each
    addition off by at most 2^-23 of the magnitudes so far, is off by (dim / 32 + 32) * 2^-23 of all magnitudes;
    then one rounding to the output's type, half a step."""
    return (dim / 32 + 32) * 2.0 ** -23 * total + torch.finfo(dtype).eps / 2 * out.abs()


def check(sv, rows, weight, got, dtype):
    want, total = ref.product(rows, weight)
    off = (got.cpu().double() - want).abs()
    assert (off <= bound(want, total, rows.codes.shape[-1], dtype)).all(), f"off by {(off / total.clamp(min=1e-30)).max()}"


SIZES = [  # rows, outputs, width: one of each, ends of tiles, blocks and words of scales, either arrangement
    (1, 1, 16), (1, 128, 128), (5, 130, 144), (16, 128, 512), (17, 257, 640), (3, 4096, 4096), (33, 1000, 1040),
    (64, 1000, 1024), (128, 384, 2832), (129, 300, 4096), (1, 5001, 2832), (200, 19300, 256), (333, 5001, 2832),
    (241, 9999, 528), (1000, 2777, 1040), (2100, 2500, 512), (97, 256, 8192), (4097, 640, 400),
]


@pytest.mark.parametrize("rows,outs,dim", SIZES)
@pytest.mark.parametrize("codes", [(E4, E4), (E5, E4), (E4, E5)], ids=["e4m3", "rows e5m2", "weight e5m2"])
def test_sizes(sv, rows, outs, dim, codes):
    gen = torch.Generator().manual_seed(rows * 7 + outs)
    a, w = ref.random_coded(rows, dim, codes[0], gen, sv), ref.random_coded(outs, dim, codes[1], gen, sv, 128)
    for dtype in (torch.float32, torch.bfloat16):
        got = sv.rows_product(dev(a, sv), dev(w, sv), dtype=dtype)
        assert got.shape == (rows, outs) and got.dtype == dtype
        check(sv, a, w, got, dtype)
