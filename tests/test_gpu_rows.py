"""Rows and weights to 8 bits, alone and after the norm and the gate, against their definitions in 64 bits."""
import pytest
import torch

from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as sv

    return sv


def rand(rows, dim, seed, dtype=BF16, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, dim, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))).to(dtype)


SIZES = [(1, 16), (1, 128), (3, 144), (7, 4096), (130, 272), (257, 1040), (1, 8192), (19, 2832), (2, 131072), (1000, 16)]


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("code", [E4, E5])
def test_rows_quantise(sv, rows, dim, dtype, code):
    x = rand(rows, dim, 3, dtype)
    got = sv.rows_quantise(x.cuda(), code=code)
    assert got.codes.shape == x.shape and got.codes.dtype == code and got.scale.shape == (rows, ref.blocks(dim))
    codes, scale = ref.quantise(x.double(), code)
    assert torch.equal(got.codes.cpu().double(), codes) and torch.equal(ref.scale_values(got.scale), scale)


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("code", [E4, E5])
def test_weight_quantise(sv, rows, dim, dtype, code):
    x = rand(rows, dim, 4, dtype)
    got = sv.weight_quantise(x.cuda(), code=code)
    assert got.scale.shape == (ref.blocks(rows), ref.blocks(dim))
    codes, scale = ref.quantise(x.double(), code, 128)
    assert torch.equal(got.codes.cpu().double(), codes) and torch.equal(ref.scale_values(got.scale), scale)


# 32-bit steps of the norm, each off by 2^-24 of its result at most: the sum of squares is a chain of up to 64 and a
# tree of 10 (a square root halves their effect), with the division, eps, the root, two products and the sum: < 2^-18
NORM_SLACK = 2.0 ** -18
NORM_SIZES = [(1, 16), (1, 4096), (5, 144), (3, 1024), (4, 1040), (65, 2048), (6, 2832), (2, 8192), (3, 16400), (2, 32768)]


@pytest.mark.parametrize("rows,dim", NORM_SIZES)
@pytest.mark.parametrize("x_type,r_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32), (BF16, None), (F32, None)])
@pytest.mark.parametrize("code,w_type", [(E4, F32), (E5, BF16), (E4, None)])
def test_norm(sv, rows, dim, x_type, r_type, code, w_type):
    x = rand(rows, dim, 5, x_type)
    r = None if r_type is None else rand(rows, dim, 6, r_type)
    w = None if w_type is None else (1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(7))).to(w_type)
    coded, total = sv.rows_norm(x.cuda(), None if w is None else w.cuda(), None if r is None else r.cuda(), eps=1e-5, code=code)
    y, h = ref.norm(x, r, w, 1e-5)
    ref.check_coded(coded, y, code, NORM_SLACK)
    if r is None:
        assert total is None
    else:
        assert total.dtype == r_type and torch.equal(total.cpu(), (x.float() + r.float()).to(r_type))


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("code,act", [(E4, "silu"), (E4, "gelu_tanh"), (E5, "silu")])
def test_gate(sv, rows, dim, dtype, code, act):
    g, u = rand(rows, dim, 8, dtype, 0.5) * 3, rand(rows, dim, 9, dtype, 0.5)
    coded = sv.rows_gate(g.cuda(), u.cuda(), act=act, code=code)
    y, z = ref.gate(g, u, act)
    # the exponential is off by 2^-21 and its argument, in units of log 2 and through up to four roundings, by 2^-22 of
    # it; the sum, the division (2 units) and the product by 2^-22
    ref.check_coded(coded, y, code, 2.0 ** -20 + z.abs() * 2.0 ** -22)
