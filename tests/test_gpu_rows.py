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


def test_what_is_not_finite(sv):
    """Infinities and NaN become NaN and enter no scale, whether alone in a block or with others."""
    x = rand(260, 400, 20, F32)
    x[3, 5], x[3, 200], x[77, 390] = float("inf"), float("nan"), -float("inf")
    x[100, 128:256] = float("nan")
    x[200, :128] = float("inf")
    for dtype in (F32, BF16):
        for call, block in ((sv.rows_quantise, 1), (sv.weight_quantise, 128)):
            y = x.to(dtype)
            got = call(y.cuda())
            codes, scale = ref.quantise(y.double(), E4, block)
            assert torch.equal(ref.scale_values(got.scale), scale)
            assert torch.equal(got.codes.cpu().double().nan_to_num(nan=1e9), codes.nan_to_num(nan=1e9))
    one = torch.ones_like(x)
    for coded in (sv.rows_gate(x.cuda(), one.cuda()), sv.rows_gate(one.cuda(), x.cuda())):
        assert torch.equal(coded.codes.float().isnan().cpu(), ~x.isfinite())
    # a row with an infinity or a NaN: zeros and NaN, or NaN alone; other rows are as ever
    coded, _ = sv.rows_norm(x.cuda())
    rows = x.isfinite().all(1)
    y, _ = ref.norm(x[rows], None, None, 1e-6)
    some = [t.cpu().view(torch.uint8)[rows].view(t.dtype) for t in coded]
    ref.check_coded(sv.Coded(*some), y, E4, NORM_SLACK)
    bad = coded.codes.float().cpu()[~rows]
    assert (bad.isnan() | (bad == 0)).all() and bad.isnan().any(1).all()


def test_zeros_and_the_smallest(sv):
    x = torch.zeros(4, 256)
    x[1, 3], x[2, 130], x[3] = 1e-40, 2.0 ** -120, 2.0 ** -110
    for coded in (sv.rows_quantise(x.cuda()), sv.rows_norm(torch.zeros(4, 256).cuda())[0]):
        assert not coded.codes.float().isnan().any()
    got = sv.rows_quantise(x.cuda())
    codes, scale = ref.quantise(x.double(), E4)
    assert torch.equal(ref.scale_values(got.scale), scale) and torch.equal(got.codes.cpu().double(), codes)


def test_borders_of_scales_and_codes(sv):
    """448 and 57344 times powers of two, the next number up, and the middles between codes."""
    for code, top in ((E4, 448.0), (E5, 57344.0)):
        x = torch.zeros(64, 128)
        for i in range(32):
            x[2 * i, 0] = top * 2.0 ** (i - 16)
            x[2 * i + 1, 0] = torch.nextafter(x[2 * i, 0], torch.tensor(1e9))
        steps = torch.arange(127) * 2.0 ** -10
        x[:, 1:] = x[:, :1] * steps
        got = sv.rows_quantise(x.cuda(), code=code)
        codes, scale = ref.quantise(x.double(), code)
        assert torch.equal(ref.scale_values(got.scale), scale) and torch.equal(got.codes.cpu().double(), codes)


def test_slices_and_leading_dimensions(sv):
    """Halves of one tensor, every other row, rows broadcast to many: as their dense copies."""
    both = rand(12, 2 * 288, 21).cuda()
    g, u = both[:, :288], both[:, 288:]
    a, b = sv.rows_gate(g, u), sv.rows_gate(g.contiguous(), u.contiguous())
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    x = both[::2, :288]
    assert torch.equal(sv.rows_quantise(x).codes.view(torch.uint8), sv.rows_quantise(x.contiguous()).codes.view(torch.uint8))
    three = both.view(3, 4, 576)[..., :288]
    c = sv.rows_quantise(three)
    assert c.codes.shape == (3, 4, 288) and c.scale.shape == (3, 4, 3)
    assert torch.equal(c.codes.view(torch.uint8).view(12, 288), sv.rows_quantise(g).codes.view(torch.uint8))
    r = both[:1, :288].expand(12, 288)
    one, s1 = sv.rows_norm(g, residual=r)
    two, s2 = sv.rows_norm(g, residual=r.contiguous())
    assert torch.equal(s1, s2) and torch.equal(one.codes.view(torch.uint8), two.codes.view(torch.uint8))
    row = sv.rows_quantise(both[0, :288])
    assert row.codes.shape == (288,) and row.scale.shape == (3,) and torch.equal(row.codes.view(torch.uint8), c.codes.view(torch.uint8)[0, 0])


def test_the_sum_in_place(sv):
    x, r = rand(33, 2048, 22).cuda(), rand(33, 2048, 23, F32).cuda()
    want, total = sv.rows_norm(x, residual=r)
    kept = r.clone()
    got, back = sv.rows_norm(x, residual=kept, out_sum=kept)
    assert back is kept and torch.equal(kept, total) and torch.equal(got.codes.view(torch.uint8), want.codes.view(torch.uint8))


def guarded(shape, dtype):
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 2048,), 77, dtype=torch.uint8, device="cuda")
    return whole[1024:1024 + n].view(dtype).view(shape), whole


@pytest.mark.parametrize("rows,dim", [(1, 16), (7, 144), (130, 1040)])
def test_nothing_else_is_written(sv, rows, dim):
    x = rand(rows, dim, 24).cuda()
    for call, above in ((lambda o: sv.rows_quantise(x, out=o), rows), (lambda o: sv.weight_quantise(x, out=o), ref.blocks(rows)),
                        (lambda o: sv.rows_norm(x, out=o), rows), (lambda o: sv.rows_gate(x, x, out=o), rows)):
        (c, whole_c), (s, whole_s) = guarded((rows, dim), E4), guarded((above, ref.blocks(dim)), torch.float8_e8m0fnu)
        call(sv.Coded(c, s))
        for whole in (whole_c, whole_s):
            assert (whole[:1024] == 77).all() and (whole[-1024:] == 77).all()
    assert sv.rows_quantise(x[:0]).codes.shape == (0, dim) and sv.rows_norm(x[:0], residual=x[:0])[1].shape == (0, dim)


def test_elements_past_32_bits(sv):
    """More than 2^32 elements: the last rows are where they belong."""
    x = torch.zeros(131100, 32768, dtype=BF16, device="cuda")
    last = rand(40, 32768, 25)
    x[-40:] = last.cuda()
    codes, scale = ref.quantise(last.double(), E4)
    got = sv.rows_quantise(x)
    assert torch.equal(got.codes[-40:].cpu().double(), codes) and torch.equal(ref.scale_values(got.scale[-40:]), scale)
    got = sv.rows_gate(x, x)
    assert torch.equal(got.codes[-40:].view(torch.uint8), sv.rows_gate(last.cuda(), last.cuda()).codes.view(torch.uint8))
    got, total = sv.rows_norm(x, residual=x)
    want, _ = sv.rows_norm(last.cuda(), residual=last.cuda())
    assert torch.equal(got.codes[-40:].view(torch.uint8), want.codes.view(torch.uint8)) and torch.equal(total[-40:].cpu(), last * 2)
    del total
    got = sv.weight_quantise(x)
    tail = 131100 - 131100 // 128 * 128
    codes, scale = ref.quantise(last[-tail:].double(), E4, 128)
    assert torch.equal(got.codes[-tail:].cpu().double(), codes) and torch.equal(ref.scale_values(got.scale[-1:]), scale)
