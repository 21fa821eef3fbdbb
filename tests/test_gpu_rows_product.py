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


@pytest.mark.parametrize("rows", [1, 31, 33, 48, 70, 100, 130, 160, 170, 200, 223, 240, 250])
def test_tiles(sv, rows):
    """76 weight tiles of 256 leave one tile of rows to each pair of SMs: tiles of every size."""
    gen = torch.Generator().manual_seed(rows)
    a, w = ref.random_coded(rows, 272, E4, gen, sv), ref.random_coded(19400, 272, E4, gen, sv, 128)
    check(sv, a, w, sv.rows_product(dev(a, sv), dev(w, sv), dtype=torch.float32), torch.float32)


@pytest.mark.parametrize("rows,outs,dim", [(1, 700, 1040), (20, 8192, 1536), (160, 2049, 2832), (300, 520, 16400), (1, 300, 131072)])
def test_parts_of_k(sv, rows, outs, dim):
    gen = torch.Generator().manual_seed(5)
    a, w = ref.random_coded(rows, dim, E4, gen, sv), ref.random_coded(outs, dim, E4, gen, sv, 128)
    for dtype in (torch.float32, torch.bfloat16):
        check(sv, a, w, sv.rows_product(dev(a, sv), dev(w, sv), dtype=dtype), dtype)


def test_scales_of_every_size(sv):
    """Blocks whose scales' product is 1 though each is at an end of the range, next to blocks that add nothing."""
    gen = torch.Generator().manual_seed(6)
    a, w = ref.random_coded(40, 512, E4, gen, sv, spread_of=1), ref.random_coded(300, 512, E4, gen, sv, 128, spread_of=1)
    byte, other = a.scale.view(torch.uint8), w.scale.view(torch.uint8)
    byte[:, 0], other[:, 0] = 250, 4
    byte[:, 1], other[:, 1] = 3, 251
    byte[:, 2], other[:, 2] = 20, 10  # 2^-224
    check(sv, a, w, sv.rows_product(dev(a, sv), dev(w, sv), dtype=torch.float32), torch.float32)


def test_nan(sv):
    gen = torch.Generator().manual_seed(7)
    a, w = ref.random_coded(50, 528, E4, gen, sv), ref.random_coded(400, 528, E4, gen, sv, 128)
    clean = sv.rows_product(dev(a, sv), dev(w, sv), dtype=torch.float32)
    a.codes.view(torch.uint8)[7, 500] = 0x7F
    a.scale.view(torch.uint8)[9, 3] = 255
    w.codes.view(torch.uint8)[300, 1] = 0xFF
    got = sv.rows_product(dev(a, sv), dev(w, sv), dtype=torch.float32)
    bad = torch.zeros(50, 400, dtype=torch.bool)
    bad[7], bad[9], bad[:, 300] = True, True, True
    assert torch.equal(got.isnan().cpu(), bad) and torch.equal(got[~bad.cuda()], clean[~bad.cuda()])
    w.scale.view(torch.uint8)[1, 0] = 255
    bad[:, 128:256] = True
    assert torch.equal(sv.rows_product(dev(a, sv), dev(w, sv), dtype=torch.float32).isnan().cpu(), bad)


@pytest.mark.parametrize("rows,outs,dim", [(3, 130, 272), (70, 5000, 528), (500, 5000, 528)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nothing_else_is_written(sv, rows, outs, dim, dtype):
    """Rows of a wider tensor, at a stride that is no multiple of 16 bytes and at one that is; the rest stays."""
    gen = torch.Generator().manual_seed(8)
    a, w = dev(ref.random_coded(rows, dim, E4, gen, sv), sv), dev(ref.random_coded(outs, dim, E4, gen, sv, 128), sv)
    want = sv.rows_product(a, w, dtype=dtype)
    for extra, at in ((3, 1), (24, 8)):
        whole = torch.full((rows + 2, outs + extra), 7.0, dtype=dtype, device="cuda")
        got = sv.rows_product(a, w, out=whole[1:-1, at:at + outs])
        assert torch.equal(got, want)
        whole[1:-1, at:at + outs] = 7
        assert (whole == 7).all()


def test_strided_operands(sv):
    """Columns of wider codes, scales among others, and leading dimensions."""
    gen = torch.Generator().manual_seed(9)
    a, w = ref.random_coded(6 * 35, 1024, E4, gen, sv), ref.random_coded(700, 1024, E4, gen, sv, 128)
    part = sv.Coded(a.codes[:, 256:896], a.scale[:, 2:7]), sv.Coded(w.codes[:, 256:896], w.scale[:, 2:7])
    on = [sv.Coded(x.codes.cuda()[:, 256:896], x.scale.cuda()[:, 2:7]) for x in (a, w)]
    got = sv.rows_product(*on, dtype=torch.float32)
    check(sv, *[sv.Coded(x.codes.contiguous(), x.scale.contiguous()) for x in part], got, torch.float32)
    three = sv.Coded(on[0].codes.unflatten(0, (6, 35)), on[0].scale.unflatten(0, (6, 35)))
    assert torch.equal(sv.rows_product(three, on[1], dtype=torch.float32), got.view(6, 35, 700))


def test_no_rows_and_no_outputs(sv):
    gen = torch.Generator().manual_seed(10)
    a, w = dev(ref.random_coded(5, 64, E4, gen, sv), sv), dev(ref.random_coded(9, 64, E4, gen, sv, 128), sv)
    assert sv.rows_product(sv.Coded(a.codes[:0], a.scale[:0]), w).shape == (0, 9)
    assert sv.rows_product(a, sv.Coded(w.codes[:0], w.scale[:0])).shape == (5, 0)


@pytest.mark.parametrize("rows,outs,dim", [(1, 4096, 4096), (160, 2560, 2560), (1000, 4000, 1024)])
def test_the_same_bits_every_time(sv, rows, outs, dim):
    gen = torch.Generator().manual_seed(11)
    a, w = dev(ref.random_coded(rows, dim, E4, gen, sv), sv), dev(ref.random_coded(outs, dim, E4, gen, sv, 128), sv)
    first = sv.rows_product(a, w, dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(sv.rows_product(a, w, dtype=torch.float32), first)


def test_outputs_past_32_bits(sv):
    """More than 2^32 outputs: the last rows are where they belong."""
    gen = torch.Generator().manual_seed(12)
    w = ref.random_coded(65600, 128, E4, gen, sv, 128)
    tail = ref.random_coded(300, 128, E4, gen, sv)
    codes = torch.zeros(66000, 128, dtype=torch.uint8, device="cuda").view(E4)
    scale = torch.full((66000, 1), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    codes.view(torch.uint8)[-300:] = tail.codes.view(torch.uint8).cuda()
    scale.view(torch.uint8)[-300:] = tail.scale.view(torch.uint8).cuda()
    got = sv.rows_product(sv.Coded(codes, scale), dev(w, sv))
    assert not got[:-300].any()
    check(sv, tail, w, got[-300:], torch.bfloat16)


@pytest.mark.parametrize("rows,outs,dim", [
    (1, 1, 100000), (16, 9, 6656), (1, 300, 14336), (200, 250, 12672), (70, 250, 5008), (37, 777, 2048), (9, 2048, 16384), (33, 1025, 16400),
    (240, 250, 131072), (240, 3840, 16384)])
def test_many_parts_of_k(sv, rows, outs, dim):
    """Four to eight parts, narrow and wide tiles, parts that get no equal share; each time the same bits."""
    gen = torch.Generator().manual_seed(12)
    a, w = ref.random_coded(rows, dim, E4, gen, sv), ref.random_coded(outs, dim, E4, gen, sv, 128)
    for dtype in (torch.float32, torch.bfloat16):
        got = sv.rows_product(dev(a, sv), dev(w, sv), dtype=dtype)
        check(sv, a, w, got, dtype)
        assert all(torch.equal(sv.rows_product(dev(a, sv), dev(w, sv), dtype=dtype), got) for _ in range(3))
