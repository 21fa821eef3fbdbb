"""Attention over the 8-bit cache where scales and scores lie far from 1.

Bounds: those of test_gpu_cache, whose absolute part goes by the value scale
here, and the grid of the weights written out: a token's weight times its value
scale is held to half of 2^-9 of a number of which the largest of its 128 tokens
has 224 or more, 2^-17 of that largest one."""
import math

import pytest
import torch

from tests import cache_reference as cr
from tests.test_gpu_cache import Case, sv, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


def grid(case, ref):
    """How far the weights' grid may move each output."""
    off = torch.zeros_like(ref["out"])
    group = ref["lse"].shape[2] // case.pool.heads
    for (b, i, h), (see, x, _) in ref["xs"].items():
        j = see.nonzero()[:, 0]
        page, row = case.table[b][j // case.pool.block].long(), j % case.pool.block
        scale = case.pool.scale[1, page, h // group]
        weight = torch.exp(x - ref["lse"][b, i, h]) * scale
        most = torch.zeros(int(j.max()) // 128 + 1, dtype=torch.float64).scatter_reduce(0, j // 128, weight, "amax")
        off[b, i, h] = 2.0 ** -17 * most[j // 128] @ case.pool.codes[1, page, h // group, row].abs()
    return off


def check(case, sv, unit, copies=90):  # noqa: F811
    """Alone, where an SM takes a tile or two, and `copies` times over, where it takes whole sequences."""
    ref = case.reference()
    none = torch.isneginf(ref["lse"])
    bound = (2.0 ** -8 * ref["out"].abs() + (1.5 * 2.0 ** -8 + 2 * ref["dx"][..., None]) * ref["mean"] + grid(case, ref)
             + 2.0 ** -30 * unit)
    cache = case.pool.to(sv)
    for n in (1, copies):
        def again(x):
            return x.cuda().repeat(n, *[1] * (x.dim() - 1))
        form = {k: again(v) if k in ("num_new", "prefix", "parent") else v.cuda() if k == "slopes" else v
                for k, v in case.form.items()}
        out, lse = sv.cache_attend(again(case.q), cache, again(case.table), again(case.lengths), **form)
        out, lse = out.cpu().double().unflatten(0, (n, -1)), lse.cpu().double().unflatten(0, (n, -1))
        assert torch.isfinite(out).all()
        assert (none == torch.isneginf(lse)).all() and (out[:, none] == 0).all()
        assert ((lse - ref["lse"]).abs()[:, ~none] <= ref["dx"][~none]).all()
        far = ((out - ref["out"]).abs() - bound)[:, ~none]
        assert (far <= 0).all(), (n, float(far.max() / unit))


COLUMNS = [dict(new=2, heads=8, kv_heads=1), dict(new=4, heads=16, kv_heads=2), dict(new=7, heads=16, kv_heads=2)]
SCALES = [-100, -40, 2, 20, 100]


def at_scale(case, exponent):
    case.pool.scale[1] = 2.0 ** exponent
    return 2.0 ** exponent * case.pool.codes[1].abs().mean().item()


@pytest.mark.parametrize("exponent", SCALES)
@pytest.mark.parametrize("columns", COLUMNS, ids=[16, 32, 48])
@pytest.mark.parametrize("dim,code", [(64, "e4m3"), (128, "e5m2"), (128, "e4m3")])
def test_value_scales_with_a_bias_that_leaves_tiles_nothing(sv, exponent, columns, dim, code):  # noqa: F811
    case = Case([650, 700, 90], dim=dim, block=32, code=code, seed=51, **columns)
    case.form["slopes"] = torch.linspace(0.3, 3.0, columns["heads"])
    check(case, sv, at_scale(case, exponent))


def opposed(case, nats, first=0):
    """Keys of the tokens from `first` blocks before the last on score about -nats."""
    case.q = case.q.abs()
    keys, scale, dim = case.pool.codes[0], case.pool.scale[0], case.q.shape[3]
    for b in range(len(case.lengths)):
        pages = case.table[b][: case.table.shape[1] - first].long()
        keys[pages] = -keys[pages].abs()
        size = keys[pages].abs().mean(dim=(2, 3)) * 0.8 * dim * case.form["scale"]
        scale[pages] = torch.exp2(torch.round(torch.log2(nats / size)))


@pytest.mark.parametrize("exponent", SCALES)
@pytest.mark.parametrize("columns", COLUMNS, ids=[16, 32, 48])
def test_value_scales_with_scores_that_leave_tiles_nothing(sv, exponent, columns):  # noqa: F811
    case = Case([640, 640], dim=64, block=16, seed=52, **columns)
    opposed(case, 300.0, first=6)
    check(case, sv, at_scale(case, exponent))


@pytest.mark.parametrize("exponent", SCALES)
@pytest.mark.parametrize("columns", COLUMNS, ids=[16, 32, 48])
@pytest.mark.parametrize("length", [300, 2100])
def test_value_scales_with_high_and_low_scores(sv, exponent, columns, length):  # noqa: F811
    case = Case([length], dim=128, block=64, seed=53, **columns)
    case.form["scale"] *= 12
    check(case, sv, at_scale(case, exponent))
    case = Case([length], dim=128, block=64, seed=54, **columns)
    opposed(case, 33.0)
    check(case, sv, at_scale(case, exponent))


def test_scales_of_blocks_that_nobody_sees(sv):  # noqa: F811
    """A scale next to a window, past a prefix or of later queries' tokens decides nothing."""
    case = Case([260], 9, heads=16, kv_heads=2, dim=64, block=16, window=20, prefix=[16], seed=55)
    unit = at_scale(case, -100)
    for blk in (1, 2, 3, 7, 9, 13):  # tokens 16 to 223: outside the prefix and every window
        case.pool.scale[1, case.table[0, blk]] = 2.0 ** 110
    check(case, sv, unit)


@pytest.mark.parametrize("form", [dict(), dict(window=3), dict(window=130), dict(window=40, prefix=[3, 0, 130, 2])], ids=str)
@pytest.mark.parametrize("nats", [200.0, 600.0, 2000.0])
@pytest.mark.parametrize("columns", [dict(new=5, heads=4, kv_heads=2), dict(new=5, heads=12, kv_heads=2),
                                     dict(new=9, heads=8, kv_heads=2)], ids=[16, 32, 48])
def test_low_scores_where_a_row_does_not_see_every_tile(sv, columns, nats, form):  # noqa: F811
    """Queries on both sides of a tile's border, and tiles that only some of them see."""
    case = Case([129, 131, 260, 390], dim=64, block=16, seed=56, **columns, **form)
    opposed(case, nats)
    check(case, sv, 1.0)


@pytest.mark.parametrize("page", [-2, -1, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("block", [16, 128])
def test_every_page_out_of_range_is_reported(sv, page, block):  # noqa: F811
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    case = Case([400, 90], 3, block=block, seed=57)
    case.table[0, 1] = page
    ref = case.reference()
    cache, f, (out, lse) = case.run(sv, status=status)
    assert status.item() == sv.STATUS_BAD_PAGE
    assert ((lse.cpu() - ref["lse"]).abs() <= ref["dx"]).all()
    status.zero_()
    w = torch.zeros(len(case.pool.codes[0]), 2, block, device="cuda")
    sv.cache_weigh(case.q.cuda(), cache, case.table.cuda(), case.lengths.cuda(), lse, w, status=status, **f)
    assert status.item() == sv.STATUS_BAD_PAGE


def test_an_evicted_block_of_bad_pages_has_a_scale(sv):  # noqa: F811
    """Its tokens are zeros, its scale the smallest one: what reads it later finds numbers."""
    pool = cr.Pool(8, 2, 16, 64, positions=True, seed=58)
    table, out = torch.tensor([[-1, 0, 3]], dtype=torch.int32), torch.tensor([[6, 7]], dtype=torch.int32)
    cache, status = pool.to(sv), torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.ones(8, 2, 16, device="cuda")
    lengths, index = sv.cache_evict(cache, table.cuda(), torch.tensor([30]).int().cuda(), w, 32, 4, out.cuda(), status=status)
    assert status.item() == sv.STATUS_BAD_PAGE and lengths.tolist() == [30] and index[0, 0, :30].tolist() == list(range(30))
    for codes, scale, side in ((cache.k, cache.k_scale, 0), (cache.v, cache.v_scale, 1)):
        assert (scale[6] == 2.0 ** -100).all() and (codes[6].float() == 0).all()
        assert torch.equal(scale[7].cpu().double(), pool.scale[side, 0])
    assert (w[6] == 0).all() and (cache.positions[6] == 0).all()
    # a second eviction of them, and attention over them, give numbers
    q = torch.randn(1, 1, 4, 64).to(torch.bfloat16).cuda()
    value, lse = sv.cache_attend(q, cache, out.cuda(), lengths)
    assert torch.isfinite(value).all() and torch.isfinite(lse).all()
    sv.cache_evict(cache, out.cuda(), lengths, w, 32, 4, torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"))
    assert not torch.isnan(cache.k.float()).any() and (cache.k_scale > 0).all()


@pytest.mark.parametrize("columns", COLUMNS, ids=[16, 32, 48])
@pytest.mark.parametrize("apart", [0, 8, 12, 16, 24])
@pytest.mark.parametrize("block", [16, 64])
def test_dimensions_that_only_small_blocks_fill(sv, columns, apart, block):  # noqa: F811
    """The stated precision of weights: 2^-8 of each, or 2^-17 of the largest weight times the largest scale of its
    128 tokens.  Where large-scaled blocks hold zeros, the second part shows."""
    case = Case([500], dim=64, block=block, seed=59, **columns)
    case.pool.scale[1] = 1.0
    large = case.table[0, :: 2].long()
    case.pool.scale[1, large] = 2.0 ** apart
    case.pool.codes[1, large, :, :, :32] = 0
    ref = case.reference()
    _, _, (out, lse) = case.run(sv)
    assert ((lse.cpu() - ref["lse"]).abs() <= ref["dx"]).all()
    step, group = torch.zeros_like(ref["out"]), columns["heads"] // columns["kv_heads"]
    for (b, i, h), (see, x, _) in ref["xs"].items():
        j = see.nonzero()[:, 0]
        page, row, tile = case.table[b][j // block].long(), j % block, j // 128
        p, scale = torch.exp(x - ref["lse"][b, i, h]), case.pool.scale[1, page, h // group]

        def most(y):
            return torch.zeros(4, dtype=torch.float64).scatter_reduce(0, tile, y, "amax")[tile]

        step[b, i, h] = 2.0 ** -17 * (most(p) * most(scale)) @ case.pool.codes[1, page, h // group, row].abs()
    bound = (2.0 ** -8 * ref["out"].abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * ref["dx"][..., None]) * ref["mean"] + step
             + 2.0 ** -30 * 2.0 ** apart)
    far = (out.cpu().double() - ref["out"]).abs() - bound
    assert (far <= 0).all(), float(far.max())


def test_a_nan_value_reaches_the_rows_that_see_it_even_without_weight(sv):  # noqa: F811
    """Some rows see it with an exponential of 0, some do not see it; the latter are as without it."""
    kw = dict(lengths=[300], new=4, heads=8, kv_heads=2, block=16, window=150)
    clean, case = Case(seed=60, **kw), Case(seed=60, **kw)
    for x in (clean, case):
        opposed(x, 400.0, first=5)
    at = 300 - 4 - 150 + 2  # the windows of queries 0 and 1 reach it
    case.pool.codes[1, case.table[0, at // 16], :, at % 16, 7] = math.nan
    ref = clean.reference()
    _, _, (out, lse) = case.run(sv)
    assert torch.isnan(out[0, :2]).any(-1).all() and torch.isfinite(out[0, 2:]).all()
    assert ((lse.cpu() - ref["lse"]).abs() <= ref["dx"]).all()
    _, _, (want, _) = clean.run(sv)
    assert torch.equal(out[0, 2:], want[0, 2:])


@pytest.mark.parametrize("columns,r,s", [(COLUMNS[0], 2.0 ** -10, 2.0 ** -21), (COLUMNS[1], 2.0 ** -10, 2.0 ** -21),
                                         (COLUMNS[2], 2.0 ** -8, 2.0 ** -17)], ids=[16, 32, 48])
@pytest.mark.parametrize("apart", [6, 14, 18, 20])
def test_weights_to_the_stated_precision(sv, columns, r, s, apart):  # noqa: F811
    """Of a weight r, or s of the largest weight times scale of its 128 tokens; a dimension that the heavy blocks
    leave at 0 shows the second part."""
    case = Case([500], dim=64, block=32, seed=62, **columns)
    case.pool.scale[1] = 1.0
    large = case.table[0, :: 2].long()
    case.pool.scale[1, large] = 2.0 ** apart
    case.pool.codes[1, large, :, :, :32] = 0
    case.pool.codes[0] = 0  # equal scores and values of one sign: the weights' errors add up
    case.pool.codes[1] = case.pool.codes[1].abs()
    ref = case.reference()
    _, _, (out, _) = case.run(sv)
    step, group = torch.zeros_like(ref["out"]), columns["heads"] // columns["kv_heads"]
    for (b, i, h), (see, x, _) in ref["xs"].items():
        j = see.nonzero()[:, 0]
        page, row, tile = case.table[b][j // 32].long(), j % 32, j // 128
        p, scale = torch.exp(x - ref["lse"][b, i, h]), case.pool.scale[1, page, h // group]
        most = torch.zeros(2, 4, dtype=torch.float64).scatter_reduce(1, tile.expand(2, -1), torch.stack([p, scale]), "amax")
        step[b, i, h] = s * most.prod(0)[tile] @ case.pool.codes[1, page, h // group, row].abs()
    bound = 2.0 ** -8 * ref["out"].abs() + (r + 2 * ref["dx"][..., None]) * ref["mean"] + step + 2.0 ** -30
    far = ((out.cpu().double() - ref["out"]).abs() - bound)[..., :32]
    assert (far <= 0).all(), float(far.max())


@pytest.mark.parametrize("small", [0, 4, 6, 9, 12])
@pytest.mark.parametrize("columns", COLUMNS, ids=[16, 32, 48])
def test_queries_to_the_stated_precision(sv, columns, small):  # noqa: F811
    """Exact down to 2^-14 of the row's largest element, 2^-21 of it below: that one meets keys of 0 here.  Beside it
    32-bit sums of 64 products."""
    case = Case([300], dim=64, block=16, seed=63, **columns)
    case.q = (case.q.float() * 2.0 ** -small).to(torch.bfloat16)
    case.q[..., 5] = 200.0
    case.pool.codes[0, ..., 5] = 0
    case.form["scale"] = 2.0 ** small / 8
    ref = case.reference()
    _, _, (_, lse) = case.run(sv)
    group = columns["heads"] // columns["kv_heads"]
    for (b, i, h), (see, x, _) in ref["xs"].items():
        k, _ = case.pool.tokens(0, case.table[b], h // group, 300)
        q, k = case.q[b, i, h].double(), k[see].abs()
        below = (q.abs() < 2.0 ** -14 * 200).double() * 2.0 ** -21 * 200
        err = case.form["scale"] * (k @ below + 2.0 ** -18 * k @ q.abs()) + 2.0 ** -22 * x.abs()
        p = torch.exp(x - ref["lse"][b, i, h])
        off = float((p * err).sum()) + 2.0 ** -20 * (1 + abs(float(ref["lse"][b, i, h])))
        assert abs(float(lse[b, i, h]) - float(ref["lse"][b, i, h])) <= off


@pytest.mark.parametrize("length", [90, 3000])
def test_scores_without_bounds_are_not_silent(sv, length):  # noqa: F811
    """Scores of 10^12: NaN where one is positive, as if nothing were seen where all are negative, never zeros with a
    finite lse."""
    case = Case([length], 3, heads=8, kv_heads=2, seed=64)
    case.form["scale"] = 1e12
    _, _, (out, lse) = case.run(sv)
    assert torch.isnan(out).all() and torch.isposinf(lse).all()
    case.form["scale"] = 0.125
    opposed(case, 33.0)
    case.form["scale"] = 1e12
    _, _, (out, lse) = case.run(sv)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("lengths,blocks,block", [([60, 40], 4, 16), ([40000], 625, 64), ([70000], 1100, 64)])
def test_evict_reports_a_bad_page_whose_tokens_it_drops(sv, lengths, blocks, block):  # noqa: F811
    pages, B = len(lengths) * (blocks + 2), len(lengths)
    x = torch.zeros(pages, 1, block, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = sv.KVCache(x, x.clone(), torch.ones(pages, 1, device="cuda"), torch.ones(pages, 1, device="cuda"))
    table = table_for(B, blocks + 2, pages, 65)
    w = torch.rand(pages, 1, block, generator=torch.Generator().manual_seed(65)).cuda() + 1
    for bad, want in ((None, 0), (-5, sv.STATUS_BAD_PAGE), (pages, sv.STATUS_BAD_PAGE)):
        t = table.clone()
        if bad is not None:
            t[0, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kept, index = sv.cache_evict(cache, t[:, :blocks].cuda(), torch.tensor(lengths).int().cuda(), w.clone(), 20, 4,
                                     t[:, blocks:].cuda(), status=status)
        assert status.item() == want and kept.tolist() == [20] * B
        if bad is not None:  # its tokens weigh less than any number
            assert not ((index[0, 0] >= block) & (index[0, 0] < 2 * block)).any()
