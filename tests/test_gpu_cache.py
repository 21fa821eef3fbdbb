"""The 8-bit cache's operators on the GPU against their float64 definitions.

Bounds.  A bf16 output is rounded once: 2^-8 of its value.  Before that, each
weight p of the sum enters as two 4-bit significands (2^-8 p), from a 16-bit
value (2^-11 p), on a grid of 2^-17 of the largest p of its 128 tokens (2^-10 of
it over all of them): less than 1.5 * 2^-8 of sum p |v| together.  The scores'
bound is in cache_reference.attend; lse and weights are 32-bit sums of them.
Codes, scales and indices are exact."""
import math

import pytest
import torch

from tests import cache_reference as cr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as m
    from speculative_decoding_verification_45_gb300 import _native

    _native.build()
    return m


def table_for(batch, blocks, pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[: batch * blocks].reshape(batch, blocks).int()


def dev(x):
    return x if x is None or not isinstance(x, torch.Tensor) else x.cuda()


class Case:
    def __init__(self, lengths, new, heads=8, kv_heads=2, dim=64, block=16, code="e4m3", positions=False, seed=0, **form):
        g = torch.Generator().manual_seed(seed + 100)
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        B = len(lengths)
        blocks = max(1, -(-max(lengths) // block))
        self.pool = cr.Pool(B * blocks + 3, kv_heads, block, dim, code, positions, seed)
        self.table = table_for(B, blocks, B * blocks + 3, seed)
        if positions:
            self.pool.spread_positions(self.table)
        self.q = torch.randn(B, new, heads, dim, generator=g).to(torch.bfloat16)
        self.form = dict(scale=1 / math.sqrt(dim))
        for k, v in form.items():
            self.form[k] = torch.tensor(v, dtype=torch.int32) if k in ("num_new", "prefix", "parent") else v
        if form.get("slopes") is True:
            self.form["slopes"] = torch.exp2(-torch.arange(1, heads + 1).float() / 2)

    def reference(self):
        f = dict(self.form)
        scale = f.pop("scale")
        return cr.attend(self.pool, self.table, self.lengths, self.q, scale, **f)

    def run(self, sv, nhd=False, **kw):
        cache = self.pool.to(sv, nhd=nhd)
        f = {k: dev(v) for k, v in self.form.items()}
        return cache, f, sv.cache_attend(self.q.cuda(), cache, self.table.cuda(), self.lengths.cuda(), **f, **kw)


def check_attend(ref, out, lse):
    out, lse = out.cpu().double(), lse.cpu().double()
    none = torch.isneginf(ref["lse"])
    assert torch.equal(none, torch.isneginf(lse))
    nan = torch.isnan(ref["lse"])
    assert torch.equal(nan, torch.isnan(lse))
    live = ~none & ~nan
    assert (out[none] == 0).all()
    assert ((lse - ref["lse"]).abs()[live] <= ref["dx"][live]).all(), float((lse - ref["lse"]).abs()[live].max())
    bound = 2.0 ** -8 * ref["out"].abs() + (1.5 * 2.0 ** -8 + 2 * ref["dx"][..., None]) * ref["mean"] + 2.0 ** -30
    far = ((out - ref["out"]).abs() - bound)[live]
    assert (far <= 0).all(), float(far.max())


def check_both(sv, case, **kw):
    ref = case.reference()
    cache, f, (out, lse) = case.run(sv, **kw)
    check_attend(ref, out, lse)
    w0 = torch.rand(len(case.pool.codes[0]), case.pool.heads, case.pool.block)
    w = sv.cache_weigh(case.q.cuda(), cache, case.table.cuda(), case.lengths.cuda(), lse, w0.cuda(), **f)
    want, bound = cr.weigh(case.pool, case.table, case.lengths, ref, lse.cpu(), w0)
    far = (w.cpu().double() - want).abs() - bound
    assert (far <= 0).all(), float(far.max())
    return ref, out, lse


def test_many_short_sequences(sv):
    """Several short units to a CTA, of one tile and of a few, empty ones among them."""
    lengths = [(b * 37) % 290 for b in range(330)]
    new = [min(2, (b + 1) % 3, x) for b, x in enumerate(lengths)]
    check_both(sv, Case(lengths, 2, heads=6, kv_heads=3, num_new=new, seed=20))


def test_more_sequences_than_threads(sv):
    lengths = [1 + (b * 13) % 60 for b in range(1300)]
    new = [(b % 5) > 0 for b in range(1300)]  # every fifth asks nothing
    check_both(sv, Case(lengths, 1, heads=1, kv_heads=1, num_new=new, seed=22))


def test_nobody_asks(sv):
    case = Case([50, 300], 2, num_new=[0, 0])
    _, _, (out, lse) = case.run(sv)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_odd_queries_stay_in_their_rows(sv):
    """NaN, infinities and zeros in some rows; the others are as without them."""
    case = Case([200, 333], 3, heads=8, kv_heads=2, dim=128, seed=23)
    ref = case.reference()
    case.q[0, 1, 3, 7] = math.nan
    case.q[1, 2, 0, :] = math.inf
    case.q[1, 0, 5, 100] = -math.inf
    _, _, (out, lse) = case.run(sv)
    odd = torch.zeros(2, 3, 8, dtype=torch.bool)
    odd[0, 1, 3] = odd[1, 2, 0] = odd[1, 0, 5] = True
    assert torch.isnan(out.cpu()[odd]).all() and torch.isnan(lse.cpu()[odd]).all()
    out, lse = out.cpu(), lse.cpu()
    for key in ("out", "lse", "mean", "dx"):
        ref[key][odd] = 0
    out[odd], lse[odd] = 0, 0
    check_attend(ref, out, lse)


def test_pages_past_four_gigabytes(sv):
    """The same tokens on the first pages of a small pool and the last ones of a large one give the same bits."""
    pages, heads, block, dim = 36000, 8, 128, 128  # 4.7 GB each side
    small = cr.Pool(12, heads, block, dim, positions=True, seed=24)
    table, out_table = torch.arange(8).reshape(2, 4).int(), torch.tensor([[8, 9], [10, 11]]).int()
    g = torch.Generator().manual_seed(24)
    q = torch.randn(2, 3, 16, dim, generator=g).to(torch.bfloat16).cuda()
    new = torch.randn(2, 3, heads, dim, generator=g).to(torch.bfloat16).cuda()
    weights = torch.rand(12, heads, block, generator=g)
    lens = torch.tensor([300, 411]).int().cuda()
    slopes = torch.rand(16, generator=g).cuda()
    got = []
    for base in (0, pages - 12):
        n = 12 if base == 0 else pages
        a = small.to(sv)
        if base:
            big = []
            for t in a:
                x = torch.zeros((n, *t.shape[1:]), dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
                x[base:] = t.view(torch.uint8) if t.element_size() == 1 else t
                big.append(x.view(t.dtype))
            a = sv.KVCache(*big)
        w = torch.zeros(n, heads, block, device="cuda")
        w[base:] = weights.cuda()
        t, o = (table + base).cuda(), (out_table + base).cuda()
        sv.cache_append(a, t, lens, new, new)
        out, lse = sv.cache_attend(q, a, t, lens + 3, slopes=slopes)
        sv.cache_weigh(q, a, t, lens + 3, lse, w, slopes=slopes)
        kept, index = sv.cache_evict(a, t, lens + 3, w, 200, 20, o)
        got.append([out, lse, kept, index, w[base:], a.k.view(torch.uint8)[base:], a.v.view(torch.uint8)[base:],
                    a.k_scale[base:], a.v_scale[base:], a.positions[base:]])
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_many_row_tiles(sv):
    """More queries than one row tile holds, in sequences that are hardly longer."""
    lengths = [70 + 9 * b for b in range(24)]
    new = [min(64, 5 + 7 * b) for b in range(24)]
    check_both(sv, Case(lengths, 64, heads=16, kv_heads=4, dim=128, block=32, num_new=new, seed=21))


TREE = [[0, 0, 0, 1, 1, 2, 3], [0, 0, 1, 2, 3, 4, 5]]


@pytest.mark.parametrize("kw", [
    dict(lengths=[1], new=1),
    dict(lengths=[0, 1, 2, 17], new=1, num_new=[0, 1, 1, 1]),
    dict(lengths=[5, 16, 33, 128, 129, 300], new=3),
    dict(lengths=[700, 1, 260], new=1, heads=3, kv_heads=3, dim=128, block=64),
    dict(lengths=[130, 64], new=5, heads=16, kv_heads=2, dim=128, block=32, code="e5m2"),
    dict(lengths=[500], new=4, heads=32, kv_heads=2, dim=128, block=128),
    dict(lengths=[333, 90], new=17, heads=12, kv_heads=4, dim=64, block=64),
    dict(lengths=[400, 200], new=60, heads=6, kv_heads=2, num_new=[60, 33]),
    dict(lengths=[150, 220], new=100, heads=8, kv_heads=1, dim=128, num_new=[100, 0]),
    dict(lengths=[2100], new=2, heads=4, kv_heads=1, block=32),
], ids=lambda k: f"L{k['lengths']}n{k['new']}")
def test_causal(sv, kw):
    check_both(sv, Case(**kw))


@pytest.mark.parametrize("form", [
    dict(softcap=20.0), dict(slopes=True), dict(slopes=True, positions=True, softcap=5.0),
    dict(window=1), dict(window=50), dict(window=100000), dict(prefix=[0, 40, 1000]), dict(window=20, prefix=[4, 150, 300]),
    dict(window=30, prefix=[10, 0, 129], softcap=30.0, slopes=True, code="e5m2"),
], ids=str)
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64)])
def test_forms(sv, form, dim, block):
    check_both(sv, Case([37, 400, 290], 9, dim=dim, block=block, seed=3, **form))


@pytest.mark.parametrize("kw", [
    dict(lengths=[7, 100], new=7, parent=TREE),
    dict(lengths=[130, 260], new=7, parent=TREE, num_new=[5, 7], heads=32, dim=128, block=128),
    dict(lengths=[140, 200], new=7, parent=TREE, window=8, prefix=[3, 0], slopes=True, positions=True),
    dict(lengths=[400], new=256, heads=4, kv_heads=2, parent=[[0] + [i * 7 % (i + 1) * (i % 3 > 0) for i in range(255)]]),
], ids=lambda k: f"L{k['lengths']}")
def test_trees(sv, kw):
    check_both(sv, Case(seed=5, **kw))


def test_a_bad_parent_is_no_parent(sv):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    case = Case([60, 50], 4, parent=[[0, 0, 2, 1], [7, 0, -3, 2]])
    cache, f, (out, lse) = case.run(sv, status=status)
    check_attend(case.reference(), out, lse)
    assert status.item() == sv.STATUS_BAD_TREE


@pytest.mark.parametrize("nhd", [False, True])
def test_layouts_and_strided_queries(sv, nhd):
    case = Case([333, 90], 5, heads=16, kv_heads=4, dim=128, block=32, seed=8)
    check_both(sv, case, nhd=nhd)
    wide = torch.randn(2, 5, 3, 16, 128).to(torch.bfloat16).cuda()
    wide[:, :, 1] = case.q.cuda()
    cache = case.pool.to(sv, nhd=nhd)
    out, lse = sv.cache_attend(wide[:, :, 1], cache, case.table.cuda(), case.lengths.cuda())
    check_attend(case.reference(), out, lse)


def test_what_is_not_seen_changes_nothing(sv):
    """NaN codes after the length, outside every window, and at tokens that some queries see."""
    kw = dict(lengths=[150, 200], new=7, parent=TREE, window=70)
    clean, case = Case(seed=6, **kw), Case(seed=6, **kw)
    last = case.table[0, 149 // 16]
    case.pool.codes[:, last, :, 150 % 16:] = math.nan
    case.pool.codes[:, case.table[1, 0]] = math.nan
    case.pool.scale[:, case.table[1, 0]] = 2.0 ** 60
    node = 200 - 7 + 4  # sequence 1 is a chain: nodes 4, 5, 6 see it
    case.pool.codes[1, case.table[1, node // 16], :, node % 16, 5] = math.nan
    node = 150 - 7 + 2  # sequence 0: nodes 2 and 5 see node 2
    case.pool.codes[0, case.table[0, node // 16], :, node % 16, 3] = math.nan
    ref = clean.reference()
    _, f, (out, lse) = case.run(sv)
    cache = case.pool.to(sv)
    out, lse = out.cpu(), lse.cpu()
    hit = torch.zeros(2, 7, dtype=torch.bool)
    hit[1, 4:] = True
    hit[0, [2, 5]] = True
    assert torch.isnan(out[1, 4:, :, 5]).all() and torch.isnan(out[0, [2, 5]]).all()
    for key in ("out", "lse", "mean", "dx"):
        ref[key][hit] = 0
    lse[hit], out[hit] = 0, 0
    check_attend(ref, out, lse)


def test_large_and_tiny_scores(sv):
    for factor in (1e-6, 30.0, 2000.0):
        case = Case([300, 290], 3, seed=9, dim=128)
        case.form["scale"] *= factor
        check_both(sv, case)
    case = Case([260], 2, seed=10)
    case.q.zero_()
    check_both(sv, case)
    # scores that rise along the cache by hundreds, and fall
    for sign in (1, -1):
        case = Case([600], 2, seed=11, heads=2, kv_heads=1)
        for blk in range(case.table.shape[1]):
            case.pool.scale[0, case.table[0, blk]] = 2.0 ** (blk // 6 if sign > 0 else 6 - blk // 6)
        case.form["scale"] = 1.0
        check_both(sv, case)


def test_a_heavy_first_token_and_a_long_light_tail(sv):
    case = Case([3000], 1, heads=2, kv_heads=1, dim=64, seed=12)
    case.pool.codes[0] = cr.round8(case.pool.codes[0] / 64, "e4m3")
    page, rows = case.table[0, 0], case.pool.codes[0, case.table[0, 0], 0]
    rows[0] = cr.round8(case.q[0, 0, 0].double() * 60, "e4m3")
    case.pool.scale[0] = 2.0 ** -4
    check_both(sv, case)


def far_out(case, times):
    """The case's table with its first page `times` over, and the lengths to match."""
    table = torch.cat([case.table[:, :1].expand(-1, times), case.table[:, 1:]], 1).contiguous()
    return table.cuda(), (case.lengths + (times - 1) * case.pool.block).int().cuda()


@pytest.mark.parametrize("dim", [64, 128])
def test_a_window_far_from_its_prefix(sv, dim):
    """Between the prefix and the window lie 200 million tokens that nobody sees."""
    case = Case([300], 2, heads=20, kv_heads=1, dim=dim, block=128, window=4, prefix=[5], seed=31)
    ref, _, lse = check_both(sv, case)
    cache = case.pool.to(sv)
    table, lengths = far_out(case, 1562500)
    f = {k: dev(v) for k, v in case.form.items()}
    out, lse = sv.cache_attend(case.q.cuda(), cache, table, lengths, **f)
    check_attend(ref, out, lse)
    w = torch.zeros(len(case.pool.codes[0]), 1, 128)
    got = sv.cache_weigh(case.q.cuda(), cache, table, lengths, lse, w.cuda(), **f)
    want, bound = cr.weigh(case.pool, case.table, case.lengths, ref, lse.cpu(), w)
    assert ((got.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("offset", [100_000_001, 2 ** 31 - 2000, -2 ** 31])
def test_far_positions(sv, offset):
    """A bias goes by the distance, however far out both positions are."""
    case = Case([333, 70], 3, heads=6, kv_heads=2, positions=True, slopes=True, seed=32)
    case.pool.positions -= case.pool.positions.min()
    assert case.pool.positions.max() < 2000
    case.pool.positions += offset
    check_both(sv, case)


def test_a_bias_at_the_end_of_a_long_cache(sv):
    case = Case([500], 3, heads=4, kv_heads=2, block=128, window=200, slopes=True, seed=33)
    ref = case.reference()
    table, lengths = far_out(case, 1000000)
    f = {k: dev(v) for k, v in case.form.items()}
    out, lse = sv.cache_attend(case.q.cuda(), case.pool.to(sv), table, lengths, **f)
    check_attend(ref, out, lse)


def test_blocks_of_very_different_value_scales(sv):
    case = Case([256], 1, dim=64, seed=13)
    for blk in range(case.table.shape[1]):
        case.pool.scale[1, case.table[0, blk]] = 2.0 ** (-20 if blk % 2 else 3)
    check_both(sv, case)


def test_invalid_lengths_and_pages(sv):
    case = Case([40, 50, 60, 70], 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    case.lengths = torch.tensor([-1, 2, 10 ** 6, 70], dtype=torch.int32)
    _, _, (out, lse) = case.run(sv, status=status)
    assert status.item() == sv.STATUS_BAD_LENGTH
    assert torch.isneginf(lse[:3]).all() and (out[:3] == 0).all()
    good = Case([40, 50, 60, 70], 3)
    check_attend({k: v[3:] for k, v in good.reference().items() if k != "xs"}, out[3:], lse[3:])
    case = Case([40, 50, 60, 70], 3)
    case.table[1, 1] = -1
    case.table[3, 0] = 1000
    status.zero_()
    _, _, (out, lse) = case.run(sv, status=status)
    assert status.item() == sv.STATUS_BAD_PAGE
    check_attend(case.reference(), out, lse)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def equal_cache(pool, cache):
    for side, (codes, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert torch.equal(scale.cpu().double(), pool.scale[side])
        assert torch.equal(codes.cpu().double().nan_to_num(nan=1e9), pool.codes[side].nan_to_num(nan=1e9))
    if pool.positions is not None:
        assert torch.equal(cache.positions.cpu(), pool.positions)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", [
    dict(lengths=[0], n=1), dict(lengths=[15, 16, 0, 7], n=5), dict(lengths=[3, 40, 30], n=16, block=32),
    dict(lengths=[31, 0], n=17, num_new=[17, 0], block=32, dim=128), dict(lengths=[1, 100], n=200, block=128, dim=128),
    dict(lengths=[5, 60, 64], n=70, num_new=[70, 3, 64], block=64, code="e5m2", positions=True),
], ids=lambda k: str(k) if isinstance(k, dict) else str(k).split(".")[-1])
def test_append(sv, kw, dtype):
    lengths, n, dim, block = kw["lengths"], kw["n"], kw.get("dim", 64), kw.get("block", 16)
    g = torch.Generator().manual_seed(n)
    B, KH = len(lengths), 3
    blocks = -(-(max(lengths) + n) // block)
    pool = cr.Pool(B * blocks + 2, KH, block, dim, kw.get("code", "e4m3"), kw.get("positions", False), 1)
    table = table_for(B, blocks, B * blocks + 2, 2)
    kv = torch.randn(B, n, 2, KH, dim, generator=g).mul(3).to(dtype)
    kv[:, 0, 0, 0] *= 64  # a token that raises its block's scale
    kv[:, n // 2, 1, 1] = 0
    num_new = None if "num_new" not in kw else torch.tensor(kw["num_new"], dtype=torch.int32)
    positions = torch.randint(0, 999, (B, n), generator=g).int() if kw.get("positions") else None
    lens = torch.tensor(lengths, dtype=torch.int32)
    for _ in range(2):  # a second time over the same tokens: nothing but the first call's scales can change it
        cache = pool.to(sv)
        d = kv.cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.cache_append(cache, table.cuda(), lens.cuda(), d[:, :, 0], d[:, :, 1], num_new=dev(num_new),
                        positions=dev(positions), status=status)
        cr.append(pool, table, lengths, kv[:, :, 0], kv[:, :, 1], num_new, positions)
        equal_cache(pool, cache)
        assert status.item() == 0


def test_append_unaligned_input_and_nhd_pool(sv):
    pool = cr.Pool(6, 2, 16, 64, seed=4)
    table = table_for(1, 4, 6, 4)
    flat = torch.randn(1 + 20 * 2 * 64 * 2).to(torch.bfloat16)
    kv = flat[1:].reshape(1, 20, 2, 2, 64)
    cache = pool.to(sv, nhd=True)
    d = flat.cuda()[1:].reshape(1, 20, 2, 2, 64)
    sv.cache_append(cache, table.cuda(), torch.tensor([9]).int().cuda(), d[:, :, 0], d[:, :, 1])
    cr.append(pool, table, [9], kv[:, :, 0], kv[:, :, 1])
    equal_cache(pool, cache)


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
def test_append_values_at_the_ends_of_the_range(sv, code):
    x = torch.tensor([0.0, -0.0, 1e-40, 3e38, -3e38, math.inf, -math.inf, math.nan, 448.0, 448.001, 449.0, 57344.0,
                      57345.0, 1e-30, 2.0 ** -100, 240.0])
    k = torch.zeros(1, 16, 1, 64)
    k[0, :, 0, :] = x[:, None]
    k[0, :, 0, 1] = 1.0
    for n in (1, 2, 16):  # block by block of growing content
        for first in range(0, 16, n):
            pool, table = cr.Pool(3, 1, 16, 64, code, seed=2), torch.tensor([[2, 0]], dtype=torch.int32)
            cache = pool.to(sv)
            part = k[:, first:first + n].contiguous()
            sv.cache_append(cache, table.cuda(), torch.tensor([4]).int().cuda(), part.cuda(), part.cuda())
            cr.append(pool, table, [4], part, part)
            equal_cache(pool, cache)


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shift", [1, 23, 24, 25, 28, 31, 40, 130])
def test_scales_far_apart_in_a_block(sv, code, shift):
    """Codes move by 2^-shift, when a block's scale grows and when an eviction brings blocks together."""
    pool, table = cr.Pool(6, 2, 16, 64, code, seed=shift), torch.tensor([[2, 0]], dtype=torch.int32)
    top = 448.0 if code == "e4m3" else 57344.0
    for page in (2, 0):
        pool.codes[:, page, :, :, 0] = top
        pool.scale[:, page] = 2.0 ** -60
    pool.scale[:, 0] = 2.0 ** (-60 + shift)
    cache, w = pool.to(sv), torch.rand(6, 2, 16, generator=torch.Generator().manual_seed(shift))
    out = torch.tensor([[4, 5]], dtype=torch.int32)
    dw = w.cuda()
    sv.cache_evict(cache, table.cuda(), torch.tensor([30]).int().cuda(), dw, 20, 6, out.cuda())
    cr.evict(pool, table, [30], w, 20, 6, out)
    equal_cache(pool, cache)
    k = torch.full((1, 3, 2, 64), top * 2.0 ** (-60 + shift))
    sv.cache_append(cache, table[:, :1].contiguous().cuda(), torch.tensor([9]).int().cuda(), k.cuda(), k.cuda())
    cr.append(pool, table, [9], k, k)
    equal_cache(pool, cache)


def test_append_refuses_bad_data(sv):
    pool = cr.Pool(8, 2, 16, 64, seed=4)
    table = torch.tensor([[0, 1], [2, 3], [-1, 99], [4, 5]], dtype=torch.int32)
    k = torch.randn(4, 3, 2, 64).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = pool.to(sv)
    lengths, num_new = torch.tensor([30, -5, 14, 1]).int(), torch.tensor([3, 1, 3, 7]).int()
    sv.cache_append(cache, table.cuda(), lengths.cuda(), k.cuda(), k.cuda(), num_new=num_new.cuda(), status=status)
    equal_cache(pool, cache)  # nothing was written
    assert status.item() == sv.STATUS_BAD_LENGTH | sv.STATUS_BAD_PAGE


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kw", [
    dict(lengths=[1], keep=1, recent=0), dict(lengths=[0, 5, 60, 200], keep=20, recent=4),
    dict(lengths=[300, 64, 65], keep=64, recent=64, block=64), dict(lengths=[300, 100], keep=100, recent=0, block=32, dim=128),
    dict(lengths=[1500, 513], keep=130, recent=7, block=128, dim=128, code="e5m2", positions=True),
    dict(lengths=[777], keep=500, recent=13, positions=True),
], ids=str)
@pytest.mark.parametrize("weights", ["spread", "ties", "odd"])
def test_evict(sv, kw, weights):
    lengths, keep, block = kw["lengths"], kw["keep"], kw.get("block", 16)
    B, KH = len(lengths), 2
    blocks, out_blocks = max(1, -(-max(lengths) // block)), -(-keep // block)
    pages = B * (blocks + out_blocks) + 2
    pool = cr.Pool(pages, KH, block, kw.get("dim", 64), kw.get("code", "e4m3"), kw.get("positions", False), 3)
    both = table_for(B, blocks + out_blocks, pages, 3)
    table, out_table = both[:, :blocks].contiguous(), both[:, blocks:].contiguous()
    g = torch.Generator().manual_seed(keep)
    w = torch.randn(pages, KH, block, generator=g).exp()
    if weights == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    if weights == "odd":
        w = torch.randn(w.shape, generator=g)
        pick = torch.randint(0, 8, w.shape, generator=g)
        for i, x in enumerate([math.nan, math.inf, -math.inf, -0.0, 0.0]):
            w[pick == i] = x
    cache, dw = pool.to(sv), w.cuda()
    kept, index = sv.cache_evict(cache, table.cuda(), torch.tensor(lengths).int().cuda(), dw, keep, kw["recent"],
                                 out_table.cuda())
    want_kept, want_index = cr.evict(pool, table, lengths, w, keep, kw["recent"], out_table)
    assert torch.equal(kept.cpu(), want_kept) and torch.equal(index.cpu(), want_index)
    equal_cache(pool, cache)
    assert torch.equal(dw.cpu().nan_to_num(nan=1e9), w.nan_to_num(nan=1e9))


@pytest.mark.parametrize("kw", [
    dict(lengths=[9000, 8192, 300, 0], heads=2), dict(lengths=[40001], heads=1), dict(lengths=[32768, 32761], heads=3),
    dict(lengths=[17000, 4, 16383], heads=11, keep=3000, recent=0), dict(lengths=[33000], heads=2, keep=64, recent=64),
    dict(lengths=[33000, 2999, 3000, 3001], heads=1, keep=3000, recent=2999),
], ids=str)
@pytest.mark.parametrize("weights", ["spread", "ties", "none"])
def test_evict_from_long_sequences(sv, kw, weights):
    """Lengths at which several CTAs share a sequence's selection, uneven shares and empty ones among them."""
    lengths, heads, keep, recent = kw["lengths"], kw["heads"], kw.get("keep", 700), kw.get("recent", 33)
    block, B = 64, len(kw["lengths"])
    blocks, out_blocks = -(-max(lengths) // block), -(-keep // block)
    pages = B * (blocks + out_blocks)
    x = torch.zeros(pages, heads, block, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    one = torch.ones(pages, heads, device="cuda")
    table = table_for(B, blocks + out_blocks, pages, 41)
    g = torch.Generator().manual_seed(keep + heads)
    w = torch.randn(pages, heads, block, generator=g).exp()
    if weights == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    if weights == "none":
        w.zero_()
    kept, index = sv.cache_evict(sv.KVCache(x, x.clone(), one, one.clone()), table[:, :blocks].cuda(),
                                 torch.tensor(lengths).int().cuda(), w.cuda(), keep, recent, table[:, blocks:].cuda())
    assert kept.tolist() == [min(n, keep) for n in lengths]
    for b, n in enumerate(lengths):
        for h in range(heads):
            got = index[b, h].cpu()
            if n <= keep:
                want = torch.arange(n)
            else:
                j = torch.arange(n - recent)
                heavy = w[table[b, j // block].long(), h, j % block].sort(descending=True, stable=True).indices[:keep - recent]
                want = torch.cat([heavy.sort().values, torch.arange(n - recent, n)])
            assert torch.equal(got[:len(want)].long(), want) and (got[len(want):] == -1).all()


def test_evict_in_place_of_the_lengths(sv):
    """More (sequence, head) pairs than run at once: the later ones must not see the new lengths."""
    B, KH, blocks, keep = 90, 16, 40, 32
    pages = B * (blocks + 2)
    x = torch.zeros(pages, KH, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = sv.KVCache(x, x.clone(), torch.ones(pages, KH, device="cuda"), torch.ones(pages, KH, device="cuda"))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).reshape(B, blocks + 2).int().cuda()
    lengths = torch.randint(0, 641, (B,), generator=torch.Generator().manual_seed(3)).int().cuda()
    w = torch.rand(pages, KH, 16, generator=torch.Generator().manual_seed(4)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, index = sv.cache_evict(cache, table[:, :blocks], lengths, w.clone(), keep, 8, table[:, blocks:])
    for _ in range(5):
        own = lengths.clone()
        got, again = sv.cache_evict(cache, table[:, :blocks], own, w.clone(), keep, 8, table[:, blocks:], out_lengths=own,
                                    status=status)
        assert got is own and torch.equal(own, kept) and torch.equal(again, index)
    assert status.item() == 0 and torch.equal(kept, lengths.clamp(max=keep))


def test_evict_from_more_tokens_than_shared_memory_holds(sv):
    """70,000 tokens in the table: the keys are read from memory at each step."""
    pages = 70000 // 128 + 1
    pool = cr.Pool(pages + 2, 1, 128, 64, seed=1)
    table = table_for(1, pages, pages, 5)
    w = torch.randn(pages + 2, 1, 128, generator=torch.Generator().manual_seed(1)).exp()
    cache, dw = pool.to(sv), w.cuda()
    out = torch.tensor([[pages, pages + 1]], dtype=torch.int32)
    _, index = sv.cache_evict(cache, table.cuda(), torch.tensor([69999]).int().cuda(), dw, 200, 50, out.cuda())
    _, want = cr.evict(pool, table, [69999], w, 200, 50, out)
    assert torch.equal(index.cpu(), want)
    equal_cache(pool, cache)


def test_evict_refuses_bad_data(sv):
    pool = cr.Pool(8, 1, 16, 64, seed=4)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = pool.to(sv)
    w = torch.ones(8, 1, 16, device="cuda")
    kept, index = sv.cache_evict(cache, table.cuda(), torch.tensor([99, 20]).int().cuda(), w, 4, 2,
                                 torch.tensor([[6], [-1]]).int().cuda(), status=status)
    assert kept.tolist() == [0, 4] and index[0, 0].tolist() == [-1] * 4
    assert status.item() == sv.STATUS_BAD_LENGTH | sv.STATUS_BAD_PAGE
    equal_cache(pool, cache)


# ---------------------------------------------------------------------------
# streams, graphs, repetition
# ---------------------------------------------------------------------------
def test_the_same_bits_again_on_another_stream_and_from_a_graph(sv):
    case = Case([3000, 700, 20], 5, heads=16, kv_heads=2, dim=128, block=64, seed=14)
    cache = case.pool.to(sv)
    q, table, lens = case.q.cuda(), case.table.cuda(), case.lengths.cuda()
    out, lse = sv.cache_attend(q, cache, table, lens)
    w = sv.cache_weigh(q, cache, table, lens, lse, torch.zeros(len(case.pool.codes[0]), 2, 64, device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out2, lse2, w2 = torch.empty_like(out), torch.empty_like(lse), torch.zeros_like(w)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        sv.cache_attend(q, cache, table, lens, out=out2, lse=lse2, stream=side)
    sv.cache_weigh(q, cache, table, lens, lse2, w2, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(w, w2)
    graph = torch.cuda.CUDAGraph()
    w2.zero_()
    with torch.cuda.graph(graph):
        sv.cache_attend(q, cache, table, lens, out=out2, lse=lse2)
        sv.cache_weigh(q, cache, table, lens, lse2, w2)
    for t in (out2, lse2, w2):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(w, w2)
    # a captured call follows what the lengths and the table say when it is replayed
    lens.sub_(5)
    graph.replay()
    torch.cuda.synchronize()
    case.lengths -= 5
    check_attend(case.reference(), out2, lse2)


def test_append_and_evict_in_a_graph(sv):
    pool = cr.Pool(12, 2, 16, 64, seed=15)
    table, out_table = torch.arange(8).reshape(2, 4).int(), torch.tensor([[8], [9]]).int()
    k = torch.randn(2, 4, 2, 64).to(torch.bfloat16)
    w = torch.rand(12, 2, 16)
    cache, lens, dk, dw = pool.to(sv), torch.tensor([20, 33]).int().cuda(), k.cuda(), w.cuda()
    dt, do = table.cuda(), out_table.cuda()
    after = torch.tensor([24, 37]).int().cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.cache_append(cache, dt, lens, dk, dk)
        kept, index = sv.cache_evict(cache, dt, after, dw, 16, 4, do)
    graph.replay()
    torch.cuda.synchronize()
    cr.append(pool, table, [20, 33], k, k)
    want_kept, want_index = cr.evict(pool, table, [24, 37], w, 16, 4, out_table)
    assert torch.equal(kept.cpu(), want_kept) and torch.equal(index.cpu(), want_index)
    equal_cache(pool, cache)


def test_no_sequences_and_no_new_tokens(sv):
    case = Case([40], 1)
    cache = case.pool.to(sv)
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = sv.cache_attend(torch.empty(0, 2, 8, 64, dtype=torch.bfloat16, device="cuda"), cache, none, lens)
    assert out.shape == (0, 2, 8, 64) and lse.shape == (0, 2, 8)
    out, lse = sv.cache_attend(torch.empty(1, 0, 8, 64, dtype=torch.bfloat16, device="cuda"), cache, case.table.cuda(),
                               case.lengths.cuda())
    assert out.shape == (1, 0, 8, 64)
    sv.cache_append(cache, case.table.cuda(), case.lengths.cuda(), *[torch.empty(1, 0, 2, 64, device="cuda")] * 2)
    torch.cuda.synchronize()
