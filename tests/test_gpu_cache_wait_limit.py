"""Waits inside the cache's kernels that run out: the call ends, the status says so,
nothing outside the outputs is written, and the next call is as ever."""
import pytest
import torch

from tests.test_gpu_cache import Case, dev, sv  # noqa: F401

pytestmark = pytest.mark.gpu

TREE = [[0, 0, 0, 1, 1, 2, 3], [0, 0, 1, 2, 3, 4, 5]]
CASES = {
    "one token": dict(lengths=[300], new=1),
    "units in parts": dict(lengths=[9000, 20], new=5, heads=16, kv_heads=2, dim=128, block=64),
    "many units": dict(lengths=[(37 * b) % 500 for b in range(200)], new=1, num_new=[min(1, 37 * b % 500) for b in range(200)]),
    "row tiles": dict(lengths=[700, 600], new=60, heads=16, kv_heads=2, dim=64, block=32),
    "tree with a bias": dict(lengths=[400, 290], new=7, heads=32, kv_heads=4, dim=128, parent=TREE, slopes=True, positions=True),
}


@pytest.fixture
def limit(sv):  # noqa: F811
    from speculative_decoding_verification_45_gb300 import _native

    lib = _native.load()

    def to(clocks):
        assert lib.spec_cache_set_wait_limit(clocks) == 0

    yield to
    to(2 ** 31 - 1)


def guarded(shape, dtype):
    """A tensor between two others, all of one value; and the whole."""
    n = 1
    for x in shape:
        n *= x
    whole = torch.full((n + 2048,), 7.0, dtype=dtype, device="cuda")
    return whole[1024:1024 + n].view(shape), whole


@pytest.mark.parametrize("name", CASES)
def test_a_wait_that_runs_out_is_reported(sv, limit, name):  # noqa: F811
    case = Case(seed=71, **CASES[name])
    cache, f = case.pool.to(sv), {k: dev(v) for k, v in case.form.items()}
    q, table, lengths = case.q.cuda(), case.table.cuda(), case.lengths.cuda()
    out, lse = sv.cache_attend(q, cache, table, lengths, **f)
    weights = torch.zeros(case.pool.codes.shape[1:4], device="cuda")
    sv.cache_weigh(q, cache, table, lengths, lse, weights, **f)
    codes = [x.view(torch.uint8).clone() for x in cache[:2]]
    for clocks in (0, 100, 300, 1000, 3000, 10000, 30000, 2 ** 31 - 1):
        limit(clocks)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (o, whole_o), (z, whole_z) = guarded(out.shape, out.dtype), guarded(lse.shape, lse.dtype)
        sv.cache_attend(q, cache, table, lengths, out=o, lse=z, status=status, **f)
        assert status.item() in (0, sv.STATUS_INTERNAL)
        if status.item() == 0:
            assert torch.equal(o, out) and torch.equal(z, lse)
        ended = [status.item()]
        status.zero_()
        w, whole_w = guarded(weights.shape, weights.dtype)
        w.zero_()
        sv.cache_weigh(q, cache, table, lengths, lse, w, status=status, **f)
        assert status.item() in (0, sv.STATUS_INTERNAL)
        if status.item() == 0:
            assert torch.equal(w, weights)
        ended.append(status.item())
        for whole in (whole_o, whole_z, whole_w):
            assert (whole[:1024] == 7).all() and (whole[-1024:] == 7).all()
        assert all(torch.equal(x, y.view(torch.uint8)) for x, y in zip(codes, cache[:2]))
        if clocks == 0:
            assert ended == [sv.STATUS_INTERNAL] * 2
        if clocks == 2 ** 31 - 1:
            assert ended == [0, 0]


def test_the_limit_is_checked(sv):  # noqa: F811
    from speculative_decoding_verification_45_gb300 import _native

    assert _native.load().spec_cache_set_wait_limit(-1) == sv.SPEC_ERR_INVALID_ARG
