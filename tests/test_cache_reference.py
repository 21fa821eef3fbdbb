"""The host reference of the 8-bit cache's operators, pinned by values that follow from the definitions."""
import math

import pytest
import torch

from tests import cache_reference as cr


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
def test_rounding_agrees_with_the_codes_of_the_type(code):
    every = torch.arange(256, dtype=torch.uint8).view(cr.F8[code]).double()
    every = every[torch.isfinite(every)]
    assert torch.equal(cr.round8(every, code), every)
    x = torch.randn(20000, dtype=torch.float64).float() * 20
    assert torch.equal(cr.round8(x.double(), code), x.to(cr.F8[code]).double())


def test_scale_is_the_smallest_power_of_two_that_fits():
    for amax, s in [(448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (224.5, 1.0), (0.0, 2.0 ** -100), (1e-38, 2.0 ** -100)]:
        assert cr.scale_for(torch.tensor([0.0, -amax, math.nan, math.inf], dtype=torch.float64), "e4m3") == s


def test_mask_forms():
    assert cr.mask(5, 2, 0).tolist() == [True, True, True, True, False]
    assert cr.mask(5, 2, 1, window=2).tolist() == [False, False, False, True, True]
    assert cr.mask(5, 2, 1, window=2, prefix=1).tolist() == [True, False, False, True, True]
    tree = [0, 0, 0, 1]  # root 0; 1 and 2 under it; 3 under 1
    assert cr.mask(6, 4, 3, parent=tree).tolist() == [True, True, True, True, False, True]
    assert cr.mask(6, 4, 2, parent=tree).tolist() == [True, True, True, False, True, False]
    assert cr.mask(6, 4, 2, parent=[0, 0, 5, 0]).tolist() == [True, True, False, False, True, False]


def test_equal_scores_give_the_mean_and_equal_weights():
    pool = cr.Pool(2, 1, 16, 64)
    table = torch.tensor([[1, 0]])
    q = torch.zeros(1, 1, 2, 64)
    ref = cr.attend(pool, table, [20], q, 1.0)
    v, _ = pool.tokens(1, table[0], 0, 20)
    assert torch.allclose(ref["out"][0, 0, 0], v.mean(0))
    assert torch.allclose(ref["lse"], torch.full((1, 1, 2), math.log(20), dtype=torch.float64))
    w, _ = cr.weigh(pool, table, [20], ref, ref["lse"], torch.zeros(2, 1, 16))
    assert torch.allclose(w[1, 0], torch.full((16,), 2 / 20, dtype=torch.float64)) and w[0, 0, 4:].abs().sum() == 0


def test_append_moves_older_codes_when_the_scale_grows():
    pool = cr.Pool(1, 1, 16, 64)
    pool.codes.zero_()
    pool.codes[0, 0, 0, 0, 0], pool.scale[0, 0, 0] = 3.0, 0.5  # a key of 1.5
    k = torch.zeros(1, 1, 1, 64)
    k[0, 0, 0, 3] = 1000.0
    cr.append(pool, torch.tensor([[0]]), [1], k, torch.zeros_like(k))
    assert float(pool.scale[0, 0, 0]) == 4.0
    assert float(pool.codes[0, 0, 0, 0, 0]) == 0.375 and float(pool.codes[0, 0, 0, 1, 3]) == 256.0


def test_evict_keeps_the_heaviest_the_newest_and_the_lower_of_equals():
    pool = cr.Pool(4, 1, 16, 64)
    w = torch.zeros(4, 1, 16)
    w[0, 0, [2, 5, 9]] = torch.tensor([1.0, 3.0, 1.0])
    w[0, 0, 1] = math.nan
    kept, index = cr.evict(pool, torch.tensor([[0]]), [12], w, 5, 2, torch.tensor([[3]]))
    assert kept.tolist() == [5] and index[0, 0].tolist() == [2, 5, 9, 10, 11]
    assert w[3, 0, :5].tolist() == [1.0, 3.0, 1.0, 0.0, 0.0]
