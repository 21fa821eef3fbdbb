"""A round of a candidate tree over the 8-bit cache: the accepted path's keys and
values are written again behind the tokens before the tree, where the next
round's queries find them in order."""
import pytest
import torch

from tests import cache_reference as cr
from tests.test_gpu_cache import check_attend, sv, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
def test_the_accepted_path_is_written_again(sv, code):  # noqa: F811
    g = torch.Generator().manual_seed(61)
    before, n, heads, kv_heads, dim, block = [37, 127, 0], 7, 8, 2, 64, 16
    parent = torch.tensor([[0, 0, 0, 1, 1, 2, 4], [0, 0, 1, 0, 3, 4, 5], [0, 0, 1, 2, 3, 4, 5]], dtype=torch.int32)
    # as tree_verify gives them: accepted nodes, then -1, and their number
    out_path = torch.tensor([[1, 4, 6, -1, -1, -1, -1], [3, 4, -1, -1, -1, -1, -1], [-1] * 7], dtype=torch.int32)
    accepted = torch.tensor([3, 2, 0], dtype=torch.int32)
    path = torch.cat([torch.zeros_like(out_path[:, :1]), out_path[:, :-1].clamp(min=0)], 1).long()  # the root first
    taken = accepted + 1
    lengths = torch.tensor(before, dtype=torch.int32)
    pool = cr.Pool(40, kv_heads, block, dim, code, seed=61)
    table = table_for(3, 10, 40, 61)
    kv = torch.randn(3, n, 2, kv_heads, dim, generator=g).to(torch.bfloat16)
    q = torch.randn(3, n, heads, dim, generator=g).to(torch.bfloat16)
    cache, dt, dl, dkv = pool.to(sv), table.cuda(), lengths.cuda(), kv.cuda()

    sv.cache_append(cache, dt, dl, dkv[:, :, 0], dkv[:, :, 1])
    cr.append(pool, table, before, kv[:, :, 0], kv[:, :, 1])
    out, lse = sv.cache_attend(q.cuda(), cache, dt, dl + n, parent=parent.cuda())
    check_attend(cr.attend(pool, table, lengths + n, q, dim ** -0.5, parent=parent), out, lse)

    # the path's rows of the same keys and values, over the tree
    rows = dkv.gather(1, path.cuda()[:, :, None, None, None].expand_as(dkv))
    sv.cache_append(cache, dt, dl, rows[:, :, 0], rows[:, :, 1], num_new=taken.cuda())
    dl += taken.cuda()
    host = kv.gather(1, path[:, :, None, None, None].expand_as(kv))
    cr.append(pool, table, before, host[:, :, 0], host[:, :, 1], taken)
    lengths += taken
    for b in range(3):  # what lies there now is the path, to half a step of the block's codes
        for side in range(2):
            got, _ = pool.tokens(side, table[b], 0, int(lengths[b]))
            want = host[b, : int(taken[b]), side, 0].double()
            step = pool.scale[side, table[b].long(), 0].max() * (2.0 ** -6 if code == "e4m3" else 2.0 ** -14)
            assert ((got[before[b]:] - want).abs() <= want.abs() * (2.0 ** -4 if code == "e4m3" else 2.0 ** -3) + step).all()
    q2, kv2 = torch.randn(3, 2, heads, dim, generator=g).to(torch.bfloat16), kv[:, 5:7]
    sv.cache_append(cache, dt, dl, dkv[:, 5:7, 0], dkv[:, 5:7, 1])
    cr.append(pool, table, lengths, kv2[:, :, 0], kv2[:, :, 1])
    out, lse = sv.cache_attend(q2.cuda(), cache, dt, dl + 2)
    check_attend(cr.attend(pool, table, lengths + 2, q2, dim ** -0.5), out, lse)
