"""lse from another attention, heads first or sliced: weights as from a dense one."""
import pytest
import torch

from tests.test_gpu_cache import Case, dev, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 2)])
@pytest.mark.parametrize("on_a_stream", [False, True])
def test_lse_of_any_strides(sv, heads, kv_heads, on_a_stream):  # noqa: F811
    case = Case([300, 77], 3, heads=heads, kv_heads=kv_heads, seed=81)
    cache, f = case.pool.to(sv), {k: dev(v) for k, v in case.form.items()}
    q, table, lengths = case.q.cuda(), case.table.cuda(), case.lengths.cuda()
    _, lse = sv.cache_attend(q, cache, table, lengths, **f)
    want = sv.cache_weigh(q, cache, table, lengths, lse, torch.zeros(case.pool.codes.shape[1:4], device="cuda"), **f)
    wide = torch.full((2, 3, heads, 2), 5.0, device="cuda")
    wide[..., 1] = lse
    for other in (lse.transpose(1, 2).contiguous().transpose(1, 2), wide[..., 1]):
        assert not other.is_contiguous()
        w = torch.zeros_like(want)
        stream = torch.cuda.Stream() if on_a_stream else None
        if stream:
            stream.wait_stream(torch.cuda.current_stream())
        sv.cache_weigh(q, cache, table, lengths, other, w, stream=stream, **f)
        torch.cuda.synchronize()
        assert torch.equal(w, want)
    with pytest.raises(ValueError, match="lse: expected shape"):
        sv.cache_weigh(q, cache, table, lengths, lse.transpose(1, 2), want, **f)
