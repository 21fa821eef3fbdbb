"""The weights of the example's cached tokens: those that the accepted tokens' queries gave them."""
import pytest
import torch

from tests.test_gpu_cache_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def decoder(example, **kw):  # noqa: F811
    """One whose text is far from certain, so that many drafts are rejected."""
    d = example.Decoder(batch=3, vocab=16, room=400, **kw)
    d.embed *= 0.05
    d.wq *= 20
    d.wkv *= 20
    return d


def snapshot(cache):
    return [x.view(torch.uint8).clone().view(x.dtype) if x.element_size() == 1 else x.clone() for x in cache]


def replay(d, asked, rows, weights, bound):
    """Adds what the first `rows` queries of each sequence give, in float64, and how far 32 bits may be off."""
    q, cache, table, lengths, num_new = asked
    k, _, k_scale, _, positions = snapshot(cache) if not isinstance(cache, list) else cache
    block, group = k.shape[2], q.shape[2] // k.shape[1]
    for b in range(len(lengths)):
        n, m = int(lengths[b]), int(num_new[b])
        j = torch.arange(n, device=q.device)
        page, row = table[b, j // block].long(), j % block
        for h in range(q.shape[2]):
            keys = k[page, h // group, row].double() * k_scale[page, h // group].double()[:, None]
            pos = positions[page, h // group, row].double()
            for i in range(int(rows[b])):
                at = n - m + i
                qq, kk = q[b, i, h].double(), keys[: at + 1]
                bias = float(d.slopes[h]) * (pos[at] - pos[: at + 1]).abs()
                x = kk @ qq / 8 - bias
                err = 2.0 ** -17 / 8 * (float(qq.abs().max()) * kk.abs().sum(1) + kk.abs() @ qq.abs()) \
                    + 2.0 ** -20 * (1 + bias + x.abs())
                p = x.softmax(0)
                weights[page[: at + 1], h // group, row[: at + 1]] += p
                bound[page[: at + 1], h // group, row[: at + 1]] += p * (1.5 * err + 1.5 * (p * err).sum() + 2.0 ** -20)


def test_weights_are_the_accepted_queries(example, monkeypatch):  # noqa: F811
    d = decoder(example, limit=300)
    asked = []
    plain = example.sv.cache_attend

    def attend(q, cache, table, lengths, num_new=None, **form):
        asked.append((q.clone(), snapshot(cache), table.clone(), lengths.clone(), num_new.clone()))
        return plain(q, cache, table, lengths, num_new=num_new, **form)

    monkeypatch.setattr(example.sv, "cache_attend", attend)
    want, bound = torch.zeros_like(d.weights, dtype=torch.float64), torch.zeros_like(d.weights, dtype=torch.float64)
    rejected = 0
    for _ in range(20):
        accepted = d.step()[1]
        rejected += int((asked[-1][4] - 1 - accepted).sum())
        replay(d, asked.pop(), accepted + 1, want, bound)
    assert rejected > 10 and d.evictions == 0 and int(d.status) == 0
    assert ((d.weights.double() - want).abs() <= bound + 2.0 ** -20 * want).all()


def test_slots_behind_the_cached_tokens_hold_no_weight(example):  # noqa: F811
    d = decoder(example, limit=96, keep=48, recent=16)
    for _ in range(80):
        d.step()
        w = d.weights[d.table.long()].transpose(1, 2).reshape(3, d.weights.shape[1], -1)
        behind = torch.arange(w.shape[2], device=w.device) >= d.lengths[:, None]
        assert (w.masked_select(behind[:, None]) == 0).all() and (d.weights[d.other.long()] == 0).all()
    assert d.evictions > 0
