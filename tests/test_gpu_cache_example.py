"""The example that runs the cache's operators together with drafting and verification."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_45_gb300 import _native, cache_example

    _native.build()
    return cache_example


def test_rounds_with_evictions(example):
    runs = []
    for _ in range(2):
        d = example.Decoder(batch=3, limit=96, keep=48, recent=16, room=400)
        rounds = [d.step() for _ in range(70)]
        assert int(d.status) == 0 and d.evictions > 0
        assert int(d.lengths.max()) <= 96 and int(d.text_len.min()) >= 2 + 70
        assert int(d.text.min()) >= 0 and int(d.text.max()) < 512
        assert torch.isfinite(d.weights).all()
        runs.append((d.text.clone(), d.lengths.clone(), torch.stack([r[1] for r in rounds])))
    for x, y in zip(*runs):
        assert torch.equal(x, y)


def test_the_first_forward_is_attention_over_what_was_appended(example):
    """Logits of the cached forward against the same layer in float64 with the rounded keys and values."""
    d = example.Decoder(batch=2, limit=64, keep=32, recent=8)
    n, gen = 20, torch.Generator().manual_seed(1)
    tokens = torch.randint(0, 512, (2, n), generator=gen).int().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(2, n).contiguous()
    logits = d.forward(tokens, torch.full((2,), n, dtype=torch.int32, device="cuda"), pos).double()
    x = d.embed[tokens.long()]
    q = (x @ d.wq).view(2, n, d.heads, d.dim).double()
    for b in range(2):
        pages = d.table[b, : -(-n // 16)].long()
        k, v = ((c[pages].double() * s[pages].double()[..., None, None]).transpose(0, 1).reshape(d.kv_heads, -1, d.dim)[:, :n]
                for c, s in ((d.cache.k, d.cache.k_scale), (d.cache.v, d.cache.v_scale)))
        group = d.heads // d.kv_heads
        s = torch.einsum("ihd,hjd->hij", q[b], k.repeat_interleave(group, 0)) / 8
        i = torch.arange(n, device="cuda")
        s = s - d.slopes.double()[:, None, None] * (i[:, None] - i).abs()
        s = s.masked_fill(i[None, :] > i[:, None], -torch.inf)
        out = torch.einsum("hij,hjd->ihd", s.softmax(-1), v.repeat_interleave(group, 0)).reshape(n, -1)
        want = (x[b].double() + out) @ d.embed.double().t()
        # out is rounded to bf16, and so is the sum with x; the product over 512 of them, and logits in bf16
        scale = want.abs().mean()
        assert ((logits[b] - want).abs().max() / scale) < 0.1
