"""The example whose projections run in 8 bits: rounds of it, and its forward against the same layer in 64 bits."""
import pytest
import torch

from tests import rows_reference as ref
from tests.test_gpu_cache_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rounds(example):  # noqa: F811
    runs = []
    for _ in range(2):
        d = example.Decoder(batch=3, limit=96, keep=48, recent=16, room=400, eight_bit=True)
        rounds = [d.step() for _ in range(60)]
        assert int(d.status) == 0 and d.evictions > 0
        assert int(d.text_len.min()) >= 2 + 60 and int(d.text.min()) >= 0 and int(d.text.max()) < 512
        assert torch.isfinite(d.weights).all()
        runs.append((d.text.clone(), d.lengths.clone(), torch.stack([r[1] for r in rounds])))
    for x, y in zip(*runs):
        assert torch.equal(x, y)


def test_every_projection_is_the_product_of_its_codes(example, monkeypatch):  # noqa: F811
    """Each product of a forward against the definition of its own operands, in 64 bits."""
    d, seen, sv = example.Decoder(batch=2, limit=64, keep=32, recent=8, eight_bit=True), [], example.sv
    plain = sv.rows_product

    def product(rows, weight, **kw):
        out = plain(rows, weight, **kw)
        seen.append((rows, weight, out))
        return out

    monkeypatch.setattr(sv, "rows_product", product)
    n = 5
    tokens = torch.randint(0, 512, (2, n), generator=torch.Generator().manual_seed(1)).int().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(2, n).contiguous()
    logits = d.forward(tokens, torch.full((2,), n, dtype=torch.int32, device="cuda"), pos)
    assert logits.shape == (2, n, 512) and logits.dtype == torch.bfloat16
    assert [w.codes.shape[0] for _, w, _ in seen] == [768, 512, 4096, 512, 512]
    for rows, weight, out in seen:
        want, total = ref.product(rows, weight)
        off = (out.cpu().double().reshape(want.shape) - want).abs()
        width = weight.codes.shape[1]
        assert (off <= (width / 32 + 32) * 2.0 ** -23 * total + 2.0 ** -8 * want.abs()).all()


def test_the_command(example, capsys):  # noqa: F811
    example.main(["--rounds", "12", "--batch", "2", "--eight-bit"])
    assert "status 0" in capsys.readouterr().out
