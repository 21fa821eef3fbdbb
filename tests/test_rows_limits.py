"""Sizes that 32 bits do not hold, and those at the limits, through the binding of 8-bit rows (no GPU needed).

The tensors are of the meta device, which has no memory behind it; nothing here reads any."""
import pytest
import torch

import speculative_decoding_verification_45_gb300 as sv
from speculative_decoding_verification_45_gb300 import rows

BF16, E4, E8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu
MANY, WIDE = (1 << 32) + 5, (1 << 32) + 16


class Reached(Exception):
    pass


class Nothing:
    """In place of the calls in C: nothing is as usual."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture(autouse=True)
def checks_alone(monkeypatch):
    """Tensors say that they live on the current device, none is made, and the library is not called."""

    def reached():
        raise Reached

    monkeypatch.setattr(rows, "_quick", Nothing())
    monkeypatch.setattr(rows, "_current", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(rows, "_new", lambda shape, dtype, stream: meta(*shape, dtype=dtype))
    monkeypatch.setattr(rows._native, "load", reached)


def meta(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="meta")


def coded(rows, dim, weight=False):
    return sv.Coded(meta(rows, dim, dtype=E4), meta(-(-rows // 128) if weight else rows, -(-dim // 128), dtype=E8))


CALLS = [
    lambda rows, dim: sv.rows_quantise(meta(rows, dim)),
    lambda rows, dim: sv.rows_quantise(meta(1, dim).expand(rows, dim)),
    lambda rows, dim: sv.rows_quantise(meta(1, rows, dim)),
    lambda rows, dim: sv.rows_quantise(meta(rows, dim), out=coded(rows, dim)),
    lambda rows, dim: sv.weight_quantise(meta(rows, dim)),
    lambda rows, dim: sv.rows_norm(meta(rows, dim)),
    lambda rows, dim: sv.rows_norm(meta(rows, dim), meta(dim), meta(rows, dim)),
    lambda rows, dim: sv.rows_gate(meta(rows, dim), meta(rows, dim)),
    lambda rows, dim: sv.rows_product(coded(rows, dim), coded(4, dim, True)),
    lambda rows, dim: sv.rows_product(coded(4, dim), coded(rows, dim, True)),
    lambda rows, dim: sv.rows_product(coded(4, dim), coded(rows, dim, True), out=meta(4, rows)),
]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("rows,dim", [(MANY, 16), ((1 << 30) + 1, 16), (1, WIDE), (1, 131088)])
def test_past_the_limits(call, rows, dim):
    with pytest.raises(ValueError, match="at most"):
        call(rows, dim)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("rows,dim", [(1 << 30, 16), (1, 131072)])
def test_at_the_limits(call, rows, dim):
    with pytest.raises(Reached):
        call(rows, dim)
