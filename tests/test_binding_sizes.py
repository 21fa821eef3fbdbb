"""Sizes that 32 bits do not hold, through the binding of the verification calls and the cache (no GPU needed).

The tensors are of the meta device, which has no memory behind it; nothing here reads any."""
import pytest
import torch

import speculative_decoding_verification_45_gb300 as sv
from speculative_decoding_verification_45_gb300 import _native, cache

MANY = (1 << 32) + 5
F32, I32, E4 = torch.float32, torch.int32, torch.float8_e4m3fn


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def checks_alone(monkeypatch):
    """Tensors say that they live on the current device, and the library is not called."""

    def reached():
        raise Reached

    monkeypatch.setattr(sv, "_device_of", lambda *t: torch.device("meta"))
    monkeypatch.setattr(sv, "_stream_handle", lambda *a: None)
    monkeypatch.setattr(cache, "_on_current", lambda device: None)
    monkeypatch.setattr(cache, "_workspace", lambda c, n, heads, dev, stream: (meta(1, dtype=torch.uint8), 1))
    monkeypatch.setattr(cache, "_stream", lambda stream, device: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(_native, "load", reached)


def meta(*shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="meta")


def verify(batch=2, gamma=3, vocab=64):
    return sv.verify(meta(batch, gamma + 1, vocab), meta(batch, gamma, vocab), meta(batch, gamma, dtype=I32), meta(batch, dtype=I32),
                     meta(batch, gamma + 1), meta(batch))


def tree(batch=2, nodes=4, vocab=64):
    return sv.tree_verify(meta(batch, nodes, vocab), meta(batch, nodes, dtype=I32), meta(batch, nodes, dtype=I32), meta(batch, dtype=I32),
                          meta(batch, nodes), meta(batch))


def sample(batch=2, vocab=64):
    return sv.sample(meta(batch, vocab), meta(batch), meta(batch))


def propose(batch=2, length=50, low=1, high=3, gamma=4):
    return sv.ngram_propose(meta(batch, length, dtype=I32), meta(batch, dtype=I32), low, high, gamma)


def parts(batch, blocks):
    pool = sv.KVCache(meta(8, 2, 16, 64, dtype=E4), meta(8, 2, 16, 64, dtype=E4), meta(8, 2), meta(8, 2))
    return pool, meta(batch, blocks, dtype=I32), meta(batch, dtype=I32)


def append(batch=2, blocks=4, n=3):
    return sv.cache_append(*parts(batch, blocks), meta(batch, n, 2, 64), meta(batch, n, 2, 64))


def attend(batch=2, blocks=4, n=3):
    return sv.cache_attend(meta(batch, n, 4, 64, dtype=torch.bfloat16), *parts(batch, blocks))


def evict(batch=2, blocks=4, keep=32, recent=4):
    return sv.cache_evict(*parts(batch, blocks), meta(8, 2, 16), keep, recent, meta(batch, -(-keep // 16), dtype=I32))


CALLS = [(verify, dict(batch=MANY)), (verify, dict(vocab=MANY)), (verify, dict(gamma=MANY)), (tree, dict(batch=MANY)),
         (tree, dict(nodes=MANY)), (tree, dict(vocab=MANY)), (sample, dict(batch=MANY)), (sample, dict(vocab=MANY)),
         (propose, dict(batch=MANY)), (propose, dict(low=MANY)), (propose, dict(high=MANY)), (propose, dict(gamma=MANY)),
         (append, dict(batch=MANY)), (append, dict(blocks=MANY)), (append, dict(n=MANY)), (attend, dict(batch=MANY)),
         (attend, dict(blocks=MANY)), (attend, dict(n=MANY)), (evict, dict(batch=MANY)), (evict, dict(keep=MANY))]


@pytest.mark.parametrize("call,sizes", CALLS)
def test_a_size_past_32_bits(call, sizes):
    with pytest.raises(ValueError, match="below 2"):
        call(**sizes)


@pytest.mark.parametrize("call", [verify, tree, sample, propose, append, attend, evict])
def test_others_reach_the_library(call):
    with pytest.raises(Reached):
        call()


@pytest.mark.parametrize("sizes", [(MANY, 4, 64), (2, MANY, 64), (2, 4, MANY)])
def test_launch_shape(sizes):
    with pytest.raises(ValueError, match="below 2"):
        sv.launch_shape(*sizes)
