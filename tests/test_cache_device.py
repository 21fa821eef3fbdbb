"""The cache's calls on a device that is not the current one are refused before anything is launched."""
import pytest
import torch

from speculative_decoding_verification_45_gb300 import cache


def test_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        cache._on_current(torch.device("cuda", 0))
    cache._on_current(torch.device("cuda", 1))


@pytest.mark.gpu
def test_every_call_asks(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as sv

    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    c = sv.KVCache(k, k.clone(), torch.ones(4, 2, device="cuda"), torch.ones(4, 2, device="cuda"))
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, q = torch.zeros(1, 1, 2, 64, device="cuda"), torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse, weights = torch.zeros(1, 1, 2, device="cuda"), torch.zeros(4, 2, 16, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: sv.cache_append(c, table, lengths, new, new), lambda: sv.cache_attend(q, c, table, lengths),
                 lambda: sv.cache_weigh(q, c, table, lengths, lse, weights),
                 lambda: sv.cache_evict(c, table, lengths, weights, 16, 4, table)):
        with pytest.raises(ValueError, match="current device"):
            call()
