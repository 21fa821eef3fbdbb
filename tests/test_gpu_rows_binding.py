"""The two ways of the binding of 8-bit rows, the calls in C and the checks in Python: one result, no reference lost."""
import gc
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
E4, E5, BF16, F32 = torch.float8_e4m3fn, torch.float8_e5m2, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as sv

    return sv


def flat(result):
    if result is None:
        return []
    if isinstance(result, torch.Tensor):
        return [result]
    return [t for r in result for t in flat(r)]


def calls(sv):
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    x, wide, f, three = rand(37, 288), rand(37, 704), rand(37, 288, dtype=F32), rand(5, 7, 1040)
    w, wf = rand(300, 288), rand(288, dtype=F32)
    part = wide[:, 96:384]
    a, b = sv.rows_quantise(x), sv.weight_quantise(w)
    wide_codes = sv.rows_quantise(rand(37, 1024))
    cut = sv.Coded(wide_codes.codes[:, 256:544], wide_codes.scale[:, 2:5])
    deep = sv.rows_quantise(three), sv.weight_quantise(rand(90, 1040))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    return [
        lambda: sv.rows_quantise(x), lambda: sv.rows_quantise(f, code=E5), lambda: sv.rows_quantise(three), lambda: sv.rows_quantise(x[3]),
        lambda: sv.rows_quantise(wide[:, :288]), lambda: sv.rows_quantise(x[:1].expand(9, 288)), lambda: sv.rows_quantise(x[::2]),
        lambda: sv.weight_quantise(w), lambda: sv.weight_quantise(wide[:, :288], code=E5),
        lambda: sv.rows_norm(x), lambda: sv.rows_norm(x, wf), lambda: sv.rows_norm(x, wf.to(BF16), f, eps=1e-3, code=E5),
        lambda: sv.rows_norm(three, None, three), lambda: sv.rows_norm(f, wf, wide[:, :288]),
        lambda: sv.rows_gate(x, x), lambda: sv.rows_gate(wide[:, :288], wide[:, 288:576], act="gelu_tanh"), lambda: sv.rows_gate(f, f, code=E5),
        lambda: sv.rows_product(a, b), lambda: sv.rows_product(a, b, dtype=F32), lambda: sv.rows_product(cut, b), lambda: sv.rows_product(*deep),
        lambda: sv.rows_product(a, b, status=status), lambda: sv.rows_product(sv.Coded(a.codes[4], a.scale[4]), b),
        lambda: sv.rows_product(tuple(a), tuple(b)),
    ], part


def test_one_result(sv, monkeypatch):
    from speculative_decoding_verification_45_gb300 import rows

    every, _ = calls(sv)
    used = []

    class Counted:
        def __getattr__(self, name):
            call = getattr(quick, name)

            def counted(*a):
                made = call(*a)
                used.append(made is not None)
                return made

            return counted

    class Nothing:
        def __getattr__(self, name):
            return lambda *a: None

    sv.rows_quantise(torch.zeros(1, 16, device="cuda"))
    quick = rows._quick
    for call in every:
        used.clear()
        monkeypatch.setattr(rows, "_quick", Counted())
        one = call()
        assert used == [True]
        monkeypatch.setattr(rows, "_quick", Nothing())
        two = call()
        monkeypatch.setattr(rows, "_quick", quick)
        assert type(one) is type(two)
        for p, q in zip(flat(one), flat(two), strict=True):
            assert p.shape == q.shape and p.dtype == q.dtype and p.stride() == q.stride()
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_what_is_not_as_usual_is_refused_by_the_checks(sv):
    x, a = torch.zeros(4, 32, device="cuda"), sv.rows_quantise(torch.zeros(4, 32, device="cuda"))
    b = sv.weight_quantise(torch.zeros(8, 32, device="cuda"))
    for call, exc in (
        (lambda: sv.rows_quantise(x.cpu()), ValueError), (lambda: sv.rows_quantise(x.half()), TypeError), (lambda: sv.rows_quantise(None), AttributeError),
        (lambda: sv.rows_quantise(x.t()), ValueError), (lambda: sv.rows_quantise(x[:, :24]), ValueError), (lambda: sv.rows_quantise(x[:, 1:17]), ValueError),
        (lambda: sv.rows_quantise(x, code=F32), TypeError), (lambda: sv.weight_quantise(x[None]), ValueError),
        (lambda: sv.rows_norm(x, eps=0.0), ValueError), (lambda: sv.rows_norm(x, x), ValueError), (lambda: sv.rows_norm(x, None, x[:2]), ValueError),
        (lambda: sv.rows_norm(torch.zeros(1, 32784, device="cuda")), sv.SpecVerifyError),
        (lambda: sv.rows_gate(x, x.bfloat16()), TypeError), (lambda: sv.rows_gate(x, x[:1]), ValueError), (lambda: sv.rows_gate(x, x, act="tanh"), ValueError),
        (lambda: sv.rows_product(b, b), ValueError), (lambda: sv.rows_product(a, a), ValueError), (lambda: sv.rows_product(a, b, dtype=torch.half), TypeError),
        (lambda: sv.rows_product(a, (b.codes.view(torch.uint8), b.scale)), TypeError), (lambda: sv.rows_product(a, (b.codes, b.scale.view(torch.uint8))), TypeError),
        (lambda: sv.rows_product(a, b, status=torch.zeros(1, device="cuda")), ValueError), (lambda: sv.rows_product(3, b), TypeError),
    ):
        with pytest.raises(exc):
            call()


def test_no_reference_is_kept(sv):
    every, _ = calls(sv)
    for call in every:
        call()
    torch.cuda.synchronize()
    gc.collect()
    held, objects = torch.cuda.memory_allocated(), len(gc.get_objects())
    counts = [sys.getrefcount(o) for o in (torch.float32, torch.bfloat16, E4, E5, torch.float8_e8m0fnu, sv.Coded, None)]
    for _ in range(200):
        for call in every:
            call()
    torch.cuda.synchronize()
    gc.collect()
    assert torch.cuda.memory_allocated() == held and len(gc.get_objects()) <= objects + 50
    after = [sys.getrefcount(o) for o in (torch.float32, torch.bfloat16, E4, E5, torch.float8_e8m0fnu, sv.Coded, None)]
    assert all(abs(p - q) < 100 for p, q in zip(counts, after))


def test_threads(sv):
    """Calls of several threads at once, each on a stream of its own."""
    every, _ = calls(sv)
    torch.cuda.synchronize()
    want = [flat(call()) for call in every]
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                for call, right in zip(every, want):
                    got = flat(call())
                    if not all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, right, strict=True)):
                        wrong.append(call)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
