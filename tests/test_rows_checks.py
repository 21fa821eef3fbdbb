"""What the calls of 8-bit rows refuse, on the host: the binding's checks of tensors and the
library's checks of sizes, before anything is launched (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_45_gb300 as sv
from speculative_decoding_verification_45_gb300 import _native, rows

FAKE = 0x10000
E8 = torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def lib():
    _native.build()
    return _native.load()


def coded(**over):
    c = _native.Coded(codes=FAKE, scale=FAKE, stride=256, scale_stride=2, rows=4, dim=256, code=0)
    for name, value in over.items():
        setattr(c, name, value)
    return ctypes.byref(c)


# Never dereferenced: every case below fails validation or has no rows.
def quantise(lib, c, x=FAKE, stride=256, dtype=1, block_rows=1):
    return lib.spec_rows_quantise(x, stride, dtype, c, block_rows, None)


def norm(lib, c, **o):
    a = dict(x=FAKE, xs=256, xt=1, r=FAKE, rs=256, rt=1, w=FAKE, wt=0, eps=1e-6, s=FAKE, ss=256)
    a.update(o)
    return lib.spec_rows_norm(a["x"], a["xs"], a["xt"], a["r"], a["rs"], a["rt"], a["w"], a["wt"], a["eps"], a["s"], a["ss"],
                              c, None)


def gate(lib, c, g=FAKE, gs=256, u=FAKE, us=256, dtype=1, act=0):
    return lib.spec_rows_gate(g, gs, u, us, dtype, act, c, None)


def product(lib, c, w=None, out=FAKE, stride=4, dtype=1, status=None):
    return lib.spec_rows_product(c, w if w is not None else coded(), out, stride, dtype, status, None)


BAD = [
    (dict(codes=0), 1), (dict(codes=FAKE + 8), 1), (dict(scale=0), 1), (dict(stride=240), 1), (dict(stride=264), 1),
    (dict(stride=1 << 40), 1), (dict(scale_stride=1), 1), (dict(rows=-1), 1), (dict(rows=(1 << 30) + 1), 1), (dict(dim=0), 1),
    (dict(dim=8), 1), (dict(dim=250), 1), (dict(dim=131088, stride=131088, scale_stride=1025), 2), (dict(code=2), 2),
]


@pytest.mark.parametrize("call", [quantise, norm, gate, product])
@pytest.mark.parametrize("over,code", BAD)
def test_coded(lib, call, over, code):
    assert call(lib, coded(**over)) == code


@pytest.mark.parametrize("call", [quantise, norm, gate, product])
def test_no_rows_is_no_work(lib, call):
    assert call(lib, coded(rows=0, codes=0, scale=0)) == 0


@pytest.mark.parametrize("over,code", [
    (dict(x=0), 1), (dict(x=FAKE + 8), 1), (dict(stride=252), 1), (dict(dtype=0, stride=254), 1), (dict(stride=-256), 1),
    (dict(dtype=2), 2), (dict(block_rows=64), 2), (dict(block_rows=0), 2),
])
def test_quantise(lib, over, code):
    assert quantise(lib, coded(), **over) == code


def test_a_weight_of_too_many_rows(lib):
    assert quantise(lib, coded(rows=1 << 23), block_rows=128) == 2


@pytest.mark.parametrize("over,code", [
    (dict(x=0), 1), (dict(xs=252), 1), (dict(xt=5), 2), (dict(r=FAKE + 2), 1), (dict(rs=4), 1), (dict(rt=5), 2),
    (dict(w=FAKE + 8), 1), (dict(wt=5), 2), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(eps=1e-40), 1), (dict(s=0), 1), (dict(r=0), 1), (dict(s=FAKE + 8), 1), (dict(ss=248), 1),
])
def test_norm(lib, over, code):
    assert norm(lib, coded(), **over) == code


def test_a_row_too_long_to_normalise(lib):
    assert norm(lib, coded(dim=32784, stride=32784, scale_stride=257)) == 2


@pytest.mark.parametrize("over,code", [(dict(g=0), 1), (dict(u=FAKE + 4), 1), (dict(gs=4), 1), (dict(us=-8), 1), (dict(dtype=3), 2),
                                       (dict(act=2), 2)])
def test_gate(lib, over, code):
    assert gate(lib, coded(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(w=coded(dim=128)), 1), (dict(w=coded(code=3)), 2), (dict(w=coded(codes=FAKE + 1)), 1), (dict(out=0), 1),
    (dict(out=FAKE + 1), 1), (dict(dtype=0, out=FAKE + 2), 1), (dict(stride=3), 1), (dict(dtype=2), 2), (dict(status=FAKE + 2), 1),
    (dict(w=coded(rows=0, codes=0, scale=0)), 0),
])
def test_product(lib, over, code):
    assert product(lib, coded(), **over) == code


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
class Nothing:
    """In place of the calls in C: nothing is as usual."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture(autouse=True)
def checks_alone(monkeypatch):
    monkeypatch.setattr(rows, "_quick", Nothing())


@pytest.fixture
def on_device(monkeypatch):
    """Host tensors that say they live on the current device, of which the checks before a launch see no more."""
    monkeypatch.setattr(rows, "_current", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)


def here(*shape, dtype=torch.bfloat16):
    size = math.prod(shape) * 4 + 64
    base = torch.zeros(size, dtype=torch.uint8)
    base = base[-base.data_ptr() % 16:]
    return base[: math.prod(shape) * dtype.itemsize].view(dtype).view(*shape)


def codes(*shape):
    return here(*shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def scales(*shape):
    return here(*shape, dtype=torch.uint8).view(E8)


def test_host_tensors_are_refused(monkeypatch):
    monkeypatch.setattr(rows, "_current", lambda: 0)
    x = torch.zeros(2, 32)
    w = sv.Coded(x.to(torch.float8_e4m3fn), torch.zeros(1, 1, dtype=torch.uint8).view(E8))
    for call in (lambda: sv.rows_quantise(x), lambda: sv.weight_quantise(x), lambda: sv.rows_norm(x), lambda: sv.rows_gate(x, x),
                 lambda: sv.rows_product(w, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_another_device_is_refused(on_device, monkeypatch):
    monkeypatch.setattr(rows, "_current", lambda: 1)
    for call in (lambda: sv.rows_quantise(here(2, 32)), lambda: sv.rows_norm(here(2, 32)), lambda: sv.rows_gate(here(2, 32), here(2, 32)),
                 lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1)))):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()


@pytest.mark.parametrize("call,exc,msg", [
    (lambda: sv.rows_quantise(here(2, 32, dtype=torch.float16)), TypeError, "x: expected"),
    (lambda: sv.rows_quantise(here(2, 24)), ValueError, "multiple of 16"),
    (lambda: sv.rows_quantise(here(2, 20)), ValueError, "multiples of 16 bytes"),
    (lambda: sv.rows_quantise(here(2, 0)), ValueError, "some width"),
    (lambda: sv.rows_quantise(here(64, 32).t()), ValueError, "dense"),
    (lambda: sv.rows_quantise(here(4, 6, 32)[:, :4]), ValueError, "one stride"),
    (lambda: sv.rows_quantise(here(4, 40)[:, :32]), None, None),
    (lambda: sv.rows_quantise(here(4, 36)[:, :32]), ValueError, "multiples of 16 bytes"),
    (lambda: sv.rows_quantise(here(4, 64)[:, 4:36]), ValueError, "multiples of 16 bytes"),
    (lambda: sv.rows_quantise(here(2, 32), code=torch.float8_e8m0fnu), TypeError, "float8_e4m3fn"),
    (lambda: sv.rows_quantise(here(2, 32), out=sv.Coded(codes(2, 32), here(2, 1, dtype=torch.uint8))), TypeError, "out.scale"),
    (lambda: sv.rows_quantise(here(2, 32), out=sv.Coded(codes(3, 32), scales(2, 1))), ValueError, "out.codes"),
    (lambda: sv.weight_quantise(here(2, 2, 32)), ValueError, "outputs, width"),
    (lambda: sv.weight_quantise(here(200, 32), out=sv.Coded(codes(200, 32), scales(200, 1))), ValueError, "out.scale"),
    (lambda: sv.rows_norm(here(2, 32), eps=0.0), ValueError, "eps"),
    (lambda: sv.rows_norm(here(2, 32), eps=float("nan")), ValueError, "eps"),
    (lambda: sv.rows_norm(here(2, 32), here(48)), ValueError, "weight"),
    (lambda: sv.rows_norm(here(2, 32), here(1, 32)), ValueError, "weight"),
    (lambda: sv.rows_norm(here(2, 32), None, here(3, 32)), ValueError, "residual"),
    (lambda: sv.rows_norm(here(2, 32), out_sum=here(2, 32)), ValueError, "needs a residual"),
    (lambda: sv.rows_norm(here(2, 32), None, here(2, 32), out_sum=here(2, 32, dtype=torch.float32)), TypeError, "out_sum"),
    (lambda: sv.rows_norm(here(2, 32), None, here(2, 32), out_sum=here(1, 32).expand(2, 32)), ValueError, "overlap"),
    (lambda: sv.rows_gate(here(2, 32), here(2, 48)), ValueError, "up"),
    (lambda: sv.rows_gate(here(2, 32), here(2, 32, dtype=torch.float32)), TypeError, "up"),
    (lambda: sv.rows_gate(here(2, 32), here(2, 32), act="relu"), ValueError, "act"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(4, 48), scales(1, 1))), ValueError, "wide"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(1, 1)), sv.Coded(codes(4, 32), scales(1, 1))), ValueError, "rows.scale"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(200, 32), scales(200, 1))), ValueError, "weight.scale"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), here(2, 1, dtype=torch.uint8)), sv.Coded(codes(4, 32), scales(1, 1))), TypeError, "scale"),
    (lambda: sv.rows_product(sv.Coded(here(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1))), TypeError, "rows.codes"),
    (lambda: sv.rows_product(sv.Coded(codes(1, 32).expand(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1))), ValueError, "overlap"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(2, 2, 32), scales(1, 1))), ValueError, "weight.codes"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1)), dtype=torch.float16), TypeError, "dtype"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1)), out=here(2, 5)), ValueError, "out"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1)), out=here(1, 4).expand(2, 4)), ValueError, "overlap"),
    (lambda: sv.rows_product(sv.Coded(codes(2, 32), scales(2, 1)), sv.Coded(codes(4, 32), scales(1, 1)), out=here(2, 4),
                             status=torch.zeros(1, dtype=torch.int64)), ValueError, "status"),
])
def test_refusals(on_device, monkeypatch, call, exc, msg):
    if exc is None:  # passes every check: it would be launched
        class Reached(Exception):
            pass

        def reached():
            raise Reached

        monkeypatch.setattr(rows, "_new", lambda shape, dtype, stream: codes(*shape) if dtype is torch.float8_e4m3fn else scales(*shape))
        monkeypatch.setattr(rows._native, "load", reached)
        exc = Reached
    with pytest.raises(exc, match=msg):
        call()


def test_steps():
    x = torch.zeros(3, 5, 40)
    assert rows._step(x[..., :32], "x") == 40 and rows._step(x[:, :1, :32], "x") == 200 and rows._step(x[:1, :1, :32], "x") == 32
    assert rows._step(torch.zeros(1, 32).expand(4, 32), "x") == 0
    with pytest.raises(ValueError, match="one stride"):
        rows._step(x[:, :3, :32], "x")
