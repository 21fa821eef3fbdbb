"""What the 8-bit cache's calls refuse, on the host: the binding's checks of
tensors and the library's checks of sizes, before anything is launched (no GPU
needed)."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_45_gb300 as sv
from speculative_decoding_verification_45_gb300 import _native, cache

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    _native.build()
    return _native.load()


def make(**over):
    c = _native.Cache(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, table_stride=8, batch=2,
                      max_blocks=8, num_pages=16, kv_heads=2, block=16, dim=64, code=0)
    c.k_stride[:] = [2048, 1024, 64]
    c.v_stride[:] = [2048, 1024, 64]
    for name, value in over.items():
        if name.endswith("_stride") and isinstance(value, list):
            getattr(c, name)[:] = value
        else:
            setattr(c, name, value)
    return c


BAD_CACHE = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=FAKE + 8), 1), (dict(v=FAKE + 1), 1), (dict(k_scale=0), 1),
    (dict(v_scale=FAKE + 2), 1), (dict(positions=FAKE + 4), 1), (dict(block_table=0), 1), (dict(table_stride=7), 1),
    (dict(batch=-1), 1), (dict(max_blocks=0), 1), (dict(num_pages=0), 1), (dict(kv_heads=0), 1), (dict(block=24), 2),
    (dict(dim=96), 2), (dict(code=2), 2), (dict(k_stride=[2048, 1024, 72]), 1), (dict(v_stride=[0, 1024, 64]), 1),
    (dict(k_stride=[1 << 41, 1024, 64]), 1), (dict(max_blocks=1 << 28, table_stride=1 << 28), 1),
    (dict(max_blocks=(1 << 26) + 1, table_stride=1 << 28), 1),
]
# Never dereferenced: every case below fails validation, or has an empty batch or no new token.
three = (ctypes.c_int64 * 3)(256, 128, 64)


def form(**over):
    return ctypes.byref(_native.CacheForm(**{"scale": 0.125, **over}))


def append(lib, c, **o):
    a = dict(lengths=FAKE, k=FAKE, v=FAKE, n=4, dtype=1, num_new=None, positions=None, status=None)
    a.update(o)
    return lib.spec_cache_append(ctypes.byref(c), a["lengths"], a["k"], a["v"], three, three, a["n"], a["dtype"],
                                 a["num_new"], a["positions"], a["status"], None)


def attend(lib, c, **o):
    a = dict(lengths=FAKE, q=FAKE, n=4, heads=4, form=form(), out=FAKE, lse=FAKE, work=FAKE, size=1 << 40, status=None,
             stride=three)
    a.update(o)
    return lib.spec_cache_attend(ctypes.byref(c), a["lengths"], a["q"], a["stride"], a["n"], a["heads"], a["form"],
                                 a["out"], a["lse"], a["work"], a["size"], a["status"], None)


def weigh(lib, c, **o):
    a = dict(lengths=FAKE, q=FAKE, n=4, heads=4, form=form(), lse=FAKE, weights=FAKE, work=FAKE, size=1 << 40)
    a.update(o)
    return lib.spec_cache_weigh(ctypes.byref(c), a["lengths"], a["q"], three, a["n"], a["heads"], a["form"], a["lse"],
                                a["weights"], a["work"], a["size"], None, None)


def evict(lib, c, **o):
    a = dict(lengths=FAKE, weights=FAKE, keep=40, recent=8, table=FAKE, stride=3, out=FAKE, index=FAKE)
    a.update(o)
    return lib.spec_cache_evict(ctypes.byref(c), a["lengths"], a["weights"], a["keep"], a["recent"], a["table"],
                                a["stride"], a["out"], a["index"], None, None)


@pytest.mark.parametrize("call", [append, attend, weigh, evict])
@pytest.mark.parametrize("over,code", BAD_CACHE)
def test_cache_description(lib, call, over, code):
    assert call(lib, make(**over)) == code


@pytest.mark.parametrize("call", [append, attend, weigh, evict])
def test_empty_batch_is_no_work(lib, call):
    assert call(lib, make(batch=0)) == 0


@pytest.mark.parametrize("over,code", [
    (dict(lengths=0), 1), (dict(k=0), 1), (dict(v=FAKE + 1), 1), (dict(n=-1), 1), (dict(dtype=3), 2),
    (dict(dtype=0, k=FAKE + 2), 1), (dict(num_new=FAKE + 1), 1), (dict(positions=FAKE + 2), 1), (dict(status=FAKE + 3), 1),
    (dict(n=0), 0),
])
def test_append(lib, over, code):
    assert append(lib, make(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(lengths=0), 1), (dict(q=0), 1), (dict(q=FAKE + 8), 1), (dict(n=-1), 1), (dict(heads=0), 1), (dict(heads=3), 1),
    (dict(form=None), 1), (dict(form=form(window=-1)), 1), (dict(form=form(softcap=-1.0)), 1),
    (dict(form=form(scale=float("nan"))), 1), (dict(form=form(softcap=float("inf"))), 1),
    (dict(form=form(parent=FAKE), n=257), 1), (dict(form=form(slopes=FAKE + 1)), 1), (dict(form=form(prefix=FAKE + 2)), 1),
    (dict(n=1 << 29, heads=4), 2), (dict(n=0), 0),
])
def test_attend_and_weigh(lib, over, code):
    assert attend(lib, make(), **over) == code
    assert weigh(lib, make(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(out=0), 1), (dict(out=FAKE + 8), 1), (dict(lse=0), 1), (dict(lse=FAKE + 2), 1), (dict(work=FAKE + 8), 1),
    (dict(size=-1), 1), (dict(stride=(ctypes.c_int64 * 3)(256, 128, 60)), 1),
])
def test_attend_only(lib, over, code):
    assert attend(lib, make(), **over) == code


def test_weigh_only(lib):
    assert weigh(lib, make(), lse=0) == 1 and weigh(lib, make(), weights=FAKE + 2) == 1
    assert weigh(lib, make(), work=0) == 1 and weigh(lib, make(), work=FAKE + 8) == 1


@pytest.mark.parametrize("over,code", [
    (dict(lengths=0), 1), (dict(weights=0), 1), (dict(keep=0), 1), (dict(recent=-1), 1), (dict(recent=41), 1),
    (dict(table=0), 1), (dict(stride=2), 1), (dict(out=0), 1), (dict(index=0), 1),
])
def test_evict(lib, over, code):
    assert evict(lib, make(), **over) == code


def test_workspace_size(lib):
    got = ctypes.c_int64(-1)
    assert lib.spec_cache_attend_workspace(ctypes.byref(make()), 4, 4, None) == 1
    assert lib.spec_cache_attend_workspace(ctypes.byref(make()), 4, 3, ctypes.byref(got)) == 1
    assert lib.spec_cache_attend_workspace(ctypes.byref(make(dim=32)), 4, 4, ctypes.byref(got)) == 2


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def host(block=16, dim=64, code=torch.float8_e4m3fn):
    k = torch.zeros(4, 2, block, dim, dtype=torch.uint8).view(code)
    return sv.KVCache(k, k.clone(), torch.ones(4, 2), torch.ones(4, 2)), torch.zeros(1, 2, dtype=torch.int32), \
        torch.zeros(1, dtype=torch.int32)


def test_host_tensors_are_refused():
    c, table, lengths = host()
    with pytest.raises(ValueError, match="CUDA"):
        sv.cache_append(c, table, lengths, torch.zeros(1, 1, 2, 64), torch.zeros(1, 1, 2, 64))


def test_codes_must_be_8_bit_floats():
    c, table, lengths = host()
    with pytest.raises(TypeError, match="float8"):
        sv.cache_attend(None, c._replace(k=c.k.float()), table, lengths)
    with pytest.raises(TypeError, match="float8"):
        sv.cache_attend(None, c._replace(v=c.v.view(torch.float8_e5m2)), table, lengths)


def test_the_cache_has_four_dimensions():
    c, table, lengths = host()
    with pytest.raises(ValueError, match="num_pages"):
        sv.cache_attend(None, c._replace(k=c.k[0]), table, lengths)


def test_strides():
    assert cache._strides(torch.zeros(2, 5, 3, 64), "x", 16) == (960, 192, 64)
    assert cache._strides(torch.zeros(1, 3, 1, 24)[:, :1], "x", 16) == (16, 16, 16)
    with pytest.raises(ValueError, match="multiples of 16"):
        cache._strides(torch.zeros(2, 2, 3, 24), "x", 16)
    with pytest.raises(ValueError, match="dense"):
        cache._strides(torch.zeros(2, 2, 16, 32).transpose(2, 3), "x", 16)


@pytest.mark.parametrize("t,exc,msg", [
    (torch.zeros(3, dtype=torch.int64), TypeError, "expected torch.int32"), (torch.zeros(2, dtype=torch.int32), ValueError, "shape"),
    (torch.zeros(6, dtype=torch.int32)[::2], ValueError, "contiguous"),
])
def test_small_arrays(t, exc, msg):
    with pytest.raises(exc, match=msg):
        cache._check(t, "x", torch.int32, (3,), torch.device("cpu"))
    with pytest.raises(ValueError, match="must live on"):
        cache._check(torch.zeros(3, dtype=torch.int32), "x", torch.int32, (3,), torch.device("cuda", 0))


@pytest.mark.parametrize("over,exc,msg", [
    (dict(q=torch.zeros(1, 3, 64)), ValueError, "q: expected shape"),
    (dict(q=torch.zeros(1, 3, 3, 64)), ValueError, "multiple of 2"),
    (dict(q=torch.zeros(1, 3, 4, 64)), TypeError, "bfloat16"),
    (dict(q=torch.zeros(1, 300, 4, 64, dtype=torch.bfloat16), parent=torch.zeros(1, 300)), ValueError, "at most 256"),
    (dict(window=2 ** 31), ValueError, "below 2"), (dict(window=2 ** 32 + 5), ValueError, "below 2"),
    (dict(window=-1), ValueError, "negative"), (dict(softcap=-2.0), ValueError, "negative"),
    (dict(slopes=torch.zeros(2)), ValueError, "slopes"), (dict(prefix=torch.zeros(1)), TypeError, "prefix"),
    (dict(num_new=torch.zeros(2, dtype=torch.int32)), ValueError, "num_new"),
])
def test_forms(over, exc, msg):
    a = dict(q=torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16), num_new=None, scale=None, softcap=0.0, slopes=None,
             window=0, prefix=None, parent=None)
    a.update(over)
    with pytest.raises(exc, match=msg):
        cache._form(make(batch=1), torch.device("cpu"), **a)
