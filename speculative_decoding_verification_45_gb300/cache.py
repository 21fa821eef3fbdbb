"""The target's key/value cache in 8 bits: Python binding of spec_cache_*.

    cache = KVCache(k, v, k_scale, v_scale)
    cache_append(cache, block_table, lengths, new_k, new_v)      # lengths: before
    lengths += n
    out, lse = cache_attend(q, cache, block_table, lengths)      # the n newest tokens ask
    cache_weigh(q, cache, block_table, lengths, lse, weights)    # weight each token received
    lengths, index = cache_evict(cache, block_table, lengths, weights, keep, recent, out_table)

Every call checks its tensors, enqueues its kernels on the current stream (or
``stream``) and returns; include/spec_verify.h states the operations, layouts and
error behaviour.  All tensors are CUDA tensors on the cache's device, which is
the current one.  ``status`` tells of bad lengths, pages and trees, and of a wait
in a kernel that ran out: without it such a call looks like any other.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple

import torch

from . import _native

_CODES = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
MAX_TREE_NODES = 256
_BLOCKS, _DIMS = (16, 32, 64, 128), (64, 128)
_Three = ctypes.c_int64 * 3


class KVCache(NamedTuple):
    """Blocks ("pages") of cached tokens.

    k, v              [num_pages, kv_heads, block, dim] float8_e4m3fn or
                      float8_e5m2, any strides that are multiples of 16 with
                      the last dimension dense (a [num_pages, block, kv_heads,
                      dim] pool is passed as its transpose(1, 2))
    k_scale, v_scale  [num_pages, kv_heads] float32: value = code * scale
    positions         [num_pages, kv_heads, block] int32 or None: each token's
                      position in its text for the bias by distance
    """

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    positions: torch.Tensor | None = None


def _fail(rc: int, where: str):
    from . import SpecVerifyError

    raise SpecVerifyError(rc, where)


def _check(t, name, dtype, shape, device):
    """The address of a tensor that is what it has to be."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, found {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _strides(t, name, multiple):
    """Strides of all but the last dimension, which has to be dense (sizes of one do not matter)."""
    a, b, c, last = t.stride()
    st = (a, b, c)
    if last == 1 and a and b and c and not (a | b | c) % multiple:
        return st
    if last != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    st = tuple(x if n > 1 else multiple for n, x in zip(t.shape[:-1], st))
    if any(x % multiple for x in st):
        raise ValueError(f"{name}: strides must be multiples of {multiple}, got {tuple(t.stride())}")
    return st


def _on_current(device):
    """The kernels are launched on the current device, where the cache has to be."""
    current = torch.cuda.current_device()
    if device.index != current:
        raise ValueError(f"cache.k lives on {device}, but the current device is cuda:{current}: call under "
                         f"torch.cuda.device({device.index})")


def _describe(cache, block_table, lengths):
    """The spec_cache of these tensors, checked; their device; the lengths' address."""
    k, v, k_scale, v_scale, positions = cache
    if k.dim() != 4:
        raise ValueError("cache.k must be a [num_pages, kv_heads, block, dim] tensor")
    code = _CODES.get(k.dtype)
    if code is None or v.dtype != k.dtype:
        raise TypeError(f"cache.k and cache.v must both be float8_e4m3fn or float8_e5m2, got {k.dtype} and {v.dtype}")
    if not k.is_cuda:
        raise ValueError("cache.k must be a CUDA tensor")
    dev, shape = k.device, k.shape
    _on_current(dev)
    if v.shape != shape or v.device != dev:
        raise ValueError(f"cache.v: expected shape {tuple(shape)} on {dev}, got {tuple(v.shape)} on {v.device}")
    pages, heads, block, dim = shape
    if block not in _BLOCKS or dim not in _DIMS:
        raise ValueError(f"cache: block must be 16, 32, 64 or 128 and dim 64 or 128, got {block} and {dim}")
    if block_table.dim() != 2:
        raise ValueError("block_table must be a [batch, blocks] tensor")
    batch, blocks = block_table.shape
    _native.fit("cache", pages, heads, batch, blocks)
    step, dense = block_table.stride()
    if block_table.dtype != torch.int32 or block_table.device != dev or (blocks > 1 and dense != 1):
        raise ValueError(f"block_table must be int32 on {dev} with dense rows")
    c = _native.Cache(
        k.data_ptr(), v.data_ptr(), _check(k_scale, "cache.k_scale", torch.float32, (pages, heads), dev),
        _check(v_scale, "cache.v_scale", torch.float32, (pages, heads), dev),
        None if positions is None else _check(positions, "cache.positions", torch.int32, (pages, heads, block), dev),
        block_table.data_ptr(),
        _strides(k, "cache.k", 16), _strides(v, "cache.v", 16), step if batch > 1 else blocks, batch,
        blocks, pages, heads, block, dim, code)
    return c, dev, _check(lengths, "lengths", torch.int32, (batch,), dev)


def _status(t, device):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.device != device or t.numel() < 1 or not t.is_contiguous():
        raise ValueError(f"status must be a contiguous int32 tensor on {device} with at least one element")
    return t.data_ptr()


def _stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream):
    """A new tensor whose block belongs to the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dense(t, stream):
    """The tensor, or a dense copy that the call's stream makes and uses."""
    if t.is_contiguous():
        return t
    if stream is None:
        return t.contiguous()
    with torch.cuda.stream(stream):
        return t.contiguous()


def _output(t, name, dtype, shape, device, stream):
    """An output that the caller gave, or a new one; and its address."""
    if t is not None:
        return t, _check(t, name, dtype, shape, device)
    t = _new(shape, dtype, device, stream)
    return t, t.data_ptr()


def cache_append(cache, block_table, lengths, k, v, num_new=None, positions=None, status=None, stream=None):
    """Write new tokens into the cache in 8 bits (spec_cache_append).

    k, v: [batch, n, kv_heads, dim] bfloat16 or float32, any strides with the
    last dimension dense (slices of a fused projection need no copy).  Token i <
    num_new[b] becomes cached token lengths[b] + i; ``lengths`` [batch] int32
    holds the tokens before the call and is not changed.  A block's scale is the
    smallest power of two that its values fit, and grows (its older codes moving
    with it) when new tokens need it.  ``num_new`` [batch] int32 or None (n
    each); ``positions`` [batch, n] int32 or None (the index), stored where the
    cache has positions.  ``status``: optional int32 CUDA tensor whose first
    element receives STATUS_* bits.
    """
    c, dev, len_ptr = _describe(cache, block_table, lengths)
    if k.dim() != 4 or k.shape[0] != c.batch or k.shape[2] != c.kv_heads or k.shape[3] != c.dim:
        raise ValueError(f"k: expected shape ({c.batch}, n, {c.kv_heads}, {c.dim}), got {tuple(k.shape)}")
    if k.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"k: expected bfloat16 or float32, got {k.dtype}")
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError(f"v: expected {tuple(k.shape)} {k.dtype}, got {tuple(v.shape)} {v.dtype}")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must live on {dev}")
    n = k.shape[1]
    _native.fit("k", n)
    new = None if num_new is None else _check(num_new, "num_new", torch.int32, (c.batch,), dev)
    pos = None if positions is None else _check(positions, "positions", torch.int32, (c.batch, n), dev)
    rc = _native.load().spec_cache_append(
        ctypes.byref(c), len_ptr, k.data_ptr(), v.data_ptr(), _Three(*_strides(k, "k", 1)), _Three(*_strides(v, "v", 1)),
        n, 1 if k.dtype == torch.bfloat16 else 0, new, pos, _status(status, dev), _stream(stream, dev))
    if rc:
        _fail(rc, "spec_cache_append")


def _form(c, dev, q, num_new, scale, softcap, slopes, window, prefix, parent):
    if q.dim() != 4 or q.shape[0] != c.batch or q.shape[3] != c.dim or q.shape[2] < 1 or q.shape[2] % c.kv_heads:
        raise ValueError(f"q: expected shape ({c.batch}, n, a multiple of {c.kv_heads}, {c.dim}), got {tuple(q.shape)}")
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q: expected torch.bfloat16, got {q.dtype}")
    if q.device != dev:
        raise ValueError(f"q must live on {dev}, found {q.device}")
    n, heads = q.shape[1], q.shape[2]
    _native.fit("q", n, heads)
    if parent is not None and n > MAX_TREE_NODES:
        raise ValueError(f"a candidate tree has at most {MAX_TREE_NODES} nodes, got {n}")
    if window < 0 or not 0 <= softcap < math.inf:
        raise ValueError("window and softcap must not be negative")
    if window >= 1 << 31:
        raise ValueError(f"window must be below 2^31 (0: none), got {window}")
    f = _native.CacheForm(
        1 / math.sqrt(c.dim) if scale is None else scale, softcap, window,
        None if slopes is None else _check(slopes, "slopes", torch.float32, (heads,), dev),
        None if prefix is None else _check(prefix, "prefix", torch.int32, (c.batch,), dev),
        None if parent is None else _check(parent, "parent", torch.int32, (c.batch, n), dev),
        None if num_new is None else _check(num_new, "num_new", torch.int32, (c.batch,), dev))
    return f, n, heads, _Three(*_strides(q, "q", 8))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(batch, kv_heads, block, dim, n, heads, device):
    """Bytes that spec_cache_attend_workspace asks for; they follow from these sizes and the device, which is current."""
    fake = 16  # an address for the check of the description; nothing is read
    c = _native.Cache(fake, fake, fake, fake, None, fake, (16,) * 3, (16,) * 3, 1, batch, 1, 1, kv_heads, block, dim, 0)
    need = ctypes.c_int64()
    rc = _native.load().spec_cache_attend_workspace(ctypes.byref(c), n, heads, ctypes.byref(need))
    if rc:
        _fail(rc, "spec_cache_attend_workspace")
    return need.value


def _workspace(c, n, heads, dev, stream):
    """A workspace for one call, and its size."""
    size = _workspace_bytes(c.batch, c.kv_heads, c.block, c.dim, n, heads, dev.index)
    return _new(size, torch.uint8, dev, stream), size


def cache_attend(q, cache, block_table, lengths, num_new=None, scale=None, softcap=0.0, slopes=None, window=0,
                 prefix=None, parent=None, out=None, lse=None, status=None, stream=None):
    """Attention of the newest tokens over the cache (spec_cache_attend).

    q: [batch, n, heads, dim] bfloat16; query i < num_new[b] (None: n) is cached
    token lengths[b] - num_new[b] + i, so ``lengths`` counts the new tokens too.
    Returns (out [batch, n, heads, dim] bfloat16, lse [batch, n, heads] float32).

    scale    factor of q.k, 1/sqrt(dim) when None
    softcap  scores become softcap * tanh(score / softcap) where it is > 0
    slopes   [heads] float32: score -= slope * |distance in position|
    window   > 0: a query sees the last ``window`` tokens up to its own
    prefix   [batch] int32: tokens before it are seen by every query
    parent   [batch, n] int32: the n queries are a candidate tree, as in
             tree_verify (node 0 the root); a node sees its ancestors.
             Before the next round the accepted path's rows are appended
             once more, at the length before the tree (out_path says which)

    Rows that see nothing, and rows i >= num_new[b], are zeros with lse -inf.

    Precision: scores, sums and lse in 32 bits; query elements to 2^-21 of the
    largest of their row or better; softmax weights to 2^-10 of themselves, but
    no finer than 2^-21 of the largest weight (times value scale) among their 128
    tokens.  With n * heads / kv_heads above 32, weights to 2^-8 of themselves, as
    in bf16, and no finer than 2^-17 of that.  spec_verify.h has it in full.
    """
    c, dev, len_ptr = _describe(cache, block_table, lengths)
    f, n, heads, stride = _form(c, dev, q, num_new, scale, softcap, slopes, window, prefix, parent)
    out, out_ptr = _output(out, "out", torch.bfloat16, (c.batch, n, heads, c.dim), dev, stream)
    lse, lse_ptr = _output(lse, "lse", torch.float32, (c.batch, n, heads), dev, stream)
    work, size = _workspace(c, n, heads, dev, stream)
    rc = _native.load().spec_cache_attend(ctypes.byref(c), len_ptr, q.data_ptr(), stride, n, heads, ctypes.byref(f), out_ptr,
                               lse_ptr, work.data_ptr(), size, _status(status, dev), _stream(stream, dev))
    if rc:
        _fail(rc, "spec_cache_attend")
    return out, lse


def cache_weigh(q, cache, block_table, lengths, lse, weights, num_new=None, scale=None, softcap=0.0, slopes=None,
                window=0, prefix=None, parent=None, status=None, stream=None):
    """Add the attention weight that each cached token received (spec_cache_weigh).

    ``lse`` is what cache_attend returned for the same q and form, or that of
    another attention with any strides (copied if it is not dense); ``weights``
    [num_pages, kv_heads, block] float32 grows by the sum over queries and query
    heads of exp(score - lse).  Returns ``weights``.  In a speculative round this
    comes after the accept test, with the accepted tokens only (``num_new`` their
    number, ``lengths`` to match, the same q and lse): weight given to a rejected
    token would pass to the next one in its slot, since nothing clears weights but
    the caller.
    """
    c, dev, len_ptr = _describe(cache, block_table, lengths)
    f, n, heads, stride = _form(c, dev, q, num_new, scale, softcap, slopes, window, prefix, parent)
    lse = _dense(lse, stream)
    lse_ptr = _check(lse, "lse", torch.float32, (c.batch, n, heads), dev)
    w_ptr = _check(weights, "weights", torch.float32, (c.num_pages, c.kv_heads, c.block), dev)
    work, size = _workspace(c, n, heads, dev, stream)
    rc = _native.load().spec_cache_weigh(ctypes.byref(c), len_ptr, q.data_ptr(), stride, n, heads, ctypes.byref(f), lse_ptr, w_ptr,
                              work.data_ptr(), size, _status(status, dev), _stream(stream, dev))
    if rc:
        _fail(rc, "spec_cache_weigh")
    return weights


def cache_evict(cache, block_table, lengths, weights, keep: int, recent: int, out_table, out_lengths=None,
                out_index=None, status=None, stream=None):
    """Keep the heaviest and the newest tokens (spec_cache_evict).

    Of each sequence and key/value head the ``recent`` newest tokens stay and,
    of the others, the ``keep - recent`` with the largest ``weights``.  They move
    in order, with their weights and positions, to the pages of ``out_table``
    [batch, >= ceil(keep / block)] int32, which no sequence may use yet; the
    old pages are free afterwards.  Returns (lengths [batch] int32, the kept
    indices [batch, kv_heads, keep] int32, -1 after the last); ``out_lengths``
    may be ``lengths`` itself.
    """
    c, dev, len_ptr = _describe(cache, block_table, lengths)
    if keep < 1 or not 0 <= recent <= keep:
        raise ValueError(f"keep must be at least 1 and recent in [0, keep], got {keep} and {recent}")
    _native.fit("keep", keep)
    blocks = -(-keep // c.block)
    if out_table.dim() != 2 or out_table.shape[0] != c.batch or out_table.shape[1] < blocks:
        raise ValueError(f"out_table: expected shape ({c.batch}, at least {blocks}), got {tuple(out_table.shape)}")
    if out_table.dtype != torch.int32 or out_table.device != dev or (out_table.shape[1] > 1 and out_table.stride(1) != 1):
        raise ValueError(f"out_table must be int32 on {dev} with dense rows")
    w_ptr = _check(weights, "weights", torch.float32, (c.num_pages, c.kv_heads, c.block), dev)
    out_lengths, l_ptr = _output(out_lengths, "out_lengths", torch.int32, (c.batch,), dev, stream)
    out_index, i_ptr = _output(out_index, "out_index", torch.int32, (c.batch, c.kv_heads, keep), dev, stream)
    rc = _native.load().spec_cache_evict(
        ctypes.byref(c), len_ptr, w_ptr, keep, recent, out_table.data_ptr(),
        out_table.stride(0) if c.batch > 1 else out_table.shape[1], l_ptr, i_ptr, _status(status, dev),
        _stream(stream, dev))
    if rc:
        _fail(rc, "spec_cache_evict")
    return out_lengths, out_index
