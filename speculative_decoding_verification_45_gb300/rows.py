"""8-bit rows, and their product with 8-bit weights: Python binding of spec_rows_*.

    w = weight_quantise(weight)                       # once; [outputs, width] bf16 or fp32
    x, stream = rows_norm(delta, factor, residual=stream)   # residual added, normalised, in 8 bits
    logits = rows_product(x, w)                       # bf16 or fp32: a projection, or what verify reads

Codes have one power-of-two scale for each 128 elements of a row (activations) or
each 128 x 128 block (weights).  Every call checks its tensors, enqueues one kernel
on the current stream (or ``stream``) and returns; include/spec_verify.h states the
operations, layouts and error behaviour.  All tensors are CUDA tensors on the
current device; a tensor of rows may have any leading dimensions that lie at one
stride, up to 2^30 rows of up to 131,072 elements.  Results have no history:
tensors that require a gradient are read like others, and none flows back to them.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import _native
from .cache import _CODES, _fail, _status

SCALE = torch.float8_e8m0fnu
BLOCK = 128
MAX_WIDTH, MAX_ROWS = 1 << 17, 1 << 30  # SPEC_MAX_ROW, SPEC_MAX_CODED_ROWS
_Struct, _byref, _current = _native.Coded, ctypes.byref, torch._C._cuda_getDevice
_ACTS = {"silu": 0, "gelu_tanh": 1}
_FLOATS = {torch.float32: 0, torch.bfloat16: 1}


class Coded(NamedTuple):
    """A matrix in 8 bits.

    codes  [..., dim] float8_e4m3fn or float8_e5m2, dim a multiple of 16
    scale  [..., ceil(dim / 128)] float8_e8m0fnu, for each row (activations), or
           [ceil(rows / 128), ceil(dim / 128)] (weights): value = code * scale
    """

    codes: torch.Tensor
    scale: torch.Tensor


def _stream(stream, index):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


class _Unloaded:
    """Stands for the calls in C (csrc/rows/spec_rows_py.c) until the first of them: they do the usual case, and return None
    for anything else, which the checks below then tell of."""

    def __getattr__(self, name):
        global _quick
        lib, module = _native.load(), _native.load_extension()
        address = [ctypes.cast(getattr(lib, f"spec_rows_{x}"), ctypes.c_void_p).value for x in ("quantise", "norm", "gate", "product")]
        module.setup((torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2, SCALE, torch.int32), Coded, _empty,
                     torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream, tuple(address))
        _quick = module
        return getattr(module, name)


_quick = _Unloaded()

def _empty_strided(shape, stride, dtype):
    return torch.empty_strided(shape, stride, dtype=dtype, device="cuda")


# torch.empty costs 5 us a call beside launches here, and this form of it (the one that torch's compiled code calls) less
# than 1: for one token it is half of a call's time.  It is no public function: a torch without it gives the other.
try:
    _empty = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    _empty = _empty_strided


def _new(shape, dtype, stream):
    """A new tensor on the current device, whose block belongs to the stream that will write it."""
    shape = tuple(shape)
    if len(shape) == 2:
        stride = (shape[1], 1)
    else:
        stride, step = (), 1
        for x in reversed(shape):
            stride = (step, *stride)
            step *= x
    if stream is None:
        return _empty(shape, stride, dtype)
    with torch.cuda.stream(stream):
        return _empty(shape, stride, dtype)


def _step(t, name):
    """Row stride of a tensor whose leading dimensions lie at one stride."""
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    rows, step = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != step * rows:
            raise ValueError(f"{name}: rows must lie at one stride, got strides {tuple(stride)} of {tuple(shape)}")
        rows *= n
    return shape[-1] if step is None else step


def _index(t, name):
    """The current device's index, where the first tensor of a call lives."""
    index = t.get_device()
    if index < 0 or index != _current():
        _elsewhere(t, name, _current() if index >= 0 else index)
    return index


def _matrix(t, name, index, types):
    """(address, rows, width, row stride, type code) of a tensor of rows on device `index`."""
    kind = types.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in types)}, got {t.dtype}")
    if t.get_device() != index:
        _elsewhere(t, name, index)
    at, shape = t.data_ptr(), t.shape
    if not shape or not shape[-1]:
        raise ValueError(f"{name}: expected rows of some width, got shape {tuple(shape)}")
    dim = shape[-1]
    rows = t.numel() // dim
    if dim > MAX_WIDTH or rows > MAX_ROWS:  # the library's sizes have 32 bits, into which ctypes would cut these
        raise ValueError(f"{name}: at most {MAX_ROWS} rows of {MAX_WIDTH} elements, got {rows} of {dim}")
    step = dim if t.is_contiguous() else _step(t, name)
    if (at | step * t.itemsize) & 15:
        raise ValueError(f"{name}: rows must begin at multiples of 16 bytes, got a stride of {step} elements at {at:#x}")
    return at, rows, dim, step, kind


def _elsewhere(t, name, index):
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} lives on {t.device}, but the current device is cuda:{index}: call under "
                     f"torch.cuda.device({t.get_device()})")


def _made(t, name, dtype, shape, index):
    """The address of an output that the caller gave, dense."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        _elsewhere(t, name, index)
    if t.shape != torch.Size(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a dense {tuple(shape)} tensor, got {tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _coded_out(out, like, shape, rows, dim, code, stream, weight=False):
    """The Coded of `shape` that a call writes, beside `like`, and its spec_coded."""
    form = _CODES.get(code)
    if form is None:
        raise TypeError(f"code must be torch.float8_e4m3fn or torch.float8_e5m2, got {code}")
    if dim & 15:
        raise ValueError(f"the last dimension must be a multiple of 16, got {dim}")
    blocks = (dim + 127) // 128
    above = ((rows + 127) // 128, blocks) if weight else (*shape[:-1], blocks)
    if out is None:
        out = Coded(_new(shape, code, stream), _new(above, SCALE, stream))
        at, scale_at = out[0].data_ptr(), out[1].data_ptr()
    else:
        index = like.get_device()
        at, scale_at = _made(out[0], "out.codes", code, shape, index), _made(out[1], "out.scale", SCALE, above, index)
        if at & 15:
            raise ValueError(f"out.codes: must begin at a multiple of 16 bytes, got {at:#x}")
    return out, _byref(_Struct(at, scale_at, dim, blocks, rows, dim, form))


def rows_quantise(x, code=torch.float8_e4m3fn, out=None, stream=None):
    """Rows in 8 bits, a scale for each 128 elements (spec_rows_quantise).

    x: [..., dim] bfloat16 or float32, rows at one stride of a multiple of 16
    bytes.  Returns Coded(codes [..., dim], scale [..., ceil(dim / 128)]); ``out``:
    such a Coded to write into.
    """
    if out is None and stream is None:
        made = _quick.quantise(x, code, 1)
        if made is not None:
            return made
    index = _index(x, "x")
    at, rows, dim, step, dtype = _matrix(x, "x", index, _FLOATS)
    out, c = _coded_out(out, x, x.shape, rows, dim, code, stream)
    rc = _native.load().spec_rows_quantise(at, step, dtype, c, 1, _stream(stream, index))
    if rc:
        _fail(rc, "spec_rows_quantise")
    return out


def weight_quantise(weight, code=torch.float8_e4m3fn, out=None, stream=None):
    """A weight [outputs, width] in 8 bits, a scale for each 128 x 128 block (spec_rows_quantise).

    Returns Coded(codes [outputs, width], scale [ceil(outputs / 128), ceil(width /
    128)]), which rows_product takes; done once, when weights are loaded.
    """
    if out is None and stream is None:
        made = _quick.quantise(weight, code, BLOCK)
        if made is not None:
            return made
    if weight.dim() != 2:
        raise ValueError("weight must be an [outputs, width] tensor")
    index = _index(weight, "weight")
    at, rows, dim, step, dtype = _matrix(weight, "weight", index, _FLOATS)
    out, c = _coded_out(out, weight, weight.shape, rows, dim, code, stream, True)
    rc = _native.load().spec_rows_quantise(at, step, dtype, c, BLOCK, _stream(stream, index))
    if rc:
        _fail(rc, "spec_rows_quantise")
    return out


def rows_norm(x, weight=None, residual=None, eps=1e-6, code=torch.float8_e4m3fn, out=None, out_sum=None, stream=None):
    """Residual, root-mean-square norm, 8 bits (spec_rows_norm).

    h = x + residual; returns (Coded of h / sqrt(mean(h^2) + eps) * weight, h in the
    residual's type, or None without a residual).

    x, residual  [..., dim] bfloat16 or float32 each, dim <= 32768
    weight       [dim] bfloat16 or float32, or None (1)
    out, out_sum to write into; out_sum may be ``residual`` itself
    """
    if out is None and out_sum is None and stream is None:
        made = _quick.norm(x, weight, residual, eps, code)
        if made is not None:
            return made
    index = _index(x, "x")
    at, rows, dim, step, dtype = _matrix(x, "x", index, _FLOATS)
    shape = x.shape
    if not eps >= 2.0 ** -126 or eps == math.inf:
        raise ValueError(f"eps must be positive and finite, got {eps}")
    w_at, w_type = None, 0
    if weight is not None:
        w_at, one, w_dim, _, w_type = _matrix(weight, "weight", index, _FLOATS)
        if one != 1 or w_dim != dim or weight.dim() != 1:
            raise ValueError(f"weight: expected shape ({dim},), got {tuple(weight.shape)}")
    r_at = s_at = None
    r_step = s_step = r_type = 0
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual: expected shape {tuple(shape)}, got {tuple(residual.shape)}")
        r_at, _, _, r_step, r_type = _matrix(residual, "residual", index, _FLOATS)
        if out_sum is None:
            out_sum = _new(shape, residual.dtype, stream)
            s_at, s_step = out_sum.data_ptr(), dim
        else:
            if out_sum.dtype != residual.dtype:
                raise TypeError(f"out_sum: expected {residual.dtype}, got {out_sum.dtype}")
            if out_sum.shape != shape:
                raise ValueError(f"out_sum: expected shape {tuple(shape)}, got {tuple(out_sum.shape)}")
            s_at, _, _, s_step, _ = _matrix(out_sum, "out_sum", index, _FLOATS)
            if s_step < dim:
                raise ValueError("out_sum: rows must not overlap")
    elif out_sum is not None:
        raise ValueError("out_sum needs a residual")
    out, c = _coded_out(out, x, shape, rows, dim, code, stream)
    rc = _native.load().spec_rows_norm(at, step, dtype, r_at, r_step, r_type, w_at, w_type, eps, s_at, s_step, c,
                                       _stream(stream, index))
    if rc:
        _fail(rc, "spec_rows_norm")
    return out, out_sum


def rows_gate(gate, up, act="silu", code=torch.float8_e4m3fn, out=None, stream=None):
    """act(gate) * up in 8 bits (spec_rows_gate), as the second product of a feed-forward layer reads it.

    gate, up: [..., dim] bfloat16 or float32 (one type), each with its own row
    stride, so halves of one product's output need no copy.  ``act``: "silu" or
    "gelu_tanh".
    """
    kind = _ACTS.get(act)
    if out is None and stream is None and kind is not None:
        made = _quick.gate(gate, up, kind, code)
        if made is not None:
            return made
    index = _index(gate, "gate")
    if kind is None:
        raise ValueError(f"act must be 'silu' or 'gelu_tanh', got {act!r}")
    g_at, rows, dim, g_step, dtype = _matrix(gate, "gate", index, _FLOATS)
    shape = gate.shape
    if up.shape != shape:
        raise ValueError(f"up: expected shape {tuple(shape)}, got {tuple(up.shape)}")
    u_at, _, _, u_step, u_type = _matrix(up, "up", index, _FLOATS)
    if u_type != dtype:
        raise TypeError(f"up: expected {gate.dtype}, got {up.dtype}")
    out, c = _coded_out(out, gate, shape, rows, dim, code, stream)
    rc = _native.load().spec_rows_gate(g_at, g_step, u_at, u_step, dtype, kind, c, _stream(stream, index))
    if rc:
        _fail(rc, "spec_rows_gate")
    return out


_ROWS, _WEIGHT = ("rows.codes", "rows.scale"), ("weight.codes", "weight.scale")


def _coded_in(coded, names, index, weight):
    """The spec_coded of codes and scales that a product reads; its rows and width."""
    codes, scale = coded
    at, rows, dim, step, form = _matrix(codes, names[0], index, _CODES)
    if dim & 15:
        raise ValueError(f"{names[0]}: the last dimension must be a multiple of 16, got {dim}")
    if weight and codes.dim() != 2:
        raise ValueError(f"{names[0]} must be an [outputs, width] tensor")
    blocks = (dim + 127) // 128
    if scale.dtype is not SCALE:
        raise TypeError(f"{names[1]}: expected {SCALE}, got {scale.dtype}")
    if scale.get_device() != index:
        _elsewhere(scale, names[1], index)
    above = ((rows + 127) // 128, blocks) if weight else (*codes.shape[:-1], blocks)
    if scale.shape != above:
        raise ValueError(f"{names[1]}: expected shape {above}, got {tuple(scale.shape)}")
    scale_step = blocks if scale.is_contiguous() else _step(scale, names[1])
    if step < dim or scale_step < blocks:
        if rows > 1 and (step < dim or scale.numel() > blocks):
            raise ValueError(f"{names[0]}: rows must not overlap")
        step, scale_step = max(step, dim), max(scale_step, blocks)
    return _byref(_Struct(at, scale.data_ptr(), step, scale_step, rows, dim, form)), rows, dim


def rows_product(rows, weight, dtype=torch.bfloat16, out=None, status=None, stream=None):
    """rows times the transposed weight (spec_rows_product): a projection, or logits.

    rows    Coded [..., width], a scale for each row (rows_norm, rows_gate, rows_quantise)
    weight  Coded [outputs, width], a scale for each 128 x 128 (weight_quantise)
    dtype   of the result [..., outputs]: torch.bfloat16 or torch.float32; sums are 32-bit
    out     to write into, rows at any one stride (then ``dtype`` is its type)
    status  int32 CUDA tensor whose first element receives STATUS_INTERNAL where a wait in
            the kernel ran out: without it such a call, whose result is not valid, looks
            like any other
    """
    if out is None and stream is None:
        made = _quick.product(rows, weight, dtype, status)
        if made is not None:
            return made
    index = _index(rows[0], "rows.codes")
    r, count, dim = _coded_in(rows, _ROWS, index, False)
    w, outs, width = _coded_in(weight, _WEIGHT, index, True)
    if dim != width:
        raise ValueError(f"rows are {dim} wide, weight {width}")
    shape = (*rows[0].shape[:-1], outs)
    if out is None:
        kind = _FLOATS.get(dtype)
        if kind is None:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        out = _new(shape, dtype, stream)
        step = outs
    else:
        kind = _FLOATS.get(out.dtype)
        if kind is None:
            raise TypeError(f"out: expected torch.bfloat16 or torch.float32, got {out.dtype}")
        if out.get_device() != index:
            _elsewhere(out, "out", index)
        if out.shape != shape:
            raise ValueError(f"out: expected shape {shape}, got {tuple(out.shape)}")
        step = outs if out.is_contiguous() else _step(out, "out")
        if count > 1 and step < outs:
            raise ValueError("out: rows must not overlap")
        step = max(step, outs)
    if status is not None:
        status = _status(status, torch.device("cuda", index))
    rc = _native.load().spec_rows_product(r, w, out.data_ptr(), step, kind, status, _stream(stream, index))
    if rc:
        _fail(rc, "spec_rows_product")
    return out
