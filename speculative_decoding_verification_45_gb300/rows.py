"""8-bit rows, and their product with 8-bit weights: Python binding of spec_rows_*.

    w = weight_quantise(weight)                       # once; [outputs, width] bf16 or fp32
    x, stream = rows_norm(delta, factor, residual=stream)   # residual added, normalised, in 8 bits
    logits = rows_product(x, w)                       # bf16 or fp32: a projection, or what verify reads

Codes have one power-of-two scale for each 128 elements of a row (activations) or
each 128 x 128 block (weights).  Every call checks its tensors, enqueues one kernel
on the current stream (or ``stream``) and returns; include/spec_verify.h states the
operations, layouts and error behaviour.  All tensors are CUDA tensors on the
current device; a tensor of rows may have any leading dimensions that lie at one
stride.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import _native
from .cache import _CODES, _fail, _new, _status, _stream

SCALE = torch.float8_e8m0fnu
BLOCK = 128
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


def _rows(t, name):
    """Rows, width and row stride of a tensor whose leading dimensions lie at one stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have a row dimension")
    dim = shape[-1]
    if t.is_contiguous():
        return (t.numel() // dim if dim else 0), dim, dim
    stride = t.stride()
    if stride[-1] != 1 and dim > 1:
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
    return rows, dim, dim if step is None else step


def _input(t, name, shape, device, dtypes=_FLOATS):
    """Address, row stride and type code of rows that a kernel reads."""
    code = dtypes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _, dim, step = _rows(t, name)
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, found {t.device}")
    at = t.data_ptr()
    if at & 15 or step * t.element_size() & 15:
        raise ValueError(f"{name}: rows must begin at multiples of 16 bytes, got a stride of {step} elements at {at:#x}")
    return at, step, code


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    device, current = t.device, torch.cuda.current_device()
    if device.index != current:
        raise ValueError(f"{name} lives on {device}, but the current device is cuda:{current}: call under "
                         f"torch.cuda.device({device.index})")
    return device


def _made(t, name, dtype, shape, device, stream):
    """An output that the caller gave (dense), or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != torch.Size(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a dense {tuple(shape)} tensor on {device}, got {tuple(t.shape)} on {t.device}")
    return t


def _coded_out(out, shape, device, code, stream, weight=False):
    """The Coded that a call writes, and its spec_coded."""
    dim = shape[-1]
    if dim < 16 or dim % 16:
        raise ValueError(f"the last dimension must be a multiple of 16, got {dim}")
    form = _CODES.get(code)
    if form is None:
        raise TypeError(f"code must be torch.float8_e4m3fn or torch.float8_e5m2, got {code}")
    blocks = -(-dim // BLOCK)
    above = (-(-shape[0] // BLOCK),) if weight else shape[:-1]
    codes, scale = (None, None) if out is None else out
    codes = _made(codes, "out.codes", code, shape, device, stream)
    scale = _made(scale, "out.scale", SCALE, (*above, blocks), device, stream)
    c = _native.Coded(codes.data_ptr(), scale.data_ptr(), dim, blocks, codes.numel() // dim, dim, form)
    return Coded(codes, scale), c


def rows_quantise(x, code=torch.float8_e4m3fn, out=None, stream=None):
    """Rows in 8 bits, a scale for each 128 elements (spec_rows_quantise).

    x: [..., dim] bfloat16 or float32, rows at one stride of a multiple of 16
    bytes.  Returns Coded(codes [..., dim], scale [..., ceil(dim / 128)]); ``out``:
    such a Coded to write into.
    """
    device = _device(x, "x")
    at, step, dtype = _input(x, "x", x.shape, device)
    out, c = _coded_out(out, x.shape, device, code, stream)
    rc = _native.load().spec_rows_quantise(at, step, dtype, ctypes.byref(c), 1, _stream(stream, device))
    if rc:
        _fail(rc, "spec_rows_quantise")
    return out


def weight_quantise(weight, code=torch.float8_e4m3fn, out=None, stream=None):
    """A weight [outputs, width] in 8 bits, a scale for each 128 x 128 block (spec_rows_quantise).

    Returns Coded(codes [outputs, width], scale [ceil(outputs / 128), ceil(width /
    128)]), which rows_product takes; done once, when weights are loaded.
    """
    if weight.dim() != 2:
        raise ValueError("weight must be an [outputs, width] tensor")
    device = _device(weight, "weight")
    at, step, dtype = _input(weight, "weight", weight.shape, device)
    out, c = _coded_out(out, weight.shape, device, code, stream, weight=True)
    rc = _native.load().spec_rows_quantise(at, step, dtype, ctypes.byref(c), BLOCK, _stream(stream, device))
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
    device = _device(x, "x")
    shape = x.shape
    at, step, dtype = _input(x, "x", shape, device)
    if not eps >= 2.0 ** -126 or eps == math.inf:
        raise ValueError(f"eps must be positive and finite, got {eps}")
    out, c = _coded_out(out, shape, device, code, stream)
    w_at, w_type = None, 0
    if weight is not None:
        if weight.shape != shape[-1:] or not weight.is_contiguous():
            raise ValueError(f"weight: expected a dense ({shape[-1]},) tensor, got {tuple(weight.shape)}")
        w_at, _, w_type = _input(weight, "weight", weight.shape, device)
    r_at = s_at = None
    r_step = s_step = r_type = 0
    if residual is not None:
        r_at, r_step, r_type = _input(residual, "residual", shape, device)
        if out_sum is None:
            out_sum = _new(shape, residual.dtype, device, stream)
        elif out_sum.dtype != residual.dtype:
            raise TypeError(f"out_sum: expected {residual.dtype}, got {out_sum.dtype}")
        s_at, s_step, _ = _input(out_sum, "out_sum", shape, device)
        if s_step < shape[-1]:
            raise ValueError("out_sum: rows must not overlap")
    elif out_sum is not None:
        raise ValueError("out_sum needs a residual")
    rc = _native.load().spec_rows_norm(at, step, dtype, r_at, r_step, r_type, w_at, w_type, eps, s_at, s_step,
                                       ctypes.byref(c), _stream(stream, device))
    if rc:
        _fail(rc, "spec_rows_norm")
    return out, out_sum


def rows_gate(gate, up, act="silu", code=torch.float8_e4m3fn, out=None, stream=None):
    """act(gate) * up in 8 bits (spec_rows_gate), as the second product of a feed-forward layer reads it.

    gate, up: [..., dim] bfloat16 or float32 (one type), each with its own row
    stride, so halves of one product's output need no copy.  ``act``: "silu" or
    "gelu_tanh".
    """
    device = _device(gate, "gate")
    kind = _ACTS.get(act)
    if kind is None:
        raise ValueError(f"act must be 'silu' or 'gelu_tanh', got {act!r}")
    g_at, g_step, dtype = _input(gate, "gate", gate.shape, device)
    u_at, u_step, u_type = _input(up, "up", gate.shape, device)
    if u_type != dtype:
        raise TypeError(f"up: expected {gate.dtype}, got {up.dtype}")
    out, c = _coded_out(out, gate.shape, device, code, stream)
    rc = _native.load().spec_rows_gate(g_at, g_step, u_at, u_step, dtype, kind, ctypes.byref(c), _stream(stream, device))
    if rc:
        _fail(rc, "spec_rows_gate")
    return out


def _coded_in(coded, name, device, weight):
    """The spec_coded of codes and scales that a product reads."""
    codes, scale = coded
    at, step, form = _input(codes, f"{name}.codes", codes.shape, device, _CODES)
    rows, dim, _ = _rows(codes, f"{name}.codes")
    if weight and codes.dim() != 2:
        raise ValueError(f"{name}.codes must be an [outputs, width] tensor")
    if dim < 16 or dim % 16:
        raise ValueError(f"{name}.codes: the last dimension must be a multiple of 16, got {dim}")
    blocks = -(-dim // BLOCK)
    above = (-(-rows // BLOCK),) if weight else codes.shape[:-1]
    if scale.dtype != SCALE:
        raise TypeError(f"{name}.scale: expected {SCALE}, got {scale.dtype}")
    if scale.shape != torch.Size((*above, blocks)) or scale.device != device:
        raise ValueError(f"{name}.scale: expected shape {(*above, blocks)} on {device}, got {tuple(scale.shape)} on "
                         f"{scale.device}")
    _, _, scale_step = _rows(scale, f"{name}.scale")
    if rows > 1 and step < dim or scale.numel() > blocks and scale_step < blocks:
        raise ValueError(f"{name}: rows must not overlap")
    return _native.Coded(at, scale.data_ptr(), max(step, dim), max(scale_step, blocks), rows, dim, form)


def rows_product(rows, weight, dtype=torch.bfloat16, out=None, status=None, stream=None):
    """rows times the transposed weight (spec_rows_product): a projection, or logits.

    rows    Coded [..., width], a scale for each row (rows_norm, rows_gate, rows_quantise)
    weight  Coded [outputs, width], a scale for each 128 x 128 (weight_quantise)
    dtype   of the result [..., outputs]: torch.bfloat16 or torch.float32; sums are 32-bit
    out     to write into, rows at any one stride (then ``dtype`` is its type)
    """
    device = _device(rows[0], "rows.codes")
    r = _coded_in(rows, "rows", device, False)
    w = _coded_in(weight, "weight", device, True)
    if r.dim != w.dim:
        raise ValueError(f"rows are {r.dim} wide, weight {w.dim}")
    shape = (*rows[0].shape[:-1], w.rows)
    if out is None:
        if dtype not in _FLOATS:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        out = _new(shape, dtype, device, stream)
        step = w.rows
    else:
        if out.dtype not in _FLOATS:
            raise TypeError(f"out: expected torch.bfloat16 or torch.float32, got {out.dtype}")
        if out.shape != torch.Size(shape) or out.device != device:
            raise ValueError(f"out: expected shape {shape} on {device}, got {tuple(out.shape)} on {out.device}")
        _, _, step = _rows(out, "out")
        if r.rows > 1 and step < w.rows:
            raise ValueError("out: rows must not overlap")
        step = max(step, w.rows)
    rc = _native.load().spec_rows_product(ctypes.byref(r), ctypes.byref(w), out.data_ptr(), step, _FLOATS[out.dtype],
                                          _status(status, device), _stream(stream, device))
    if rc:
        _fail(rc, "spec_rows_product")
    return out
