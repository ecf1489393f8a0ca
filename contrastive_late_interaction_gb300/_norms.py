"""The binding's part between a tower's blocks: layer norm, dropout and the residual join (include/cli.h).

As `_binding`, of which this is a part: argument marshalling only, with its errors, its streams and its way of making
results.  Every matrix is [rows, width], rows any distance apart, and lies on the same device as the first; a call on a
device that is not the current one runs there.

A dropout mask comes from `rate`, `seed` (int64 [2] on the device: the seed and the step, read when the kernels run) and
`site`, the call's place among those of one step; it is drawn again by the backward, from the same three.
"""

from __future__ import annotations

import struct

import torch

from . import _binding as _b
from ._binding import (CLI_INVALID_ARGUMENT, CLI_SHAPE_MISMATCH, CLI_UNSUPPORTED, DTYPES, InvalidArgumentError,
                       ShapeMismatchError, UnsupportedError)

# The argument structs packed in one call each, as the token states' are.
_pack_norm = struct.Struct("@2i2Q8Q4Qf4x3Q")
_pack_dropout = struct.Struct("@i4x2Q8QdQI4xQ")
_pack_join = struct.Struct("@2i2Q16QdQI4x4Qf4x3Q")
assert _pack_norm.size == _b.ctypes.sizeof(_b.LayerNormArgs)
assert _pack_dropout.size == _b.ctypes.sizeof(_b.DropoutArgs)
assert _pack_join.size == _b.ctypes.sizeof(_b.DropoutLayerNormArgs)
_VERBS = {v: _b._fast(v) for v in ("layer_norm", "layer_norm_backward", "dropout", "dropout_backward",
                                   "dropout_layer_norm", "dropout_layer_norm_backward")}
_NONE = 0, 0
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(verb, lead, pack, *words):
    """The verb on `lead`'s device and that device's current stream, or raises."""
    device = lead.get_device()
    if device >= 0 and device != _current_device():
        with torch.cuda.device(device):
            rc = _VERBS[verb](pack(*words, _b._raw_stream(lead)))
    else:
        rc = _VERBS[verb](pack(*words, _b._raw_stream(lead)))
    if rc:
        _b.raise_for(rc, verb)


def _first(t, name):
    """The shape of the call's first matrix [rows, width]."""
    if not t.is_cuda:
        _b._check_cuda(t, name)
    if t.dim() != 2:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be [rows, width], not {list(t.shape)}")
    if t.dtype not in DTYPES:
        raise UnsupportedError(CLI_UNSUPPORTED, f"{name}: {t.dtype}")
    return t.shape


def _matrix(t, name, shape, dtype, lead):
    """(data, row stride) of a matrix of `shape` whose rows' elements are adjacent, on lead's device."""
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda:
        _b._check_cuda(t, name, dtype)
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be {list(shape)}, not {list(t.shape)}")
    _same_device(t, name, lead)
    row, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name}: the elements of a row must be adjacent")
    return t.data_ptr(), row


def _same_device(t, name, lead):
    if t.get_device() != lead.get_device():
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, f"{name} is on another device than the call's first matrix")


def _vector(t, name, n, lead):
    if t is None:
        return 0
    at = _b._vector(t, name, n, torch.float32)
    _same_device(t, name, lead)
    return at


def _result(out, name, shape, dtype, lead):
    """The caller's output `name`, or a new packed one, and its (data, row stride)."""
    t = out.get(name) if out else None
    if t is not None:
        return t, _matrix(t, "out " + name, shape, dtype, lead)
    t = torch.empty(shape, dtype=dtype, device=lead.device)
    return t, (t.data_ptr(), shape[1])


def _gradient(out, name, of, lead):
    """The gradient of a vector: the caller's or a new one, and its address; None where the vector is."""
    if of is None:
        return None, 0
    t = out.get(name) if out else None
    if t is not None:
        return t, _vector(t, "out " + name, of.numel(), lead)
    t = torch.empty_like(of)
    return t, t.data_ptr()


def _other(dtype, lead, what):
    """A type that goes with lead's stream type: the same, or a 16-bit one beside fp32."""
    if dtype is None:
        return lead.dtype
    if dtype not in DTYPES or (dtype is not lead.dtype and lead.dtype is not torch.float32):
        raise UnsupportedError(CLI_UNSUPPORTED, f"{what}: {dtype} beside {lead.dtype}")
    return dtype


def _mask(rate, seed, site, lead):
    """The mask's words in a struct."""
    if not 0 <= site <= 65535:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, "site must be 0 .. 65535")
    if seed is None:
        return rate, 0, site   # refused by the library unless the rate is 0
    at = _b._vector(seed, "seed", 2, torch.int64)
    _same_device(seed, "seed", lead)
    return rate, at, site


def layer_norm_backward_workspace_bytes(rows, width):
    return int(_b.lib.layer_norm_backward_workspace_bytes(rows, width))


def _workspace(workspace, wanted, rows, width, lead):
    """(tensor to keep until the call is made, address, bytes)"""
    if workspace is not None:
        lent = _b._lent(workspace)
        _same_device(workspace, "workspace", lead)
        return workspace, *lent
    if not wanted:
        return None, 0, 0
    need = _b.lib.layer_norm_backward_workspace_bytes(rows, width)
    workspace = _b._ws(need, lead.device)
    return workspace, workspace.data_ptr(), need


def layer_norm(x, gain=None, bias=None, epsilon=1e-5, dtype=None, out=None, stream=None):
    """Normalises each row of `x` [rows, width]: gain * (x - mean) / sqrt(variance + epsilon) + bias, with fp32 [width]
    gains (None: ones) and biases (None: zeros).  bf16, fp16 or fp32; `dtype` is the output's type, 16-bit beside an
    fp32 `x` if wanted.  Returns dict(output); out['output'] may be `x` itself."""
    if stream is not None:
        return _b._on(stream, layer_norm, locals())
    shape = _first(x, "x")
    to = _other(dtype, x, "dtype")
    given = _matrix(x, "x", shape, x.dtype, x)
    g, b = _vector(gain, "gain", shape[1], x), _vector(bias, "bias", shape[1], x)
    y, made = _result(out, "output", shape, to, x)
    _call("layer_norm", x, _pack_norm.pack, DTYPES[x.dtype], DTYPES[to], *shape, *given, *made, *_NONE, *_NONE, g, b, 0, 0,
          epsilon, 0, 0)
    return {"output": y}


def layer_norm_backward(x, d_output, gain=None, bias=None, epsilon=1e-5, out=None, workspace=None, stream=None):
    """The gradients of layer_norm for `x`, its gain and its bias, given that of its output.  A gain's or bias's
    gradient (fp32 [width]) is None where that is.  Returns dict(d_x, d_gain, d_bias); out['d_x'] may be `x` or, of one
    type with it, `d_output`."""
    if stream is not None:
        return _b._on(stream, layer_norm_backward, locals())
    shape = _first(x, "x")
    _first(d_output, "d_output")
    to = _other(d_output.dtype, x, "d_output")
    given, dy = _matrix(x, "x", shape, x.dtype, x), _matrix(d_output, "d_output", shape, to, x)
    g = _vector(gain, "gain", shape[1], x)
    _vector(bias, "bias", shape[1], x)
    dx, made = _result(out, "d_x", shape, x.dtype, x)
    d_gain, dg = _gradient(out, "d_gain", gain, x)
    d_bias, db = _gradient(out, "d_bias", bias, x)
    workspace, *lent = _workspace(workspace, dg or db, *shape, x)
    _call("layer_norm_backward", x, _pack_norm.pack, DTYPES[x.dtype], DTYPES[to], *shape, *given, *_NONE, *dy, *made, g, 0,
          dg, db, epsilon, *lent)
    return {"d_x": dx, "d_gain": d_gain, "d_bias": d_bias}


def dropout(x, rate, seed, site=0, out=None, stream=None):
    """Drops elements of `x` [rows, width] with probability `rate` (below 1) and scales the others by its complement's
    inverse.  bf16, fp16 or fp32.  A dropped element is 0 whatever `x` holds there.  Returns dict(output); out['output']
    may be `x` itself."""
    if stream is not None:
        return _b._on(stream, dropout, locals())
    shape = _first(x, "x")
    given = _matrix(x, "x", shape, x.dtype, x)
    mask = _mask(rate, seed, site, x)
    y, made = _result(out, "output", shape, x.dtype, x)
    _call("dropout", x, _pack_dropout.pack, DTYPES[x.dtype], *shape, *given, *made, *_NONE, *_NONE, *mask)
    return {"output": y}


def dropout_backward(d_output, rate, seed, site=0, out=None, stream=None):
    """The gradient of dropout for its input: `d_output` through the same mask.  Returns dict(d_x)."""
    if stream is not None:
        return _b._on(stream, dropout_backward, locals())
    shape = _first(d_output, "d_output")
    given = _matrix(d_output, "d_output", shape, d_output.dtype, d_output)
    mask = _mask(rate, seed, site, d_output)
    dx, made = _result(out, "d_x", shape, d_output.dtype, d_output)
    _call("dropout_backward", d_output, _pack_dropout.pack, DTYPES[d_output.dtype], *shape, *_NONE, *_NONE, *given, *made,
          *mask)
    return {"d_x": dx}


def dropout_layer_norm(x, residual, rate, seed, site=0, gain=None, bias=None, epsilon=1e-5, want_sum=True, out=None,
                       stream=None):
    """A branch's output `x` joins the residual stream, and the norm of that, in one pass: sum = residual + dropout(x),
    output = layer_norm(sum) (of the sum before it is rounded).  `residual` and the sum are of x's type or fp32; the rest
    as in dropout and layer_norm.  Returns dict(sum, output); the sum is None unless wanted.  out['sum'] may be
    `residual` and out['output'] `x`."""
    if stream is not None:
        return _b._on(stream, dropout_layer_norm, locals())
    shape = _first(x, "x")
    _first(residual, "residual")
    _other(x.dtype, residual, "x")
    given, stay = _matrix(x, "x", shape, x.dtype, x), _matrix(residual, "residual", shape, residual.dtype, x)
    mask = _mask(rate, seed, site, x)
    g, b = _vector(gain, "gain", shape[1], x), _vector(bias, "bias", shape[1], x)
    total, total_made = _result(out, "sum", shape, residual.dtype, x) if want_sum else (None, _NONE)
    y, made = _result(out, "output", shape, x.dtype, x)
    _call("dropout_layer_norm", x, _pack_join.pack, DTYPES[x.dtype], DTYPES[residual.dtype], *shape, *given, *stay,
          *total_made, *made, *_NONE, *_NONE, *_NONE, *_NONE, *mask, g, b, 0, 0, epsilon, 0, 0)
    return {"sum": total, "output": y}


def dropout_layer_norm_backward(sum, d_output, rate, seed, site=0, d_sum=None, gain=None, bias=None, epsilon=1e-5,
                                want_d_x=True, out=None, workspace=None, stream=None):
    """The gradients of dropout_layer_norm given its `sum`, its output's gradient and that of the sum further along the
    stream (`d_sum`, None: the stream ends here): d_residual = d_sum + layer_norm's, d_x = d_residual through the mask
    (None unless wanted: with rate 0 it is d_residual).  The rest as in layer_norm_backward.  Returns dict(d_residual,
    d_x, d_gain, d_bias); out['d_residual'] may be `d_sum` or `sum`, and out['d_x'] `d_output`."""
    if stream is not None:
        return _b._on(stream, dropout_layer_norm_backward, locals())
    shape = _first(sum, "sum")
    _first(d_output, "d_output")
    to = _other(d_output.dtype, sum, "d_output")
    given, dy = _matrix(sum, "sum", shape, sum.dtype, sum), _matrix(d_output, "d_output", shape, to, sum)
    onward = _NONE if d_sum is None else _matrix(d_sum, "d_sum", shape, sum.dtype, sum)
    mask = _mask(rate, seed, site, sum)
    g = _vector(gain, "gain", shape[1], sum)
    _vector(bias, "bias", shape[1], sum)
    stay, stay_made = _result(out, "d_residual", shape, sum.dtype, sum)
    dx, made = _result(out, "d_x", shape, to, sum) if want_d_x else (None, _NONE)
    d_gain, dg = _gradient(out, "d_gain", gain, sum)
    d_bias, db = _gradient(out, "d_bias", bias, sum)
    workspace, *lent = _workspace(workspace, dg or db, *shape, sum)
    _call("dropout_layer_norm_backward", sum, _pack_join.pack, DTYPES[to], DTYPES[sum.dtype], *shape, *_NONE, *_NONE,
          *given, *_NONE, *dy, *onward, *stay_made, *made, *mask, g, 0, dg, db, epsilon, *lent)
    return {"d_residual": stay, "d_x": dx, "d_gain": d_gain, "d_bias": d_bias}
