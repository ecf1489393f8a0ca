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
_VERBS = {v: (_b._fast(v), p.pack) for p, verbs in (
    (_pack_norm, ("layer_norm", "layer_norm_backward")), (_pack_dropout, ("dropout", "dropout_backward")),
    (_pack_join, ("dropout_layer_norm", "dropout_layer_norm_backward"))) for v in verbs}
_NONE = 0, 0
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_F32, _I64 = torch.float32, torch.int64


def _call(verb, lead, device, args):
    """The verb on `device`, that of `lead`, and its current stream, or raises.  `args`: the struct up to the stream."""
    call, pack = _VERBS[verb]
    if device >= 0 and device != _current_device():
        with torch.cuda.device(device):
            rc = call(pack(*args, _b._raw_stream(lead)))
    else:
        rc = call(pack(*args, _b._raw_stream(lead)))
    if rc:
        _b.raise_for(rc, verb)


# The checks below ask a tensor for little: each question costs a tenth of a microsecond.

def _first(t, name):
    """(shape, data type, device, (data, row stride)) of the call's first matrix [rows, width]."""
    if not t.is_cuda:
        _b._check_cuda(t, name)
    shape, dtype = t.shape, t.dtype
    if len(shape) != 2:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be [rows, width], not {list(shape)}")
    if dtype not in DTYPES:
        raise UnsupportedError(CLI_UNSUPPORTED, f"{name}: {dtype}")
    row, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name}: the elements of a row must be adjacent")
    return shape, dtype, t.get_device(), (t.data_ptr(), row)


def _matrix(t, name, shape, dtype, device):
    """(data, row stride) of a matrix of `shape` on `device` whose rows' elements are adjacent."""
    if t.get_device() != device:
        _elsewhere(t, name)
    if t.dtype is not dtype:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, f"{name} must be {dtype}")
    if t.shape != shape:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be {list(shape)}, not {list(t.shape)}")
    row, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name}: the elements of a row must be adjacent")
    return t.data_ptr(), row


def _elsewhere(t, name):
    _b._check_cuda(t, name)
    raise InvalidArgumentError(CLI_INVALID_ARGUMENT, f"{name} is on another device than the call's first matrix")


def _vector(t, name, n, device, dtype=_F32):
    """The address of a packed vector of n elements on `device`, 0 for None."""
    if t is None:
        return 0
    if t.get_device() != device:
        _elsewhere(t, name)
    if t.dtype is not dtype:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, f"{name} must be {dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be [{n}], packed")
    return t.data_ptr()


def _result(out, name, shape, dtype, like, device):
    """The caller's output `name`, or a new packed one, and its (data, row stride)."""
    t = out.get(name) if out else None
    if t is not None:
        return t, _matrix(t, "out " + name, shape, dtype, device)
    if dtype is like.dtype and like.is_contiguous():
        t = torch.empty_like(like)
    else:
        t = torch.empty(shape, dtype=dtype, device=like.device)
    return t, (t.data_ptr(), shape[1])


def _gradient(out, name, of, device):
    """The gradient of a vector: the caller's or a new one, and its address; None where the vector is."""
    if of is None:
        return None, 0
    t = out.get(name) if out else None
    if t is not None:
        return t, _vector(t, "out " + name, of.numel(), device)
    t = torch.empty_like(of)
    return t, t.data_ptr()


def _other(dtype, stream, what):
    """A type that goes with the stream's: the same, or a 16-bit one beside fp32."""
    if dtype is None or dtype is stream:
        return stream
    if dtype not in DTYPES or stream is not _F32:
        raise UnsupportedError(CLI_UNSUPPORTED, f"{what}: {dtype} beside {stream}")
    return dtype


def _mask(rate, seed, site, device):
    """The mask's words in a struct."""
    if not 0 <= site <= 65535:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, "site must be 0 .. 65535")
    # without a seed it is refused by the library unless the rate is 0
    return rate, _vector(seed, "seed", 2, device, _I64), site


def layer_norm_backward_workspace_bytes(rows, width):
    return int(_b.lib.layer_norm_backward_workspace_bytes(rows, width))


def _workspace(workspace, wanted, shape, like, device):
    """(tensor to keep until the call is made, address, bytes)"""
    if workspace is not None:
        lent = _b._lent(workspace)
        if workspace.get_device() != device:
            _elsewhere(workspace, "workspace")
        return workspace, *lent
    if not wanted:
        return None, 0, 0
    need = _b.lib.layer_norm_backward_workspace_bytes(*shape)
    if not need:
        return None, 0, 0
    workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    return workspace, workspace.data_ptr(), need


def layer_norm(x, gain=None, bias=None, epsilon=1e-5, dtype=None, out=None, stream=None):
    """Normalises each row of `x` [rows, width]: gain * (x - mean) / sqrt(variance + epsilon) + bias, with fp32 [width]
    gains (None: ones) and biases (None: zeros).  bf16, fp16 or fp32; `dtype` is the output's type, 16-bit beside an
    fp32 `x` if wanted.  Returns dict(output); out['output'] may be `x` itself."""
    if stream is not None:
        return _b._on(stream, layer_norm, locals())
    shape, stream_dtype, device, given = _first(x, "x")
    to = _other(dtype, stream_dtype, "dtype")
    g, b = _vector(gain, "gain", shape[1], device), _vector(bias, "bias", shape[1], device)
    y, made = _result(out, "output", shape, to, x, device)
    _call("layer_norm", x, device, (DTYPES[stream_dtype], DTYPES[to], *shape, *given, *made, 0, 0, 0, 0, g, b, 0, 0, epsilon,
                                    0, 0))
    return {"output": y}


def layer_norm_backward(x, d_output, gain=None, bias=None, epsilon=1e-5, out=None, workspace=None, stream=None):
    """The gradients of layer_norm for `x`, its gain and its bias, given that of its output.  A gain's or bias's
    gradient (fp32 [width]) is None where that is.  Returns dict(d_x, d_gain, d_bias); out['d_x'] may be `x` or, of one
    type with it, `d_output`."""
    if stream is not None:
        return _b._on(stream, layer_norm_backward, locals())
    shape, stream_dtype, device, given = _first(x, "x")
    to = _other(d_output.dtype, stream_dtype, "d_output")
    dy = _matrix(d_output, "d_output", shape, to, device)
    g = _vector(gain, "gain", shape[1], device)
    _vector(bias, "bias", shape[1], device)
    dx, made = _result(out, "d_x", shape, stream_dtype, x, device)
    d_gain, dg = _gradient(out, "d_gain", gain, device)
    d_bias, db = _gradient(out, "d_bias", bias, device)
    workspace, *lent = _workspace(workspace, dg or db, shape, x, device)
    _call("layer_norm_backward", x, device, (DTYPES[stream_dtype], DTYPES[to], *shape, *given, 0, 0, *dy, *made, g, 0, dg, db,
                                             epsilon, *lent))
    return {"d_x": dx, "d_gain": d_gain, "d_bias": d_bias}


def dropout(x, rate, seed, site=0, out=None, stream=None):
    """Drops elements of `x` [rows, width] with probability `rate` (below 1) and scales the others by its complement's
    inverse.  bf16, fp16 or fp32.  A dropped element is 0 whatever `x` holds there.  Returns dict(output); out['output']
    may be `x` itself."""
    if stream is not None:
        return _b._on(stream, dropout, locals())
    shape, dtype, device, given = _first(x, "x")
    mask = _mask(rate, seed, site, device)
    y, made = _result(out, "output", shape, dtype, x, device)
    _call("dropout", x, device, (DTYPES[dtype], *shape, *given, *made, 0, 0, 0, 0, *mask))
    return {"output": y}


def dropout_backward(d_output, rate, seed, site=0, out=None, stream=None):
    """The gradient of dropout for its input: `d_output` through the same mask.  Returns dict(d_x)."""
    if stream is not None:
        return _b._on(stream, dropout_backward, locals())
    shape, dtype, device, given = _first(d_output, "d_output")
    mask = _mask(rate, seed, site, device)
    dx, made = _result(out, "d_x", shape, dtype, d_output, device)
    _call("dropout_backward", d_output, device, (DTYPES[dtype], *shape, 0, 0, 0, 0, *given, *made, *mask))
    return {"d_x": dx}


def dropout_layer_norm(x, residual, rate, seed, site=0, gain=None, bias=None, epsilon=1e-5, want_sum=True, out=None,
                       stream=None):
    """A branch's output `x` joins the residual stream, and the norm of that, in one pass: sum = residual + dropout(x),
    output = layer_norm(sum) (of the sum before it is rounded).  `residual` and the sum are of x's type or fp32; the rest
    as in dropout and layer_norm.  Returns dict(sum, output); the sum is None unless wanted.  out['sum'] may be
    `residual` and out['output'] `x`."""
    if stream is not None:
        return _b._on(stream, dropout_layer_norm, locals())
    shape, dtype, device, given = _first(x, "x")
    stream_dtype = residual.dtype
    _other(dtype, stream_dtype, "x")
    stay = _matrix(residual, "residual", shape, stream_dtype, device)
    mask = _mask(rate, seed, site, device)
    g, b = _vector(gain, "gain", shape[1], device), _vector(bias, "bias", shape[1], device)
    total, total_made = _result(out, "sum", shape, stream_dtype, residual, device) if want_sum else (None, _NONE)
    y, made = _result(out, "output", shape, dtype, x, device)
    _call("dropout_layer_norm", x, device, (DTYPES[dtype], DTYPES[stream_dtype], *shape, *given, *stay, *total_made, *made,
                                            0, 0, 0, 0, 0, 0, 0, 0, *mask, g, b, 0, 0, epsilon, 0, 0))
    return {"sum": total, "output": y}


def dropout_layer_norm_backward(sum, d_output, rate, seed, site=0, d_sum=None, gain=None, bias=None, epsilon=1e-5,
                                want_d_x=True, out=None, workspace=None, stream=None):
    """The gradients of dropout_layer_norm given its `sum`, its output's gradient and that of the sum further along the
    stream (`d_sum`, None: the stream ends here): d_residual = d_sum + layer_norm's, d_x = d_residual through the mask
    (None unless wanted: with rate 0 it is d_residual).  The rest as in layer_norm_backward.  Returns dict(d_residual,
    d_x, d_gain, d_bias); out['d_residual'] may be `d_sum` or `sum`, and out['d_x'] `d_output`."""
    if stream is not None:
        return _b._on(stream, dropout_layer_norm_backward, locals())
    shape, stream_dtype, device, given = _first(sum, "sum")
    to = _other(d_output.dtype, stream_dtype, "d_output")
    dy = _matrix(d_output, "d_output", shape, to, device)
    onward = _NONE if d_sum is None else _matrix(d_sum, "d_sum", shape, stream_dtype, device)
    mask = _mask(rate, seed, site, device)
    g = _vector(gain, "gain", shape[1], device)
    _vector(bias, "bias", shape[1], device)
    stay, stay_made = _result(out, "d_residual", shape, stream_dtype, sum, device)
    dx, made = _result(out, "d_x", shape, to, d_output, device) if want_d_x else (None, _NONE)
    d_gain, dg = _gradient(out, "d_gain", gain, device)
    d_bias, db = _gradient(out, "d_bias", bias, device)
    workspace, *lent = _workspace(workspace, dg or db, shape, sum, device)
    _call("dropout_layer_norm_backward", sum, device, (
        DTYPES[to], DTYPES[stream_dtype], *shape, 0, 0, 0, 0, *given, 0, 0, *dy, *onward, *stay_made, *made, *mask, g, 0, dg,
        db, epsilon, *lent))
    return {"d_residual": stay, "d_x": dx, "d_gain": d_gain, "d_bias": d_bias}
