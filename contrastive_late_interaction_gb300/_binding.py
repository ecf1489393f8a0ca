"""Thin ctypes binding over the C ABI of include/cli.h (argument marshalling only).

Every function here fills the verb's argument struct from torch tensors that
already live on the GPU, calls the exported C symbol of the same name, and
turns a non-OK status into an exception.  All arithmetic happens in the CUDA
library; if it is missing, importing this module raises.  PyTorch is used only
for device memory and streams.

A verb runs on the current stream, or on `stream` where one is given.  Its
inputs have to be ready on that stream, and they and any buffers lent to it
have to stay alive until it has passed them; what the verb makes itself is
ordered by it.
"""

from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

c_size_t, c_void_p, c_int, c_float = ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int, ctypes.c_float

STATUS_NAMES = ["ok", "invalid-argument", "shape-mismatch", "unsupported", "device", "malformed", "internal"]
CLI_OK, CLI_INVALID_ARGUMENT, CLI_SHAPE_MISMATCH, CLI_UNSUPPORTED, CLI_DEVICE, CLI_MALFORMED, CLI_INTERNAL = range(7)


class CliError(RuntimeError):
    """A non-OK status from the library; `status` is the cli_status_t value."""

    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {status_name(status)} ({status})")


class InvalidArgumentError(CliError, ValueError):
    pass


class ShapeMismatchError(CliError, ValueError):
    pass


class UnsupportedError(CliError, NotImplementedError):
    pass


class MalformedError(CliError, ValueError):
    pass


class DeviceError(CliError):
    pass


class InternalError(CliError):
    pass


_ERRORS = {CLI_INVALID_ARGUMENT: InvalidArgumentError, CLI_SHAPE_MISMATCH: ShapeMismatchError,
           CLI_UNSUPPORTED: UnsupportedError, CLI_MALFORMED: MalformedError, CLI_DEVICE: DeviceError,
           CLI_INTERNAL: InternalError}


def raise_for(status: int, where: str):
    if status != CLI_OK:
        raise _ERRORS.get(int(status), CliError)(status, where)


# ----------------------------------------------------------------------------
# structs (field for field as in include/cli.h)
# ----------------------------------------------------------------------------

class Edges(ctypes.Structure):
    _fields_ = [("offsets", c_void_p), ("ids", c_void_p), ("weights", c_void_p), ("edges", c_size_t)]


class Relations(ctypes.Structure):
    _fields_ = [("attract", Edges), ("repel", Edges), ("ignore", Edges), ("negatives_named", c_int),
                ("ambient_weight", c_float)]


class PairLossSigmoidArgs(ctypes.Structure):
    _fields_ = [("count", c_size_t), ("width", c_size_t), ("ld", c_size_t), ("embeddings", c_void_p),
                ("inverse_temperature", c_void_p), ("bias", c_void_p), ("relations", Relations),
                ("loss", c_void_p), ("d_embeddings", c_void_p), ("ld_d_embeddings", c_size_t),
                ("d_inverse_temperature", c_void_p), ("d_bias", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("device_status", c_void_p), ("stream", c_void_p),
                ("row_begin", c_size_t), ("row_count", c_size_t)]


class PairLossGroupsArgs(ctypes.Structure):
    _fields_ = [("base", PairLossSigmoidArgs), ("groups", c_void_p), ("group_count", c_size_t)]


class PairLossMatryoshkaArgs(ctypes.Structure):
    _fields_ = [("base", PairLossSigmoidArgs), ("prefix_widths", c_void_p), ("prefix_count", c_size_t),
                ("prefix_loss", c_void_p)]


MATRYOSHKA_MAX_PREFIXES = 8   # CLI_MATRYOSHKA_MAX_PREFIXES in include/cli.h


class PairLossSigmoidScoresArgs(ctypes.Structure):
    _fields_ = [("rows", c_size_t), ("cols", c_size_t), ("ld", c_size_t), ("scores", c_void_p),
                ("inverse_temperature", c_void_p), ("bias", c_void_p), ("relations", Relations),
                ("sides", c_void_p), ("loss", c_void_p), ("d_scores", c_void_p), ("ld_d_scores", c_size_t),
                ("d_inverse_temperature", c_void_p), ("d_bias", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("device_status", c_void_p), ("stream", c_void_p)]


class PairLossScoresArgs(ctypes.Structure):
    _fields_ = [("form", c_int), ("args", PairLossSigmoidScoresArgs)]


FORMS = {"balanced": 1, "ranked": 2, "sigmoid": 3}


class Tape(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("offsets", c_void_p), ("count", c_size_t), ("rows", c_size_t)]


class MaxSimArgs(ctypes.Structure):
    _fields_ = [("queries", Tape), ("documents", Tape), ("width", c_size_t), ("mean", c_int),
                ("scores", c_void_p), ("ld_scores", c_size_t), ("argmax", c_void_p), ("ld_argmax", c_size_t),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("device_status", c_void_p),
                ("stream", c_void_p)]


class MaxSimNamedArgs(ctypes.Structure):
    _fields_ = [("base", MaxSimArgs), ("pairs", Edges)]


class MaxSimBackwardArgs(ctypes.Structure):
    _fields_ = [("queries", Tape), ("documents", Tape), ("width", c_size_t), ("mean", c_int),
                ("argmax", c_void_p), ("ld_argmax", c_size_t), ("d_scores", c_void_p), ("ld_d_scores", c_size_t),
                ("d_queries", c_void_p), ("d_documents", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("device_status", c_void_p), ("stream", c_void_p)]


class MaxSimBackwardNamedArgs(ctypes.Structure):
    _fields_ = [("base", MaxSimBackwardArgs), ("pairs", Edges)]


class HeadsArgs(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("row_stride", c_size_t), ("head_stride", c_size_t)]


class RotaryTableArgs(ctypes.Structure):
    _fields_ = [("positions", c_size_t), ("rotary_dim", c_size_t), ("base", ctypes.c_double), ("scaling", c_int),
                ("factor", ctypes.c_double), ("trained_positions", c_size_t), ("table", c_void_p),
                ("stream", c_void_p)]


class RotaryPartArgs(ctypes.Structure):
    _fields_ = [("rows", c_size_t), ("heads", c_size_t), ("positions", c_void_p), ("x", HeadsArgs), ("y", HeadsArgs),
                ("d_y", HeadsArgs), ("d_x", HeadsArgs), ("gain", c_void_p), ("d_gain", c_void_p)]


class RotaryArgs(ctypes.Structure):
    _fields_ = [("dtype", c_int), ("interleaved", c_int), ("head_dim", c_size_t), ("rotary_dim", c_size_t),
                ("table", c_void_p), ("table_rows", c_size_t), ("epsilon", c_float), ("q", RotaryPartArgs),
                ("k", RotaryPartArgs), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("device_status", c_void_p), ("stream", c_void_p)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("dtype", c_int), ("items", c_size_t), ("query_rows", c_size_t), ("key_rows", c_size_t),
                ("query_offsets", c_void_p), ("key_offsets", c_void_p), ("max_query_rows", c_size_t),
                ("max_key_rows", c_size_t), ("query_heads", c_size_t), ("key_heads", c_size_t),
                ("head_dim", c_size_t), ("scale", c_float), ("key_mask", c_void_p), ("q", HeadsArgs),
                ("k", HeadsArgs), ("v", HeadsArgs), ("output", HeadsArgs), ("lse", c_void_p),
                ("d_output", HeadsArgs), ("d_q", HeadsArgs), ("d_k", HeadsArgs), ("d_v", HeadsArgs),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("device_status", c_void_p),
                ("stream", c_void_p)]


class RowsArgs(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("row_stride", c_size_t)]


class DropoutMaskArgs(ctypes.Structure):
    _fields_ = [("rate", ctypes.c_double), ("seed", c_void_p), ("site", ctypes.c_uint32)]


class LayerNormArgs(ctypes.Structure):
    _fields_ = [("x_dtype", c_int), ("y_dtype", c_int), ("rows", c_size_t), ("width", c_size_t), ("x", RowsArgs),
                ("y", RowsArgs), ("d_y", RowsArgs), ("d_x", RowsArgs), ("gain", c_void_p), ("bias", c_void_p),
                ("d_gain", c_void_p), ("d_bias", c_void_p), ("epsilon", c_float), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("stream", c_void_p)]


class DropoutArgs(ctypes.Structure):
    _fields_ = [("dtype", c_int), ("rows", c_size_t), ("width", c_size_t), ("x", RowsArgs), ("y", RowsArgs),
                ("d_y", RowsArgs), ("d_x", RowsArgs), ("mask", DropoutMaskArgs), ("stream", c_void_p)]


class DropoutLayerNormArgs(ctypes.Structure):
    _fields_ = [("dtype", c_int), ("stream_dtype", c_int), ("rows", c_size_t), ("width", c_size_t), ("x", RowsArgs),
                ("residual", RowsArgs), ("sum", RowsArgs), ("y", RowsArgs), ("d_y", RowsArgs), ("d_sum", RowsArgs),
                ("d_residual", RowsArgs), ("d_x", RowsArgs), ("mask", DropoutMaskArgs), ("gain", c_void_p),
                ("bias", c_void_p), ("d_gain", c_void_p), ("d_bias", c_void_p), ("epsilon", c_float),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("stream", c_void_p)]


DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # cli_dtype_t
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


EXPORTS = {
    "cli_status_name": (ctypes.c_char_p, [c_int]),
    "pair_loss_sigmoid_fwd_bwd": (c_int, [ctypes.POINTER(PairLossSigmoidArgs)]),
    "pair_loss_sigmoid_workspace_bytes": (c_size_t, [c_size_t, c_size_t, c_size_t]),
    "pair_loss_sigmoid_groups_fwd_bwd": (c_int, [ctypes.POINTER(PairLossGroupsArgs)]),
    "pair_loss_sigmoid_matryoshka_fwd_bwd": (c_int, [ctypes.POINTER(PairLossMatryoshkaArgs)]),
    "pair_loss_sigmoid_matryoshka_workspace_bytes": (c_size_t, [c_size_t, c_size_t, c_size_t]),
    "pair_loss_sigmoid_scores_fwd_bwd": (c_int, [ctypes.POINTER(PairLossSigmoidScoresArgs)]),
    "pair_loss_sigmoid_scores_workspace_bytes": (c_size_t, [c_size_t, c_size_t]),
    "pair_loss_scores_fwd_bwd": (c_int, [ctypes.POINTER(PairLossScoresArgs)]),
    "pair_loss_scores_workspace_bytes": (c_size_t, [c_int, c_size_t, c_size_t]),
    "maxsim_scores": (c_int, [ctypes.POINTER(MaxSimArgs)]),
    "maxsim_workspace_bytes": (c_size_t, [c_size_t, c_size_t, c_size_t, c_size_t, c_size_t]),
    "maxsim_scores_named": (c_int, [ctypes.POINTER(MaxSimNamedArgs)]),
    "maxsim_named_workspace_bytes": (c_size_t, [c_size_t, c_size_t, c_size_t, c_size_t, c_size_t]),
    "maxsim_backward": (c_int, [ctypes.POINTER(MaxSimBackwardArgs)]),
    "maxsim_backward_named": (c_int, [ctypes.POINTER(MaxSimBackwardNamedArgs)]),
    "maxsim_backward_workspace_bytes": (c_size_t, [c_size_t, c_size_t, c_size_t, c_size_t, c_size_t]),
    "maxsim_backward_no_alloc": (c_int, [ctypes.POINTER(MaxSimBackwardArgs)]),
    "rotary_table": (c_int, [ctypes.POINTER(RotaryTableArgs)]),
    "rotary_heads": (c_int, [ctypes.POINTER(RotaryArgs)]),
    "rotary_heads_backward": (c_int, [ctypes.POINTER(RotaryArgs)]),
    "norm_rotary_heads": (c_int, [ctypes.POINTER(RotaryArgs)]),
    "norm_rotary_heads_backward": (c_int, [ctypes.POINTER(RotaryArgs)]),
    "norm_rotary_heads_backward_workspace_bytes": (c_size_t, [c_size_t]),
    "cross_attention": (c_int, [ctypes.POINTER(AttentionArgs)]),
    "cross_attention_workspace_bytes": (c_size_t, [ctypes.POINTER(AttentionArgs)]),
    "cross_attention_backward": (c_int, [ctypes.POINTER(AttentionArgs)]),
    "cross_attention_backward_workspace_bytes": (c_size_t, [ctypes.POINTER(AttentionArgs)]),
    "layer_norm": (c_int, [ctypes.POINTER(LayerNormArgs)]),
    "layer_norm_backward": (c_int, [ctypes.POINTER(LayerNormArgs)]),
    "layer_norm_backward_workspace_bytes": (c_size_t, [c_size_t, c_size_t]),
    "dropout": (c_int, [ctypes.POINTER(DropoutArgs)]),
    "dropout_backward": (c_int, [ctypes.POINTER(DropoutArgs)]),
    "dropout_layer_norm": (c_int, [ctypes.POINTER(DropoutLayerNormArgs)]),
    "dropout_layer_norm_backward": (c_int, [ctypes.POINTER(DropoutLayerNormArgs)]),
    "cli_selftest_bounded_wait": (c_int, [c_void_p, c_void_p, ctypes.c_uint32, c_void_p]),
}
NO_ALLOC_MAX_QUERY_ROWS = 262144   # CLI_MAXSIM_NO_ALLOC_MAX_QUERY_ROWS in include/cli.h


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"the CUDA library {path} is not built; run __graft_entry__.build() "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()
LIB_PATH = _build.LIB


def status_name(status: int) -> str:
    return lib.cli_status_name(int(status)).decode()


# ----------------------------------------------------------------------------
# marshalling helpers
# ----------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check_cuda(t, name, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, f"{name} must be device memory")
    if dtype is not None and t.dtype != dtype:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, f"{name} must be {dtype}")


def _edges(e, count):
    """(offsets int64[count+1], ids int32[E], weights float32[E] | None) on the device -> Edges."""
    if e is None:
        return Edges(None, None, None, 0)
    off, ids = e[0], e[1]
    w = e[2] if len(e) > 2 else None
    _check_cuda(off, "offsets", torch.int64)
    _check_cuda(ids, "ids", torch.int32)
    _check_cuda(w, "weights", torch.float32)
    return Edges(_ptr(off), _ptr(ids) if ids.numel() else None, _ptr(w), int(ids.numel()))


def device_edges(edges, device="cuda"):
    """Uploads a host edge set (offsets, ids[, weights] numpy arrays or an object with those fields)."""
    if edges is None:
        return None
    if hasattr(edges, "offsets"):
        off, ids, w = edges.offsets, edges.ids, edges.weights
    else:
        off, ids = edges[0], edges[1]
        w = edges[2] if len(edges) > 2 else None
    import numpy as np
    o = torch.from_numpy(np.asarray(off, dtype=np.uint64).view(np.int64).copy()).to(device)
    i = torch.from_numpy(np.asarray(ids, dtype=np.uint32).view(np.int32).copy()).to(device)
    ww = None if w is None else torch.from_numpy(np.asarray(w, dtype=np.float32).copy()).to(device)
    return (o, i, ww) if ww is not None else (o, i)


def _band(band):
    """The anchor band (row_begin, row_count) of a pooled call; None is every row.  The library checks it."""
    if band is None:
        return dict(row_begin=0, row_count=0)
    begin, count = (int(v) for v in band)
    if begin < 0 or count < 0:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "band must be (row_begin, row_count) >= 0")
    return dict(row_begin=begin, row_count=count)


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _lent(workspace):
    """(address, bytes) of a lent workspace; (0, 0) for None."""
    if workspace is None:
        return 0, 0
    _check_cuda(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _check_lent(out, workspace, device_status):
    """What a caller lends a verb to write: device memory."""
    for name, t in (out or {}).items():
        if isinstance(t, torch.Tensor):
            _check_cuda(t, "out " + name)
    _check_cuda(device_status, "device_status", torch.int32)
    _lent(workspace)


def _on(stream, verb, arguments):
    """verb(**arguments) with `stream` as the current stream.  What the verb allocates or fills comes from that
    stream's pool, in its order: a workspace that the verb drops is not handed to the caller's stream while kernels
    still use it, and a result is not made of memory that the caller's stream still reads.  Results dropped by the
    caller wait for the caller's stream.  The verb's inputs, and buffers lent to it, are the caller's to keep and to
    order."""
    caller = torch.cuda.current_stream()
    arguments["stream"] = None
    with torch.cuda.stream(stream):
        made = verb(**arguments)
    for t in made.values():
        if t is not None:
            t.record_stream(caller)
    return made


def selftest_bounded_wait(limit_us=20000, device_status=None, gave_up=None, stream=None):
    """Runs the failure path of the kernels' bounded waits (one CTA waiting on a barrier nothing arrives
    at, giving up after `limit_us`).  Returns dict(device_status, gave_up) of device int32 tensors; the
    status reads CLI_INTERNAL and gave_up the number of threads (64) once the stream reaches them."""
    if stream is not None:
        return _on(stream, selftest_bounded_wait, locals())
    dev = torch.device("cuda", torch.cuda.current_device())
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    gu = gave_up if gave_up is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    _check_cuda(st, "device_status", torch.int32)
    _check_cuda(gu, "gave_up", torch.int32)
    raise_for(lib.cli_selftest_bounded_wait(_ptr(st), _ptr(gu), int(limit_us), _stream()),
              "cli_selftest_bounded_wait")
    return dict(device_status=st, gave_up=gu)


def check_device_status(status: torch.Tensor, where: str = "device"):
    """Synchronises on the status word and raises if the device reported a fault."""
    raise_for(int(status.item()), where)


# ----------------------------------------------------------------------------
# verbs
# ----------------------------------------------------------------------------

def pair_loss_sigmoid_workspace_bytes(count, width, edges):
    return int(lib.pair_loss_sigmoid_workspace_bytes(count, width, edges))


def pair_loss_sigmoid_fwd_bwd(embeddings, inverse_temperature, bias, attract, repel=None, ignore=None,
                              negatives_named=False, ambient_weight=1.0, out=None, workspace=None,
                              device_status=None, stream=None, band=None):
    """Pooled sigmoid pair loss over bf16 embeddings [N, ld] (first `width` = embeddings.shape[1] columns
    unless `out['width']` narrows it).  Returns dict(loss, d_embeddings, d_inverse_temperature, d_bias,
    device_status) of device tensors; the device status is not synchronised here.  `band` = (row_begin,
    row_count) scores only the anchors in those rows: the results are that band's shares of the whole call's."""
    if stream is not None:
        return _on(stream, pair_loss_sigmoid_fwd_bwd, locals())
    _check_cuda(embeddings, "embeddings", torch.bfloat16)
    _check_cuda(inverse_temperature, "inverse_temperature", torch.float32)
    _check_cuda(bias, "bias", torch.float32)
    n, ld = embeddings.shape
    width = (out or {}).get("width", ld)
    dev = embeddings.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    loss = out.get("loss") if out.get("loss") is not None else torch.empty(1, device=dev)
    de = out.get("d_embeddings") if out.get("d_embeddings") is not None else torch.empty(n, width, device=dev)
    dt = out.get("d_inverse_temperature") if out.get("d_inverse_temperature") is not None else torch.empty(1, device=dev)
    db = out.get("d_bias") if out.get("d_bias") is not None else torch.empty(1, device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    A, R, I = _edges(attract, n), _edges(repel, n), _edges(ignore, n)
    total = A.edges + R.edges + I.edges
    need = pair_loss_sigmoid_workspace_bytes(n, width, total)
    ws = workspace if workspace is not None else _ws(need, dev)
    args = PairLossSigmoidArgs(
        count=n, width=width, ld=embeddings.stride(0), embeddings=_ptr(embeddings),
        inverse_temperature=_ptr(inverse_temperature), bias=_ptr(bias),
        relations=Relations(A, R, I, int(bool(negatives_named)), float(ambient_weight)),
        loss=_ptr(loss), d_embeddings=_ptr(de), ld_d_embeddings=de.stride(0),
        d_inverse_temperature=_ptr(dt), d_bias=_ptr(db), workspace=_ptr(ws), workspace_bytes=_lent(ws)[1],
        device_status=_ptr(st), stream=_stream(), **_band(band))
    raise_for(lib.pair_loss_sigmoid_fwd_bwd(ctypes.byref(args)), "pair_loss_sigmoid_fwd_bwd")
    return dict(loss=loss, d_embeddings=de, d_inverse_temperature=dt, d_bias=db, device_status=st)


def pair_loss_sigmoid_groups_fwd_bwd(embeddings, groups, inverse_temperature, bias, attract, repel=None, ignore=None,
                                     negatives_named=False, ambient_weight=1.0, out=None, workspace=None,
                                     device_status=None, stream=None, band=None):
    """The pooled sigmoid pair loss with temperature groups: `groups` (int32 [N]) selects each item's pair of
    `inverse_temperature`, `bias` (fp32 [G]) and a cell takes its anchor's.  Returns dict(loss, d_embeddings,
    d_inverse_temperature [G], d_bias [G], device_status) of device tensors."""
    if stream is not None:
        return _on(stream, pair_loss_sigmoid_groups_fwd_bwd, locals())
    _check_cuda(embeddings, "embeddings", torch.bfloat16)
    _check_cuda(groups, "groups", torch.int32)
    _check_cuda(inverse_temperature, "inverse_temperature", torch.float32)
    _check_cuda(bias, "bias", torch.float32)
    n, ld = embeddings.shape
    g = inverse_temperature.numel()
    if bias.numel() != g or groups.numel() != n:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "groups, inverse_temperature and bias disagree in size")
    width = (out or {}).get("width", ld)
    dev = embeddings.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    loss = out.get("loss") if out.get("loss") is not None else torch.empty(1, device=dev)
    de = out.get("d_embeddings") if out.get("d_embeddings") is not None else torch.empty(n, width, device=dev)
    dt = out.get("d_inverse_temperature") if out.get("d_inverse_temperature") is not None else torch.empty(g, device=dev)
    db = out.get("d_bias") if out.get("d_bias") is not None else torch.empty(g, device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    A, R, I = _edges(attract, n), _edges(repel, n), _edges(ignore, n)
    total = A.edges + R.edges + I.edges
    need = pair_loss_sigmoid_workspace_bytes(n, width, total)
    ws = workspace if workspace is not None else _ws(need, dev)
    base = PairLossSigmoidArgs(
        count=n, width=width, ld=embeddings.stride(0), embeddings=_ptr(embeddings),
        inverse_temperature=_ptr(inverse_temperature), bias=_ptr(bias),
        relations=Relations(A, R, I, int(bool(negatives_named)), float(ambient_weight)),
        loss=_ptr(loss), d_embeddings=_ptr(de), ld_d_embeddings=de.stride(0),
        d_inverse_temperature=_ptr(dt), d_bias=_ptr(db), workspace=_ptr(ws), workspace_bytes=_lent(ws)[1],
        device_status=_ptr(st), stream=_stream(), **_band(band))
    args = PairLossGroupsArgs(base=base, groups=_ptr(groups), group_count=g)
    raise_for(lib.pair_loss_sigmoid_groups_fwd_bwd(ctypes.byref(args)), "pair_loss_sigmoid_groups_fwd_bwd")
    return dict(loss=loss, d_embeddings=de, d_inverse_temperature=dt, d_bias=db, device_status=st)


def pair_loss_sigmoid_matryoshka_workspace_bytes(count, width, edges):
    return int(lib.pair_loss_sigmoid_matryoshka_workspace_bytes(count, width, edges))


def pair_loss_sigmoid_matryoshka_fwd_bwd(embeddings, prefix_widths, inverse_temperature, bias, attract, repel=None,
                                         ignore=None, negatives_named=False, ambient_weight=1.0, out=None,
                                         workspace=None, device_status=None, stream=None, band=None):
    """The pooled sigmoid pair loss summed over the normalised prefixes `prefix_widths` of bf16 embeddings
    [N, ld] (first `width` = embeddings.shape[1] columns unless `out['width']` narrows it).  Returns
    dict(loss, d_embeddings, d_inverse_temperature, d_bias, prefix_loss, device_status) of device tensors."""
    if stream is not None:
        return _on(stream, pair_loss_sigmoid_matryoshka_fwd_bwd, locals())
    _check_cuda(embeddings, "embeddings", torch.bfloat16)
    _check_cuda(inverse_temperature, "inverse_temperature", torch.float32)
    _check_cuda(bias, "bias", torch.float32)
    n, ld = embeddings.shape
    width = (out or {}).get("width", ld)
    dev = embeddings.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    widths = (c_size_t * len(prefix_widths))(*[int(p) for p in prefix_widths])
    loss = out.get("loss") if out.get("loss") is not None else torch.empty(1, device=dev)
    de = out.get("d_embeddings") if out.get("d_embeddings") is not None else torch.empty(n, width, device=dev)
    dt = out.get("d_inverse_temperature") if out.get("d_inverse_temperature") is not None else torch.empty(1, device=dev)
    db = out.get("d_bias") if out.get("d_bias") is not None else torch.empty(1, device=dev)
    pl = out.get("prefix_loss") if out.get("prefix_loss") is not None else torch.empty(max(1, len(prefix_widths)),
                                                                                         device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    A, R, I = _edges(attract, n), _edges(repel, n), _edges(ignore, n)
    total = A.edges + R.edges + I.edges
    need = pair_loss_sigmoid_matryoshka_workspace_bytes(n, width, total)
    ws = workspace if workspace is not None else _ws(need, dev)
    base = PairLossSigmoidArgs(
        count=n, width=width, ld=embeddings.stride(0), embeddings=_ptr(embeddings),
        inverse_temperature=_ptr(inverse_temperature), bias=_ptr(bias),
        relations=Relations(A, R, I, int(bool(negatives_named)), float(ambient_weight)),
        loss=_ptr(loss), d_embeddings=_ptr(de), ld_d_embeddings=de.stride(0),
        d_inverse_temperature=_ptr(dt), d_bias=_ptr(db), workspace=_ptr(ws), workspace_bytes=_lent(ws)[1],
        device_status=_ptr(st), stream=_stream(), **_band(band))
    args = PairLossMatryoshkaArgs(base=base, prefix_widths=ctypes.cast(widths, c_void_p),
                                  prefix_count=len(prefix_widths), prefix_loss=_ptr(pl))
    raise_for(lib.pair_loss_sigmoid_matryoshka_fwd_bwd(ctypes.byref(args)), "pair_loss_sigmoid_matryoshka_fwd_bwd")
    return dict(loss=loss, d_embeddings=de, d_inverse_temperature=dt, d_bias=db, prefix_loss=pl, device_status=st)


def pair_loss_sigmoid_scores_workspace_bytes(rows, cols):
    return int(lib.pair_loss_sigmoid_scores_workspace_bytes(rows, cols))


def pair_loss_sigmoid_scores_fwd_bwd(scores, inverse_temperature, bias, attract, repel=None, ignore=None,
                                     sides=None, negatives_named=False, ambient_weight=1.0, out=None,
                                     workspace=None, device_status=None, stream=None):
    """Sigmoid pair loss over an fp32 score matrix [rows, cols]."""
    if stream is not None:
        return _on(stream, pair_loss_sigmoid_scores_fwd_bwd, locals())
    _check_cuda(scores, "scores", torch.float32)
    _check_cuda(sides, "sides", torch.uint8)
    rows, cols = scores.shape
    dev = scores.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    loss = out.get("loss") if out.get("loss") is not None else torch.empty(1, device=dev)
    ds = out.get("d_scores") if out.get("d_scores") is not None else torch.empty(rows, cols, device=dev)
    dt = out.get("d_inverse_temperature") if out.get("d_inverse_temperature") is not None else torch.empty(1, device=dev)
    db = out.get("d_bias") if out.get("d_bias") is not None else torch.empty(1, device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else _ws(pair_loss_sigmoid_scores_workspace_bytes(rows, cols), dev)
    A, R, I = _edges(attract, rows), _edges(repel, rows), _edges(ignore, rows)
    args = PairLossSigmoidScoresArgs(
        rows=rows, cols=cols, ld=scores.stride(0), scores=_ptr(scores), inverse_temperature=_ptr(inverse_temperature),
        bias=_ptr(bias), relations=Relations(A, R, I, int(bool(negatives_named)), float(ambient_weight)),
        sides=_ptr(sides), loss=_ptr(loss), d_scores=_ptr(ds), ld_d_scores=ds.stride(0),
        d_inverse_temperature=_ptr(dt), d_bias=_ptr(db), workspace=_ptr(ws), workspace_bytes=_lent(ws)[1],
        device_status=_ptr(st), stream=_stream())
    raise_for(lib.pair_loss_sigmoid_scores_fwd_bwd(ctypes.byref(args)), "pair_loss_sigmoid_scores_fwd_bwd")
    return dict(loss=loss, d_scores=ds, d_inverse_temperature=dt, d_bias=db, device_status=st)


def pair_loss_scores_workspace_bytes(form, rows, cols):
    return int(lib.pair_loss_scores_workspace_bytes(FORMS[form], rows, cols))


def pair_loss_scores_fwd_bwd(form, scores, inverse_temperature, bias, attract, repel=None, ignore=None, sides=None,
                             negatives_named=False, ambient_weight=1.0, out=None, workspace=None, device_status=None,
                             stream=None):
    """Pair loss of form 'balanced', 'ranked' or 'sigmoid' over an fp32 score matrix [rows, cols]."""
    if stream is not None:
        return _on(stream, pair_loss_scores_fwd_bwd, locals())
    _check_cuda(scores, "scores", torch.float32)
    _check_cuda(sides, "sides", torch.uint8)
    rows, cols = scores.shape
    dev = scores.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    loss = out.get("loss") if out.get("loss") is not None else torch.empty(1, device=dev)
    ds = out.get("d_scores") if out.get("d_scores") is not None else torch.empty(rows, cols, device=dev)
    dt = out.get("d_inverse_temperature") if out.get("d_inverse_temperature") is not None else torch.empty(1, device=dev)
    db = out.get("d_bias") if out.get("d_bias") is not None else torch.empty(1, device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else _ws(pair_loss_scores_workspace_bytes(form, rows, cols), dev)
    A, R, I = _edges(attract, rows), _edges(repel, rows), _edges(ignore, rows)
    inner = PairLossSigmoidScoresArgs(
        rows=rows, cols=cols, ld=scores.stride(0), scores=_ptr(scores), inverse_temperature=_ptr(inverse_temperature),
        bias=_ptr(bias), relations=Relations(A, R, I, int(bool(negatives_named)), float(ambient_weight)),
        sides=_ptr(sides), loss=_ptr(loss), d_scores=_ptr(ds), ld_d_scores=ds.stride(0),
        d_inverse_temperature=_ptr(dt), d_bias=_ptr(db), workspace=_ptr(ws), workspace_bytes=_lent(ws)[1],
        device_status=_ptr(st), stream=_stream())
    args = PairLossScoresArgs(form=FORMS[form], args=inner)
    raise_for(lib.pair_loss_scores_fwd_bwd(ctypes.byref(args)), "pair_loss_scores_fwd_bwd")
    return dict(loss=loss, d_scores=ds, d_inverse_temperature=dt, d_bias=db, device_status=st)


def _tape(data, offsets):
    _check_cuda(data, "tape data", torch.bfloat16)
    _check_cuda(offsets, "tape offsets", torch.int64)
    return Tape(_ptr(data), _ptr(offsets), offsets.numel() - 1, data.shape[0])


def maxsim_workspace_bytes(nq, nd, rows_q, rows_d, width):
    return int(lib.maxsim_workspace_bytes(nq, nd, rows_q, rows_d, width))


def maxsim_backward_workspace_bytes(nq, nd, rows_q, rows_d, width):
    return int(lib.maxsim_backward_workspace_bytes(nq, nd, rows_q, rows_d, width))


def maxsim_scores(q_data, q_offsets, d_data, d_offsets, mean=False, out=None, workspace=None, device_status=None,
                  stream=None):
    """Hard MaxSim of every query against every document.  Returns dict(scores [nq, nd] fp32,
    argmax [nd, rows_q] int32 (document-major), device_status)."""
    if stream is not None:
        return _on(stream, maxsim_scores, locals())
    Q, D = _tape(q_data, q_offsets), _tape(d_data, d_offsets)
    width = q_data.shape[1]
    if d_data.shape[1] != width:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "maxsim_scores: query and document widths differ")
    dev = q_data.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    scores = out.get("scores") if out.get("scores") is not None else torch.empty(Q.count, D.count, device=dev)
    argmax = out.get("argmax") if out.get("argmax") is not None else torch.empty(D.count, Q.rows, dtype=torch.int32,
                                                                                  device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else _ws(maxsim_workspace_bytes(Q.count, D.count, Q.rows, D.rows, width),
                                                     dev)
    args = MaxSimArgs(queries=Q, documents=D, width=width, mean=int(bool(mean)), scores=_ptr(scores),
                      ld_scores=scores.stride(0), argmax=_ptr(argmax), ld_argmax=argmax.stride(0),
                      workspace=_ptr(ws), workspace_bytes=_lent(ws)[1], device_status=_ptr(st), stream=_stream())
    raise_for(lib.maxsim_scores(ctypes.byref(args)), "maxsim_scores")
    return dict(scores=scores, argmax=argmax, device_status=st)


def maxsim_named_workspace_bytes(nq, nd, rows_q, rows_d, width):
    return int(lib.maxsim_named_workspace_bytes(nq, nd, rows_q, rows_d, width))


def maxsim_scores_named(q_data, q_offsets, d_data, d_offsets, pairs, mean=False, out=None, workspace=None,
                        device_status=None, stream=None):
    """Hard MaxSim of each query against the documents `pairs` names (a CSR over the queries, as from
    `device_edges`).  Returns dict(scores [nq, nd] fp32, zero for pairs not named, argmax [nd, rows_q] int32,
    a valid row of the document for pairs not named, device_status)."""
    if stream is not None:
        return _on(stream, maxsim_scores_named, locals())
    Q, D = _tape(q_data, q_offsets), _tape(d_data, d_offsets)
    width = q_data.shape[1]
    if d_data.shape[1] != width:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "maxsim_scores_named: query and document widths differ")
    dev = q_data.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    scores = out.get("scores") if out.get("scores") is not None else torch.empty(Q.count, D.count, device=dev)
    argmax = out.get("argmax") if out.get("argmax") is not None else torch.empty(D.count, Q.rows, dtype=torch.int32,
                                                                                  device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else _ws(
        maxsim_named_workspace_bytes(Q.count, D.count, Q.rows, D.rows, width), dev)
    base = MaxSimArgs(queries=Q, documents=D, width=width, mean=int(bool(mean)), scores=_ptr(scores),
                      ld_scores=scores.stride(0), argmax=_ptr(argmax), ld_argmax=argmax.stride(0),
                      workspace=_ptr(ws), workspace_bytes=_lent(ws)[1], device_status=_ptr(st), stream=_stream())
    args = MaxSimNamedArgs(base=base, pairs=_edges(pairs, Q.count))
    raise_for(lib.maxsim_scores_named(ctypes.byref(args)), "maxsim_scores_named")
    return dict(scores=scores, argmax=argmax, device_status=st)


def maxsim_backward(q_data, q_offsets, d_data, d_offsets, argmax, d_scores, mean=False, out=None, workspace=None,
                    device_status=None, stream=None):
    """Gradient through the argmax.  Returns dict(d_queries, d_documents, device_status)."""
    if stream is not None:
        return _on(stream, maxsim_backward, locals())
    Q, D = _tape(q_data, q_offsets), _tape(d_data, d_offsets)
    _check_cuda(argmax, "argmax", torch.int32)
    _check_cuda(d_scores, "d_scores", torch.float32)
    width = q_data.shape[1]
    dev = q_data.device
    out = dict(out or {})
    _check_lent(out, workspace, device_status)
    dq = out.get("d_queries") if out.get("d_queries") is not None else torch.empty(Q.rows, width, device=dev)
    dd = out.get("d_documents") if out.get("d_documents") is not None else torch.empty(D.rows, width, device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else _ws(
        maxsim_backward_workspace_bytes(Q.count, D.count, Q.rows, D.rows, width), dev)
    args = MaxSimBackwardArgs(queries=Q, documents=D, width=width, mean=int(bool(mean)), argmax=_ptr(argmax),
                              ld_argmax=argmax.stride(0), d_scores=_ptr(d_scores), ld_d_scores=d_scores.stride(0),
                              d_queries=_ptr(dq), d_documents=_ptr(dd), workspace=_ptr(ws),
                              workspace_bytes=_lent(ws)[1], device_status=_ptr(st), stream=_stream())
    raise_for(lib.maxsim_backward(ctypes.byref(args)), "maxsim_backward")
    return dict(d_queries=dq, d_documents=dd, device_status=st)


def maxsim_backward_named(q_data, q_offsets, d_data, d_offsets, argmax, d_scores, pairs, mean=False, out=None,
                          device_status=None, stream=None):
    """Gradient through the argmax of the named pairs only (`pairs` as for maxsim_scores_named).  Returns
    dict(d_queries, d_documents, device_status)."""
    if stream is not None:
        return _on(stream, maxsim_backward_named, locals())
    Q, D = _tape(q_data, q_offsets), _tape(d_data, d_offsets)
    _check_cuda(argmax, "argmax", torch.int32)
    _check_cuda(d_scores, "d_scores", torch.float32)
    width = q_data.shape[1]
    dev = q_data.device
    out = dict(out or {})
    _check_lent(out, None, device_status)
    dq = out.get("d_queries") if out.get("d_queries") is not None else torch.empty(Q.rows, width, device=dev)
    dd = out.get("d_documents") if out.get("d_documents") is not None else torch.empty(D.rows, width, device=dev)
    st = device_status if device_status is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    base = MaxSimBackwardArgs(queries=Q, documents=D, width=width, mean=int(bool(mean)), argmax=_ptr(argmax),
                              ld_argmax=argmax.stride(0), d_scores=_ptr(d_scores), ld_d_scores=d_scores.stride(0),
                              d_queries=_ptr(dq), d_documents=_ptr(dd), workspace=None, workspace_bytes=0,
                              device_status=_ptr(st), stream=_stream())
    args = MaxSimBackwardNamedArgs(base=base, pairs=_edges(pairs, Q.count))
    raise_for(lib.maxsim_backward_named(ctypes.byref(args)), "maxsim_backward_named")
    return dict(d_queries=dq, d_documents=dd, device_status=st)


# ----------------------------------------------------------------------------
# token states
#
# These calls are often short, so their host side is kept to a few microseconds: the argument struct is packed in one
# call (its layout checked against the ctypes structure), and a tensor's checks are a few comparisons.
# ----------------------------------------------------------------------------

def _fast(name):
    """The C function `name`, taking its argument struct as packed bytes."""
    fn = lib[name]   # a function object of its own, beside lib.name
    fn.restype, fn.argtypes = EXPORTS[name][0], [ctypes.c_char_p]
    return fn


_PART = "17Q"       # rows, heads, positions, x, y, d_y, d_x, gain, d_gain
_pack_rotary = struct.Struct("@2i4Qf4x" + _PART + _PART + "4Q")
_pack_attention = struct.Struct("@i4x10Qf4x" + "Q12QQ12Q" + "4Q")
_pack_last = struct.Struct("@4Q")   # workspace, workspace_bytes, device_status, stream
_ATTENTION_LAST = _pack_attention.size - _pack_last.size
assert _pack_rotary.size == ctypes.sizeof(RotaryArgs) and _pack_attention.size == ctypes.sizeof(AttentionArgs)
_ROTARY = {v: _fast(v) for v in ("rotary_heads", "rotary_heads_backward", "norm_rotary_heads",
                                 "norm_rotary_heads_backward")}
_ATTENTION = {v: (_fast(v), _fast(v + "_workspace_bytes")) for v in ("cross_attention", "cross_attention_backward")}
_NO_GRADIENTS = (0,) * 12   # d_output, d_q, d_k, d_v


def _raw_stream(tensor):
    return torch.cuda.current_stream(tensor.device).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):   # the same without building a Stream object
    def _raw_stream(tensor):   # noqa: F811
        return torch._C._cuda_getCurrentRawStream(tensor.get_device())


def _heads(t, name, shape, dtype):
    """(data, row stride, head stride) of a tensor of `shape` [rows, heads, dim] whose heads are contiguous."""
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda:
        _check_cuda(t, name, dtype)
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be {list(shape)}, not {list(t.shape)}")
    row, head, inner = t.stride()
    if inner != 1 and shape[2] > 1:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name}: the elements of a head must be contiguous")
    return t.data_ptr(), row, head


def _vector(t, name, n, dtype):
    """The address of a packed vector of n elements, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or not t.is_cuda:
        _check_cuda(t, name, dtype)
    if t.numel() != n or not t.is_contiguous():
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be [{n}], packed")
    return t.data_ptr()


def _states(t, name):
    """The shape of a matrix [rows, heads, dim] on the device."""
    if not t.is_cuda:
        _check_cuda(t, name)
    if t.dim() != 3:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be [rows, heads, head_dim], not {list(t.shape)}")
    if t.dtype not in DTYPES:
        raise UnsupportedError(CLI_UNSUPPORTED, f"{name}: {t.dtype}")
    return t.shape


def _result(out, name, like, shape):
    """The caller's output `name`, or a new packed one of `shape`, and its words in the struct: one made here needs no
    checks."""
    t = out.get(name) if out else None
    if t is not None:
        return t, _heads(t, "out " + name, shape, like.dtype)
    if shape == like.shape and like.is_contiguous():
        t = torch.empty_like(like)
    else:
        t = torch.empty(shape, dtype=like.dtype, device=like.device)
    return t, (t.data_ptr(), shape[1] * shape[2], shape[2])


def _status(device_status, like):
    if device_status is None:
        return torch.empty(1, dtype=torch.int32, device=like.device)   # the call writes it
    _check_cuda(device_status, "device_status", torch.int32)
    return device_status


def rotary_table(positions, rotary_dim, base=10000.0, scaling="plain", factor=1.0, trained_positions=0, out=None,
                 device="cuda", stream=None):
    """The (cos, sin) table [positions, rotary_dim / 2, 2] fp32 that the rotation verbs read.  `scaling` is 'plain',
    'linear', 'ntk' or 'yarn' for contexts `factor` times the trained one.  Returns dict(table)."""
    if stream is not None:
        return _on(stream, rotary_table, locals())
    if scaling not in ROTARY_SCALINGS:
        raise UnsupportedError(CLI_UNSUPPORTED, f"rotary_table: scaling {scaling!r}")
    if positions < 0 or rotary_dim < 0 or trained_positions < 0:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "rotary_table: negative size")
    t = out.get("table") if out else None
    if t is None:
        t = torch.empty(positions, rotary_dim // 2, 2, device=device)
    _check_cuda(t, "table", torch.float32)
    if list(t.shape) != [positions, rotary_dim // 2, 2] or not t.is_contiguous():
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "rotary_table: table must be [positions, rotary_dim / 2, 2], packed")
    args = RotaryTableArgs(positions=positions, rotary_dim=rotary_dim, base=base, scaling=ROTARY_SCALINGS[scaling],
                           factor=factor, trained_positions=trained_positions, table=_ptr(t), stream=_stream())
    raise_for(lib.rotary_table(ctypes.byref(args)), "rotary_table")
    return dict(table=t)


def _part(name, t, positions, gain, dim, dtype):
    """What the parts of the rotation verbs share: the shape of `t`, and its words, rows' positions and gain."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{name} must be [rows, heads, {dim}], not {list(shape)}")
    return (shape, _heads(t, name, shape, dtype), 0 if positions is None else
            _vector(positions, name + " positions", shape[0], torch.int32),
            0 if gain is None else _vector(gain, name + "_gain", dim, torch.float32))


_NO_PART = (0,) * 17
_NO_WORKSPACE = 0, 0


def _rotary_call(verb, lead, q_part, k_part, table, interleaved, epsilon, lent, status):
    if table.dtype is not torch.float32 or not table.is_cuda:
        _check_cuda(table, "table", torch.float32)
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2 or not table.is_contiguous():
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"{verb}: table must be [positions, rotary_dim / 2, 2], packed")
    rc = _ROTARY[verb](_pack_rotary.pack(DTYPES[lead.dtype], 1 if interleaved else 0, lead.shape[2], 2 * shape[1],
                                         table.data_ptr(), shape[0], epsilon, *q_part, *k_part, *lent,
                                         status.data_ptr(), _raw_stream(lead)))
    if rc:
        raise_for(rc, verb)


def _rotate_part(out, name, t, positions, gain, dim, dtype, back):
    """(result, the part's 17 words) of a verb with one input and one output."""
    if t is None:
        return None, _NO_PART
    shape, given, pos, g = _part(name, t, positions, gain, dim, dtype)
    y, made = _result(out, name, t, shape)
    if back:
        return y, (shape[0], shape[1], pos, 0, 0, 0, 0, 0, 0, *given, *made, g, 0)
    return y, (shape[0], shape[1], pos, *given, *made, 0, 0, 0, 0, 0, 0, g, 0)


def rotary_heads(q, table, positions=None, k=None, k_positions=None, interleaved=False, out=None, device_status=None,
                 stream=None):
    """Rotates queries [rows, heads, dim] (and keys, of their own rows and heads) by their rows' positions (int32;
    None: row r is at position r), over the first 2 * table.shape[1] elements of each head.  bf16, fp16 or fp32.
    Returns dict(q, k, device_status); out['q'] may be `q` itself."""
    if stream is not None:
        return _on(stream, rotary_heads, locals())
    dtype, dim = q.dtype, _states(q, "q")[2]
    yq, q_part = _rotate_part(out, "q", q, positions, None, dim, dtype, False)
    yk, k_part = _rotate_part(out, "k", k, k_positions, None, dim, dtype, False)
    st = _status(device_status, q)
    _rotary_call("rotary_heads", q, q_part, k_part, table, interleaved, 0.0, _NO_WORKSPACE, st)
    return {"q": yq, "k": yk, "device_status": st}


def rotary_heads_backward(d_q, table, positions=None, d_k=None, k_positions=None, interleaved=False, out=None,
                          device_status=None, stream=None):
    """The gradient of rotary_heads for its inputs.  Returns dict(d_q, d_k, device_status)."""
    if stream is not None:
        return _on(stream, rotary_heads_backward, locals())
    dtype, dim = d_q.dtype, _states(d_q, "d_q")[2]
    xq, q_part = _rotate_part(out, "d_q", d_q, positions, None, dim, dtype, True)
    xk, k_part = _rotate_part(out, "d_k", d_k, k_positions, None, dim, dtype, True)
    st = _status(device_status, d_q)
    _rotary_call("rotary_heads_backward", d_q, q_part, k_part, table, interleaved, 0.0, _NO_WORKSPACE, st)
    return {"d_q": xq, "d_k": xk, "device_status": st}


def norm_rotary_heads(q, table, positions=None, q_gain=None, k=None, k_positions=None, k_gain=None, interleaved=False,
                      epsilon=1e-6, out=None, device_status=None, stream=None):
    """Normalises each head, rotate(gain * x / sqrt(mean(x^2) + epsilon)), of queries and keys in one pass.  Gains
    are fp32 [dim] (None: ones); the rest as in rotary_heads.  Returns dict(q, k, device_status)."""
    if stream is not None:
        return _on(stream, norm_rotary_heads, locals())
    dtype, dim = q.dtype, _states(q, "q")[2]
    yq, q_part = _rotate_part(out, "q", q, positions, q_gain, dim, dtype, False)
    yk, k_part = _rotate_part(out, "k", k, k_positions, k_gain, dim, dtype, False)
    st = _status(device_status, q)
    _rotary_call("norm_rotary_heads", q, q_part, k_part, table, interleaved, epsilon, _NO_WORKSPACE, st)
    return {"q": yq, "k": yk, "device_status": st}


def norm_rotary_heads_backward_workspace_bytes(head_dim):
    return int(lib.norm_rotary_heads_backward_workspace_bytes(head_dim))


def norm_rotary_heads_backward(q, d_q, table, positions=None, q_gain=None, k=None, d_k=None, k_positions=None,
                               k_gain=None, interleaved=False, epsilon=1e-6, out=None, workspace=None,
                               device_status=None, stream=None):
    """The gradients of norm_rotary_heads for its inputs `q`, `k` and its gains, given those of its outputs, `d_q`
    and `d_k`.  A gain's gradient (fp32 [dim]) is None where the gain is.  Returns dict(d_q, d_q_gain, d_k,
    d_k_gain, device_status)."""
    if stream is not None:
        return _on(stream, norm_rotary_heads_backward, locals())
    if (k is None) != (d_k is None):
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, "norm_rotary_heads_backward: k and d_k go together")
    dtype, dim = q.dtype, _states(q, "q")[2]
    xq, q_part, gq = _norm_grad_part(out, "q", q, d_q, positions, q_gain, dim, dtype)
    xk, k_part, gk = _norm_grad_part(out, "k", k, d_k, k_positions, k_gain, dim, dtype)
    st = _status(device_status, q)
    if workspace is None and (gq is not None or gk is not None):
        need = lib.norm_rotary_heads_backward_workspace_bytes(dim)
        workspace = _ws(need, q.device)
        lent = workspace.data_ptr(), need
    else:
        lent = _lent(workspace)
    _rotary_call("norm_rotary_heads_backward", q, q_part, k_part, table, interleaved, epsilon, lent, st)
    return {"d_q": xq, "d_q_gain": gq, "d_k": xk, "d_k_gain": gk, "device_status": st}


def _norm_grad_part(out, name, x, d_y, positions, gain, dim, dtype):
    """(d_x, the part's 17 words, the gain's gradient or None)."""
    if x is None:
        return None, _NO_PART, None
    shape, given, pos, g = _part(name, x, positions, gain, dim, dtype)
    dy = _heads(d_y, "d_" + name, shape, dtype)
    dx, made = _result(out, "d_" + name, x, shape)
    d_gain, dg = None, 0
    if gain is not None:
        d_gain = out.get(f"d_{name}_gain") if out else None
        if d_gain is None:
            d_gain = torch.empty_like(gain)
            dg = d_gain.data_ptr()
        else:
            dg = _vector(d_gain, f"d_{name}_gain", dim, torch.float32)
    return dx, (shape[0], shape[1], pos, *given, 0, 0, 0, *dy, *made, g, dg), d_gain


def _mask(key_mask, rows):
    if key_mask is None:
        return 0
    if key_mask.dtype not in (torch.uint8, torch.bool):
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, "key_mask must be torch.uint8 or torch.bool")
    return _vector(key_mask, "key_mask", rows, key_mask.dtype)


def _attention_sizes(q, q_offsets, k, v, k_offsets, key_mask, scale, max_query_rows, max_key_rows):
    """The struct's words up to `v`, and the number of items."""
    q_shape, k_shape, dtype = _states(q, "q"), _states(k, "k"), q.dtype
    (rows_q, hq, dim), (rows_k, hk, _) = q_shape, k_shape
    if k_offsets is None:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, "k_offsets are needed")
    items = k_offsets.numel() - 1
    max_q = rows_q if max_query_rows is None else max_query_rows
    max_k = rows_k if max_key_rows is None else max_key_rows
    if items < 0 or max_q < 0 or max_k < 0:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, "offsets must be [items + 1], maxima at least 0")
    k_shape = (rows_k, hk, dim)
    return (DTYPES[dtype], items, rows_q, rows_k, _vector(q_offsets, "q_offsets", items + 1, torch.int64),
            _vector(k_offsets, "k_offsets", items + 1, torch.int64), max_q, max_k, hq, hk, dim,
            dim ** -0.5 if scale is None else scale, _mask(key_mask, rows_k), *_heads(q, "q", q_shape, dtype),
            *_heads(k, "k", k_shape, dtype), *_heads(v, "v", k_shape, dtype)), items


def _attention_call(verb, head, tail, workspace, like, status):
    call, workspace_bytes = _ATTENTION[verb]
    ws, ws_bytes = _lent(workspace)
    last = status.data_ptr(), _raw_stream(like)
    args = _pack_attention.pack(*head, *tail, ws, ws_bytes, *last)
    if workspace is None:
        need = workspace_bytes(args)
        if need:
            workspace = _ws(need, like.device)
            args = args[:_ATTENTION_LAST] + _pack_last.pack(workspace.data_ptr(), need, *last)
    rc = call(args)
    if rc:
        raise_for(rc, verb)


def cross_attention_workspace_bytes(q, q_offsets, k, v, k_offsets, key_mask=None, max_query_rows=None,
                                    max_key_rows=None):
    """Workspace bytes for cross_attention of these arguments (their sizes alone count)."""
    head, _ = _attention_sizes(q, q_offsets, k, v, k_offsets, key_mask, 1.0, max_query_rows, max_key_rows)
    return int(_ATTENTION["cross_attention"][1](_pack_attention.pack(*head, *(0,) * 16, 0, 0, 0, 0)))


def cross_attention_backward_workspace_bytes(q, q_offsets, k, v, k_offsets, key_mask=None, max_query_rows=None,
                                             max_key_rows=None):
    """Workspace bytes for cross_attention_backward of these arguments (their sizes alone count)."""
    head, _ = _attention_sizes(q, q_offsets, k, v, k_offsets, key_mask, 1.0, max_query_rows, max_key_rows)
    return int(_ATTENTION["cross_attention_backward"][1](_pack_attention.pack(*head, *(0,) * 16, 0, 0, 0, 0)))


def _lse_ptr(lse, rows, heads):
    if lse is None:
        raise InvalidArgumentError(CLI_INVALID_ARGUMENT, "lse is needed: the forward's, with want_lse")
    if list(lse.shape) != [rows, heads]:
        raise ShapeMismatchError(CLI_SHAPE_MISMATCH, f"lse must be [{rows}, {heads}], packed")
    return _vector(lse, "lse", rows * heads, torch.float32)


def cross_attention(q, q_offsets, k, v, k_offsets, key_mask=None, scale=None, max_query_rows=None, max_key_rows=None,
                    want_lse=True, out=None, workspace=None, device_status=None, stream=None):
    """Every query row of `q` [rows, heads, dim] attends to the states `k`, `v` [states, key_heads, dim] of its item
    on the tapes `q_offsets`, `k_offsets` (int64 [items + 1]).  q_offsets None: all of `q` belongs to every item, and
    the outputs have items * rows rows.  `key_mask` (uint8 or bool [states]) drops states where it is 0; `scale`
    defaults to dim^-0.5; the two maxima bound the items' rows.  They choose the kernels, and their default, the tapes'
    rows, chooses those for long items: pass the longest item's where items are short (2048 items of one query each go
    through tiles of 128 rows otherwise).  bf16 or fp16.  Returns dict(output, lse, device_status), lse fp32 [output
    rows, heads] or None."""
    if stream is not None:
        return _on(stream, cross_attention, locals())
    head, items = _attention_sizes(q, q_offsets, k, v, k_offsets, key_mask, scale, max_query_rows, max_key_rows)
    rows_q, hq, dim = q.shape
    shape = (rows_q if q_offsets is not None else rows_q * items, hq, dim)
    o, made = _result(out, "output", q, shape)
    lse, lse_ptr = None, 0
    if want_lse:
        lse = out.get("lse") if out else None
        if lse is None:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
            lse_ptr = lse.data_ptr()
        else:
            lse_ptr = _lse_ptr(lse, *shape[:2])
    st = _status(device_status, q)
    _attention_call("cross_attention", head, (*made, lse_ptr, *_NO_GRADIENTS), workspace, q, st)
    return {"output": o, "lse": lse, "device_status": st}


def cross_attention_backward(q, q_offsets, k, v, k_offsets, output, lse, d_output, key_mask=None, scale=None,
                             max_query_rows=None, max_key_rows=None, out=None, workspace=None, device_status=None,
                             stream=None):
    """The gradients of cross_attention for `q`, `k` and `v`, given its `output` and `lse` and the output's gradient;
    the rest as there.  Returns dict(d_q, d_k, d_v, device_status)."""
    if stream is not None:
        return _on(stream, cross_attention_backward, locals())
    head, items = _attention_sizes(q, q_offsets, k, v, k_offsets, key_mask, scale, max_query_rows, max_key_rows)
    (rows_q, hq, dim), dtype = q.shape, q.dtype
    shape = (rows_q if q_offsets is not None else rows_q * items, hq, dim)
    (dq, q_made), (dk, k_made), (dv, v_made) = (_result(out, n, t, t.shape)
                                                for n, t in (("d_q", q), ("d_k", k), ("d_v", v)))
    st = _status(device_status, q)
    tail = (*_heads(output, "output", shape, dtype), _lse_ptr(lse, *shape[:2]),
            *_heads(d_output, "d_output", shape, dtype), *q_made, *k_made, *v_made)
    _attention_call("cross_attention_backward", head, tail, workspace, q, st)
    return {"d_q": dq, "d_k": dk, "d_v": dv, "device_status": st}
