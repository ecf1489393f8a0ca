"""The 64-bit reference of layer norm, dropout and the residual join against differences of itself and published words of
the generator, and the refusals of their entry points: no CUDA call is made."""

import ctypes

import pytest
import torch

import norms_reference as ref

A = 1 << 36   # fake device addresses, far apart


@pytest.fixture(scope="module")
def b():
    from contrastive_late_interaction_gb300 import build
    build.build()
    from contrastive_late_interaction_gb300 import _binding
    return _binding


# ----------------------------------------------------------------------------
# the reference
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("counter, key, want", [   # the vectors published with the generator
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([2 ** 32 - 1] * 4, [2 ** 32 - 1] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator(counter, key, want):
    assert ref.philox(counter, key) == want


@pytest.mark.parametrize("onward", [False, True])
def test_gradients_match_differences(onward):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, res, gain, bias, d_y = r(4, 9), r(4, 9), r(9), r(9), r(4, 9)
    d_sum = r(4, 9) if onward else None
    factor = ref.factors(4, 9, 0.4, 7, 8, 9)
    assert 0 < int((factor == 0).sum()) < 36

    def loss(x, res, gain, bias):
        f = ref.join(x, res, factor, gain, bias, 1e-3)
        return (f["output"][0] * d_y).sum() + ((f["sum"][0] * d_sum).sum() if onward else 0.0)
    total = ref.join(x, res, factor, gain, bias, 1e-3)["sum"][0]
    got = ref.join_backward(total, d_y, d_sum, factor, gain, 1e-3)
    for i, name in enumerate(("d_x", "d_residual", "d_gain", "d_bias")):
        args = [x, res, gain, bias]
        direction, h = r(*args[i].shape), 1e-5
        plus, minus = [[v + s * h * direction if j == i else v for j, v in enumerate(args)] for s in (1, -1)]
        want = (loss(*plus) - loss(*minus)) / (2 * h)
        assert abs((got[name][0] * direction).sum() - want) <= 1e-7 * max(1.0, abs(want)), name


# ----------------------------------------------------------------------------
# refusals
# ----------------------------------------------------------------------------

def rows(b, place, stride=64, off=0):
    return b.RowsArgs(A * place + off, stride)


def norm_args(b, **over):
    args = dict(x_dtype=0, y_dtype=0, rows=1000, width=64, x=rows(b, 1), y=rows(b, 2), d_y=rows(b, 3), d_x=rows(b, 4),
                gain=A * 5, bias=A * 6, d_gain=A * 7, d_bias=A * 8, epsilon=1e-5, workspace=A * 9,
                workspace_bytes=b.lib.layer_norm_backward_workspace_bytes(1000, 64))
    args.update(over)
    return b.LayerNormArgs(**args)


def dropout_args(b, **over):
    args = dict(dtype=0, rows=1000, width=64, x=rows(b, 1), y=rows(b, 2), d_y=rows(b, 3), d_x=rows(b, 4),
                mask=b.DropoutMaskArgs(0.1, A * 10, 0))
    args.update(over)
    return b.DropoutArgs(**args)


def join_args(b, **over):
    args = dict(dtype=0, stream_dtype=0, rows=1000, width=64, x=rows(b, 1), residual=rows(b, 2), sum=rows(b, 3),
                y=rows(b, 4), d_y=rows(b, 11), d_sum=rows(b, 12), d_residual=rows(b, 13), d_x=rows(b, 14),
                mask=b.DropoutMaskArgs(0.1, A * 10, 0), gain=A * 5, bias=A * 6, d_gain=A * 7, d_bias=A * 8, epsilon=1e-5,
                workspace=A * 9, workspace_bytes=b.lib.layer_norm_backward_workspace_bytes(1000, 64))
    args.update(over)
    return b.DropoutLayerNormArgs(**args)


MAKE = {"layer_norm": norm_args, "layer_norm_backward": norm_args, "dropout": dropout_args, "dropout_backward": dropout_args,
        "dropout_layer_norm": join_args, "dropout_layer_norm_backward": join_args}
NORMS = [v for v in MAKE if "norm" in v]
MASKED = [v for v in MAKE if "dropout" in v]
BACKWARD_NORMS = ["layer_norm_backward", "dropout_layer_norm_backward"]


def status(b, verb, **over):
    return getattr(b.lib, verb)(ctypes.byref(MAKE[verb](b, **over)))


@pytest.mark.parametrize("verb", MAKE)
def test_sizes_and_types(b, verb):
    assert getattr(b.lib, verb)(None) == b.CLI_INVALID_ARGUMENT
    assert status(b, verb, width=0) == b.CLI_SHAPE_MISMATCH
    assert status(b, verb, width=16385) == b.CLI_UNSUPPORTED
    assert status(b, verb, rows=1 << 31) == b.CLI_SHAPE_MISMATCH
    for name in ("dtype", "y_dtype", "x_dtype", "stream_dtype"):
        if name in dict(MAKE[verb](b)._fields_):
            assert status(b, verb, **{name: 3}) == b.CLI_UNSUPPORTED
            assert status(b, verb, **{name: -1}) == b.CLI_UNSUPPORTED


@pytest.mark.parametrize("one, other", [(0, 1), (1, 0), (2, 0), (2, 1)])   # (out, stream): only fp32 streams mix
def test_mixed_types(b, one, other):
    for verb in NORMS:
        names = ("y_dtype", "x_dtype") if verb.startswith("layer") else ("dtype", "stream_dtype")
        assert status(b, verb, **dict(zip(names, (one, other)))) == b.CLI_UNSUPPORTED, verb


@pytest.mark.parametrize("epsilon", [0.0, -1e-5, float("inf"), float("nan")])
def test_epsilon(b, epsilon):
    for verb in NORMS:
        assert status(b, verb, epsilon=epsilon) == b.CLI_INVALID_ARGUMENT, verb


@pytest.mark.parametrize("mask", [(-1e-9, A * 10, 0), (1.0, A * 10, 0), (float("nan"), A * 10, 0), (0.1, None, 0),
                                  (1e-300, None, 0), (0.1, A * 10 + 4, 0), (0.1, A * 10, 65536)])
def test_masks(b, mask):
    for verb in MASKED:
        assert status(b, verb, mask=b.DropoutMaskArgs(*mask)) == b.CLI_INVALID_ARGUMENT, verb


READS = {"layer_norm": ["x"], "layer_norm_backward": ["x", "d_y"], "dropout": ["x"], "dropout_backward": ["d_y"],
         "dropout_layer_norm": ["x", "residual"], "dropout_layer_norm_backward": ["sum", "d_y", "d_sum"]}
WRITES = {"layer_norm": ["y"], "layer_norm_backward": ["d_x"], "dropout": ["y"], "dropout_backward": ["d_x"],
          "dropout_layer_norm": ["y", "sum"], "dropout_layer_norm_backward": ["d_residual", "d_x"]}
OPTIONAL = [("dropout_layer_norm", "sum"), ("dropout_layer_norm_backward", "d_sum"), ("dropout_layer_norm_backward", "d_x")]


@pytest.mark.parametrize("verb", MAKE)
def test_matrices(b, verb):
    for name in READS[verb] + WRITES[verb]:
        if (verb, name) not in OPTIONAL:
            assert status(b, verb, **{name: b.RowsArgs(None, 64)}) == b.CLI_INVALID_ARGUMENT, name
        assert status(b, verb, **{name: rows(b, 20, off=1)}) == b.CLI_INVALID_ARGUMENT, name      # not on an element
        for stride in (1 << 40, (1 << 63) + 64, 2 ** 64 - 64):
            assert status(b, verb, **{name: rows(b, 20, stride)}) == b.CLI_SHAPE_MISMATCH, name
    for name in WRITES[verb]:
        assert status(b, verb, **{name: rows(b, 20, 63)}) == b.CLI_SHAPE_MISMATCH, name           # rows over one another
        assert status(b, verb, **{name: rows(b, 20, 0)}) == b.CLI_SHAPE_MISMATCH, name


@pytest.mark.parametrize("verb", MAKE)
def test_outputs_over_inputs(b, verb):
    for out in WRITES[verb]:
        for name in READS[verb]:
            place = getattr(MAKE[verb](b), name).data
            for off, stride in ((2, 64), (0, 72), (128, 64), (-128, 64)):
                assert status(b, verb, **{out: b.RowsArgs(place + off, stride)}) == b.CLI_INVALID_ARGUMENT, (out, name, off)
        if "dropout" in verb:   # the seed within an output
            assert status(b, verb, mask=b.DropoutMaskArgs(0.1, getattr(MAKE[verb](b), out).data + 8, 0)) == b.CLI_INVALID_ARGUMENT
        if "norm" in verb:
            place = getattr(MAKE[verb](b), out).data + 64
            for name in ("gain",) + (("d_gain", "d_bias") if verb in BACKWARD_NORMS else ("bias",)):
                assert status(b, verb, **{name: place}) == b.CLI_INVALID_ARGUMENT, (out, name)
    if len(WRITES[verb]) == 2:
        first, second = WRITES[verb]
        assert status(b, verb, **{second: getattr(MAKE[verb](b), first)}) == b.CLI_INVALID_ARGUMENT


def test_in_place_needs_one_type(b):
    x = rows(b, 1)
    assert status(b, "layer_norm", x_dtype=2, x=x, y=x) == b.CLI_INVALID_ARGUMENT
    r = rows(b, 3)
    assert status(b, "dropout_layer_norm_backward", stream_dtype=2, sum=r, d_x=r) == b.CLI_INVALID_ARGUMENT


def test_columns_of_one_buffer_are_apart(b):
    """Halves of the same rows: not refused as overlapping (without a GPU the call ends with a device error, or not at all)."""
    for verb, name, other in (("layer_norm", "x", "y"), ("dropout", "x", "y"), ("dropout_layer_norm", "residual", "sum")):
        assert status(b, verb, rows=0, **{name: rows(b, 1, 128), other: rows(b, 1, 128, 128)}) == b.CLI_OK
        got = status(b, verb, **{name: rows(b, 1, 128), other: rows(b, 1, 128, 126)})
        assert got == b.CLI_INVALID_ARGUMENT, verb


@pytest.mark.parametrize("verb", BACKWARD_NORMS)
def test_workspace(b, verb):
    need = b.lib.layer_norm_backward_workspace_bytes(1000, 64)
    assert need % 256 == 0 and need > 0
    for over in (dict(workspace=None), dict(workspace=A * 9 + 8), dict(workspace_bytes=need - 1)):
        assert status(b, verb, **over) == b.CLI_INVALID_ARGUMENT
    assert status(b, verb, d_bias=A * 7) == b.CLI_INVALID_ARGUMENT            # the same vector twice
    assert status(b, verb, d_gain=A * 9 + 4) == b.CLI_INVALID_ARGUMENT        # inside the workspace
    for name in ("gain", "d_gain", "d_bias"):
        assert status(b, verb, **{name: A * 15 + 2}) == b.CLI_INVALID_ARGUMENT
    few = dict(rows=16, width=1024, workspace=None)                           # one block: no partial sums
    assert b.lib.layer_norm_backward_workspace_bytes(16, 1024) == 0 < b.lib.layer_norm_backward_workspace_bytes(17, 1024)
    assert b.lib.layer_norm_backward_workspace_bytes(256, 1) == 0 < b.lib.layer_norm_backward_workspace_bytes(257, 1)
    apart = {n: b.RowsArgs(A * (30 + i), 1024) for i, n in enumerate(READS[verb] + WRITES[verb])}
    assert status(b, verb, **few, **apart) not in (b.CLI_INVALID_ARGUMENT, b.CLI_SHAPE_MISMATCH)
    assert b.lib.layer_norm_backward_workspace_bytes(100, 0) == 0
    assert b.lib.layer_norm_backward_workspace_bytes(100, 16385) == 0
    assert b.lib.layer_norm_backward_workspace_bytes(1 << 31, 64) == 0


def test_calls_on_no_rows(b):
    for verb in ("layer_norm", "dropout", "dropout_backward", "dropout_layer_norm"):
        none = {n: b.RowsArgs(None, 64) for n in READS[verb] + WRITES[verb]}
        assert status(b, verb, rows=0, **none) == b.CLI_OK, verb
