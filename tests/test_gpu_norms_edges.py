"""Layer norm, dropout and the residual join past tests/test_gpu_norms.py: the numbers, rows, strides and row counts at which
they can go wrong unseen."""

import pytest
import torch

import norms_reference as ref
from norms_sums import gradient_sums
from test_gpu_norms import BF16, F16, F32, SITE, TYPES, gen, layout, rand, seed_of, vectors, within
from test_gpu_norms import cli as _cli

pytestmark = pytest.mark.gpu
cli = _cli   # the fixture


# ----------------------------------------------------------------------------
# very large numbers
# ----------------------------------------------------------------------------

WIDTHS = [40, 200, 516, 771, 1024, 2100, 4096, 8200]


def with_large(g, rows, width, stream, scale, shift):
    """Ordinary rows, every third of them with one of `scale` around `shift` in its place; which those are."""
    plain = rand(g, rows, width, dtype=stream)
    large = torch.arange(rows, device="cuda") % 3 == 1
    x = plain.clone()
    x[large] = rand(g, int(large.sum()), width, scale=scale, shift=shift).to(stream)
    return plain, x, large


@pytest.mark.parametrize("types", [t for t in TYPES if t[1] != F16])
@pytest.mark.parametrize("scale, shift", [(1e21, 0.0), (1e21, 1e22), (1e27, 1e27), (1e28, 0.0), (1e28, 1e29), (1e30, 0.0),
                                          (1e30, 1e30), (1e32, 1e33), (1e35, 0.0)])
def test_rows_whose_squares_pass_the_range(cli, types, scale, shift):
    """They have n = 0: the output is the bias, the norm's part of the gradient 0, and nothing goes to the gain's."""
    dtype, stream = types
    for width in WIDTHS:
        g = gen(width)
        plain, x, large = with_large(g, 31, width, stream, scale, shift)
        assert torch.isfinite(x).all() and torch.isfinite(x.float().sum(1)).all()
        d_y, d_sum = rand(g, 31, width, dtype=dtype), rand(g, 31, width, dtype=stream)
        gain, bias = vectors(g, width)
        y, want = cli.layer_norm(x, gain, bias, dtype=dtype)["output"], cli.layer_norm(plain, gain, bias, dtype=dtype)["output"]
        assert torch.equal(y[~large], want[~large]) and (y[large] == bias.to(dtype)).all(), width
        b, want = cli.layer_norm_backward(x, d_y, gain, bias), cli.layer_norm_backward(plain, d_y, gain, bias)
        assert torch.equal(b["d_x"][~large], want["d_x"][~large]) and not b["d_x"][large].any(), width
        assert torch.equal(b["d_bias"], want["d_bias"]), width
        none = d_y.clone()
        none[large] = 0.0
        assert torch.equal(b["d_gain"], cli.layer_norm_backward(plain, none, gain, bias)["d_gain"]), width
        # joined
        branch = rand(g, 31, width, dtype=dtype)
        f = cli.dropout_layer_norm(branch, x, 0.2, seed_of(), SITE, gain, bias)
        want = cli.dropout_layer_norm(branch, plain, 0.2, seed_of(), SITE, gain, bias)
        assert torch.equal(f["output"][~large], want["output"][~large]) and (f["output"][large] == bias.to(dtype)).all(), width
        b = cli.dropout_layer_norm_backward(x, d_y, 0.2, seed_of(), SITE, d_sum, gain, bias)
        want = cli.dropout_layer_norm_backward(plain, d_y, 0.2, seed_of(), SITE, d_sum, gain, bias)
        assert torch.equal(b["d_residual"][~large], want["d_residual"][~large]), width
        assert torch.equal(b["d_residual"][large], d_sum[large]), width
        through = cli.dropout(d_sum, 0.2, seed_of(), SITE)["output"].to(dtype)
        assert torch.equal(b["d_x"][large], through[large]) and torch.equal(b["d_x"][~large], want["d_x"][~large]), width
        assert torch.equal(b["d_bias"], want["d_bias"]), width


@pytest.mark.parametrize("types", [t for t in TYPES if t[1] != F16])
def test_rows_whose_sum_passes_the_range(cli, types):
    """They are NaN, and no other row is."""
    dtype, stream = types
    for width in WIDTHS[2:]:
        g = gen(width)
        plain, x, large = with_large(g, 31, width, stream, 1e35, 2e36)
        assert torch.isfinite(x).all()
        d_y = rand(g, 31, width, dtype=dtype)
        gain, bias = vectors(g, width)
        y, want = cli.layer_norm(x, gain, bias, dtype=dtype)["output"], cli.layer_norm(plain, gain, bias, dtype=dtype)["output"]
        assert torch.equal(y[~large], want[~large]) and y[large].isnan().all(), width
        d, want = cli.layer_norm_backward(x, d_y, gain)["d_x"], cli.layer_norm_backward(plain, d_y, gain)["d_x"]
        assert torch.equal(d[~large], want[~large]) and d[large].isnan().all(), width


def test_large_rows_within_the_range(cli):
    """10^17: the squares of 8200 such sum to 8 * 10^37."""
    for width in WIDTHS:
        g = gen(width)
        x, d_y = rand(g, 30, width, scale=1e17, shift=3e17), rand(g, 30, width)
        gain, bias = vectors(g, width)
        within(cli.layer_norm(x, gain, bias)["output"], ref.layer_norm(x, gain, bias, 1e-5, F32), width)
        b, want = cli.layer_norm_backward(x, d_y, gain, bias), ref.layer_norm_backward(x, d_y, gain, 1e-5, F32)
        for name in ("d_x", "d_gain", "d_bias"):
            within(b[name], want[name], f"{width} {name}")


# ----------------------------------------------------------------------------
# one row of several
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("width, gap", [(1024, 5), (1024, 2), (1024, 4), (1024, 8), (200, 1), (517, 3), (4096, 6), (8200, 3)])
def test_a_row_alone_is_the_row_beside_others(cli, types, width, gap):
    """Rows of a wider buffer, whose distance decides how they are moved: each alone gives the bits it gives among the others."""
    dtype, stream = types
    g = gen(width + gap)
    rows = 9

    def wide(t):
        buffer = torch.zeros(rows, width + gap, dtype=t.dtype, device="cuda")
        buffer[:, :width] = t
        return buffer[:, :width]
    x, res = wide(rand(g, rows, width, dtype=dtype)), wide(rand(g, rows, width, dtype=stream, shift=0.5))
    d_y, d_sum = wide(rand(g, rows, width, dtype=dtype)), wide(rand(g, rows, width, dtype=stream))
    gain, bias = vectors(g, width)

    def calls(s):
        f = cli.dropout_layer_norm(x[s], res[s], 0.0, None, 0, gain, bias)
        b = cli.dropout_layer_norm_backward(res[s], d_y[s], 0.0, None, 0, d_sum[s], gain, bias)
        return {"norm": cli.layer_norm(res[s], gain, bias, dtype=dtype)["output"], "sum": f["sum"], "joined": f["output"],
                "d_x": cli.layer_norm_backward(res[s], d_y[s], gain)["d_x"], "d_residual": b["d_residual"], "d_branch": b["d_x"]}
    want = calls(slice(0, rows))
    for k in range(rows):
        for n in (1, 2):
            for name, got in calls(slice(k, k + n)).items():
                assert torch.equal(got, want[name][k:k + n]), (name, k, n)


# ----------------------------------------------------------------------------
# the sums over rows
# ----------------------------------------------------------------------------

MANY = [(257, 64), (20011, 64), (9000, 200), (5000, 1024), (3001, 517), (4000, 1100), (2500, 3200), (1200, 8192), (700, 12000)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows, width", MANY)
def test_every_row_is_counted_once(cli, types, rows, width):
    """Column c of the gradient is bit c of the row's number, or 1: whole numbers below 2^24, which add up exactly in any
    order.  A row lost or taken twice shows in the ones, one in another's place in the bits."""
    dtype, stream = types
    g = gen(rows)
    x = rand(g, rows, width, dtype=stream)
    gain, bias = vectors(g, width)
    bits = torch.ones(rows, width, dtype=torch.int64, device="cuda")
    for c in range(0, width - 17, 32):
        for k in range(16):
            bits[:, c + k] = torch.arange(rows, device="cuda") >> k & 1
    d_y = bits.to(dtype)
    want = bits.sum(0).float()
    assert torch.equal(cli.layer_norm_backward(x, d_y, gain, bias)["d_bias"], want)
    assert torch.equal(cli.dropout_layer_norm_backward(x, d_y, 0.1, seed_of(), gain=gain, bias=bias)["d_bias"], want)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows, width", [(20011, 64), (5000, 1024), (3001, 517), (1200, 8192)])
def test_gradients_of_one_row(cli, types, rows, width):
    """One row's d_y is 1, the others' 0: the bias's gradient is 1 and the gain's that row's n."""
    dtype, stream = types
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    x = rand(gen(rows), rows, width, dtype=stream)
    one, none = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    for row in (0, 1, 31, 32, sms - 1, sms, 2 * sms - 1, 2 * sms, rows // 2, rows - 2, rows - 1):
        d_y = torch.zeros(rows, width, dtype=dtype, device="cuda")
        d_y[row] = 1.0
        want = ref.layer_norm(x[row:row + 1], one, none, 1e-5, F32)
        for b in (cli.layer_norm_backward(x, d_y, one, none),
                  cli.dropout_layer_norm_backward(x, d_y, 0.1, seed_of(), gain=one, bias=none)):
            assert (b["d_bias"] == 1.0).all(), row
            within(b["d_gain"], (want[0][0], want[1][0]), row)


def test_the_last_of_rows_past_32_bits(cli):
    """Rows whose element offset passes 2^32: each is counted once, and the last ones' gradients are their own."""
    rows, width = 2200000, 2048
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    d_y = torch.ones(rows, width, dtype=BF16, device="cuda")
    one, none = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    x[-1] = rand(gen(8), width, dtype=BF16)
    b = cli.layer_norm_backward(x, d_y, one, none)
    assert (b["d_bias"] == rows).all()
    want = ref.layer_norm(x[-1:], one, none, 1e-5, F32)
    within(b["d_gain"], (want[0][0], want[1][0]), "d_gain")   # the other rows' n is 0


# ----------------------------------------------------------------------------
# many rows of every pair of types, in every layout
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["packed", "padded", "fours", "odd"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows, width", [(20011, 24), (9000, 200), (3001, 517), (4000, 1100), (1500, 2056), (700, 8200)])
def test_many_rows(cli, types, kind, rows, width):
    """A team takes several rows, and its copies' places go round: against the reference, sums over rows to within the
    additions that they have in series."""
    dtype, stream = types
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = gen(rows + width)
    x, res = rand(g, rows, width, dtype=dtype), rand(g, rows, width, dtype=stream, shift=0.5)
    d_y, d_sum = rand(g, rows, width, dtype=dtype), rand(g, rows, width, dtype=stream)
    gain, bias = vectors(g, width)
    at = [layout(t, kind) for t in (x, res, d_y, d_sum)]
    within(cli.layer_norm(at[1], gain, bias, dtype=dtype)["output"], ref.layer_norm(res, gain, bias, 1e-5, dtype), "output")
    b, want = cli.layer_norm_backward(at[1], at[2], gain, bias), ref.layer_norm_backward(res, d_y, gain, 1e-5, stream)
    within(b["d_x"], want["d_x"], "d_x")
    for name, value in gradient_sums(res, d_y, sms).items():
        within(b[name], value, name)
    kept = 2.0 ** 32 / (2 ** 32 - int(0.2 * 2 ** 32))
    factor = (cli.dropout(torch.ones(rows, width, device="cuda"), 0.2, seed_of(), SITE)["output"] != 0) * kept
    within(cli.dropout(at[0], 0.2, seed_of(), SITE)["output"], ref.dropout(x, factor, dtype), "dropped")
    f = cli.dropout_layer_norm(at[0], at[1], 0.2, seed_of(), SITE, gain, bias)
    want = ref.join(x, res, factor, gain, bias, 1e-5)
    within(f["sum"], want["sum"], "sum")
    within(f["output"], want["output"], "joined output")
    b = cli.dropout_layer_norm_backward(layout(f["sum"], kind), at[2], 0.2, seed_of(), SITE, at[3], gain, bias)
    want = ref.join_backward(f["sum"], d_y, d_sum, factor, gain, 1e-5)
    for name in ("d_residual", "d_x"):
        within(b[name], want[name], "joined " + name)
    for name, value in gradient_sums(f["sum"], d_y, sms).items():
        within(b[name], value, "joined " + name)


# ----------------------------------------------------------------------------
# columns of one buffer, and no workspace
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 2, 700])
@pytest.mark.parametrize("width, gap", [(64, 0), (61, 0), (200, 3), (1024, 8)])
def test_columns_of_one_buffer(cli, rows, width, gap):
    """Input and output side by side in the same rows, either first, are apart: as in buffers of their own, and what lies
    between them stays."""
    g = gen(width + rows)
    x, other = rand(g, rows, width, dtype=BF16), rand(g, rows, width, dtype=BF16)
    gain, bias = vectors(g, width)
    seed = seed_of()
    sums = cli.dropout_layer_norm(x, other, 0.3, seed, SITE, gain, bias)
    for first in (True, False):
        def call(into, verb):
            buffer = torch.full((rows, 2 * width + gap), 7.0, dtype=BF16, device="cuda")
            a, b = buffer[:, :width], buffer[:, width + gap:]
            src, dst = (a, b) if first else (b, a)
            src.copy_(into)
            verb(src, dst)
            assert torch.equal(src, into) and (buffer[:, width:width + gap] == 7.0).all()
            return dst
        got = call(x, lambda s, d: cli.layer_norm(s, gain, bias, out={"output": d}))
        within(got, ref.layer_norm(x, gain, bias, 1e-5, BF16), "norm")
        got = call(x, lambda s, d: cli.dropout(s, 0.3, seed, SITE, out={"output": d}))
        assert torch.equal(got, cli.dropout(x, 0.3, seed, SITE)["output"])
        got = call(other, lambda s, d: cli.dropout_layer_norm(x, s, 0.3, seed, SITE, gain, bias, out={"sum": d}))
        assert torch.equal(got, sums["sum"])
        got = call(x, lambda s, d: cli.layer_norm_backward(s, other, gain, out={"d_x": d}))
        within(got, ref.layer_norm_backward(x, other, gain, 1e-5, BF16)["d_x"], "d_x")
        got = call(other, lambda s, d: cli.dropout_backward(s, 0.3, seed, SITE, out={"d_x": d}))
        assert torch.equal(got, cli.dropout(other, 0.3, seed, SITE)["output"])


def test_gradients_of_few_rows_without_a_workspace(cli):
    """A NULL workspace is taken where none is needed, and refused where one is."""
    from contrastive_late_interaction_gb300 import _binding as b
    import ctypes
    for rows in (16, 17):
        x, d_y = rand(gen(rows), rows, 1024, dtype=BF16), rand(gen(1), rows, 1024, dtype=BF16)
        gain, bias = vectors(gen(2), 1024)
        want = cli.layer_norm_backward(x, d_y, gain, bias)
        out = {n: torch.zeros_like(t) for n, t in want.items()}
        R = b.RowsArgs
        args = b.LayerNormArgs(x_dtype=0, y_dtype=0, rows=rows, width=1024, x=R(x.data_ptr(), 1024), d_y=R(d_y.data_ptr(), 1024),
                               d_x=R(out["d_x"].data_ptr(), 1024), gain=gain.data_ptr(), d_gain=out["d_gain"].data_ptr(),
                               d_bias=out["d_bias"].data_ptr(), epsilon=1e-5,
                               stream=torch.cuda.current_stream().cuda_stream)
        got = b.lib.layer_norm_backward(ctypes.byref(args))
        if rows == 16:
            assert got == 0 and all(torch.equal(out[n], want[n]) for n in want)
        else:
            assert got == b.CLI_INVALID_ARGUMENT
