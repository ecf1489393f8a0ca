"""The 64-bit reference of the token-state operators against differences of itself, closed forms and a second
formulation (no GPU), and the refusals of their entry points."""

import ctypes

import numpy as np
import pytest
import torch

import states_reference as ref


def differences(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("shared", [False, True])
def test_attention_gradients_match_differences(shared):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q_len, k_len = [3, 0, 2], [4, 2, 0]
    rows = 2 if shared else 5
    q, k, v = r(rows, 4, 8), r(6, 2, 8), r(6, 2, 8)
    mask = torch.tensor([1, 0, 1, 1, 1, 1], dtype=torch.uint8)
    d_o = r(rows * 3 if shared else rows, 4, 8)

    def loss(q, k, v):
        o = ref.attention(q, k, v, None if shared else q_len, k_len, 0.4, mask, shared=shared)["output"][0]
        return (o * d_o).sum()

    a = ref.attention(q, k, v, None if shared else q_len, k_len, 0.4, mask, d_o, shared=shared)
    for i, name in enumerate(("d_q", "d_k", "d_v")):
        args = [q, k, v]
        direction = r(*args[i].shape)

        def at(x):
            return loss(*[x if j == i else args[j] for j in range(3)])
        want = differences(at, args[i], direction)
        assert abs((a[name][0] * direction).sum() - want) <= 1e-7 * max(1.0, abs(want)), name
    assert torch.all(a["d_k"][0][1] == 0) and torch.all(a["d_v"][0][1] == 0)      # dropped


def test_attention_of_equal_states_is_their_value():
    v = torch.randn(1, 2, 16, dtype=torch.float64)
    a = ref.attention(torch.randn(3, 2, 16), torch.ones(7, 2, 16), v.expand(7, 2, 16), [3], [7], 1.0)
    assert torch.allclose(a["output"][0], v.expand(3, 2, 16), atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(interleaved):
    tab = ref.table(64, 16)
    x = torch.randn(5, 2, 24, dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, 33, 63])
    y, _ = ref.rotate(x, tab, pos, interleaved)
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
    assert torch.equal(y[..., 16:], x[..., 16:]) and torch.allclose(y[0], x[0])
    back, _ = ref.rotate(y, tab, pos, interleaved, back=True)
    assert torch.allclose(back, x, atol=1e-6)
    a, b = x[:1], x[1:2]
    dots = [(ref.rotate(a, tab, torch.tensor([p]), interleaved)[0] *
             ref.rotate(b, tab, torch.tensor([p + 5]), interleaved)[0]).sum() for p in (0, 11, 40)]
    assert np.allclose(dots, dots[0], atol=1e-5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rotation_gradients_match_differences(interleaved):
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    tab, pos = ref.table(32, 12), torch.tensor([3, 0, 31])
    x, gain, dy = r(3, 2, 16), 1 + 0.3 * r(16), r(3, 2, 16)
    dx, _, dg, _ = ref.norm_rotate_backward(x, dy, gain, tab, pos, interleaved, 1e-3)
    fx = lambda x: (ref.norm_rotate(x, gain, tab, pos, interleaved, 1e-3)[0] * dy).sum()  # noqa: E731
    fg = lambda gain: (ref.norm_rotate(x, gain, tab, pos, interleaved, 1e-3)[0] * dy).sum()  # noqa: E731
    ex, eg = r(3, 2, 16), r(16)
    assert abs((dx * ex).sum() - differences(fx, x, ex)) <= 1e-7 * 10
    assert abs((dg * eg).sum() - differences(fg, gain, eg)) <= 1e-7 * 10


# ----------------------------------------------------------------------------
# refusals: every call returns before any CUDA call, so the addresses are never read
# ----------------------------------------------------------------------------

A = 1 << 36


@pytest.fixture(scope="module")
def b():
    from contrastive_late_interaction_gb300 import build
    build.build()
    from contrastive_late_interaction_gb300 import _binding
    return _binding


def heads(b, place, rows, heads_, dim):
    return b.HeadsArgs(A * place if place else None, heads_ * dim, dim)


def rotary_args(b, **over):
    part = dict(rows=100, heads=4, positions=A * 3, x=heads(b, 4, 100, 4, 64), y=heads(b, 5, 100, 4, 64),
                d_y=heads(b, 6, 100, 4, 64), d_x=heads(b, 7, 100, 4, 64), gain=A * 8, d_gain=A * 9)
    part.update(over.pop("part", {}))
    args = dict(dtype=0, interleaved=0, head_dim=64, rotary_dim=64, table=A * 1, table_rows=4096, epsilon=1e-6,
                q=b.RotaryPartArgs(**part), k=b.RotaryPartArgs(), workspace=A * 10, workspace_bytes=1 << 24,
                device_status=A * 2, stream=None)
    args.update(over)
    return b.RotaryArgs(**args)


@pytest.mark.parametrize("over, status", [
    (dict(dtype=3), "CLI_UNSUPPORTED"), (dict(head_dim=60), "CLI_SHAPE_MISMATCH"),
    (dict(head_dim=264, rotary_dim=64), "CLI_UNSUPPORTED"), (dict(rotary_dim=63), "CLI_SHAPE_MISMATCH"),
    (dict(rotary_dim=66), "CLI_SHAPE_MISMATCH"), (dict(rotary_dim=0), "CLI_SHAPE_MISMATCH"),
    (dict(table=None), "CLI_INVALID_ARGUMENT"), (dict(table=A + 4), "CLI_INVALID_ARGUMENT"),
    (dict(table_rows=0), "CLI_SHAPE_MISMATCH"), (dict(device_status=None), "CLI_INVALID_ARGUMENT"),
    (dict(device_status=A + 64), "CLI_INVALID_ARGUMENT"),      # within the table
    (dict(part=dict(rows=1 << 31)), "CLI_SHAPE_MISMATCH"), (dict(part=dict(heads=0)), "CLI_SHAPE_MISMATCH"),
    (dict(part=dict(heads=65536)), "CLI_SHAPE_MISMATCH"), (dict(part=dict(positions=A * 3 + 2)), "CLI_INVALID_ARGUMENT"),
])
def test_rotary_refusals(b, over, status):
    for verb in ("rotary_heads", "rotary_heads_backward", "norm_rotary_heads", "norm_rotary_heads_backward"):
        assert getattr(b.lib, verb)(ctypes.byref(rotary_args(b, **dict(over)))) == getattr(b, status), verb


def test_rotary_refuses_bad_matrices(b):
    call = lambda **part: b.lib.rotary_heads(ctypes.byref(rotary_args(b, part=part)))  # noqa: E731
    H = b.HeadsArgs
    assert call(x=H(None, 256, 64)) == b.CLI_INVALID_ARGUMENT
    assert call(x=H(A * 4 + 8, 256, 64)) == b.CLI_INVALID_ARGUMENT          # 16-byte alignment
    assert call(x=H(A * 4, 252, 64)) == b.CLI_SHAPE_MISMATCH                # strides of 16 bytes
    assert call(y=H(A * 5, 192, 64)) == b.CLI_SHAPE_MISMATCH                # rows that overlap in an output
    assert call(y=H(A * 5, 0, 64)) == b.CLI_SHAPE_MISMATCH
    assert call(y=H(A * 4 + 512, 256, 64)) == b.CLI_INVALID_ARGUMENT        # output over input, not in place
    assert call(y=H(A * 4 + 64, 512, 64), x=H(A * 4, 512, 64)) == b.CLI_INVALID_ARGUMENT
    assert call(y=H(A * 1, 256, 64)) == b.CLI_INVALID_ARGUMENT              # output over the table
    assert b.lib.rotary_heads(None) == b.CLI_INVALID_ARGUMENT
    grad = lambda **over: b.lib.norm_rotary_heads_backward(ctypes.byref(rotary_args(b, **over)))  # noqa: E731
    assert grad(epsilon=0.0) == b.CLI_INVALID_ARGUMENT
    assert grad(epsilon=float("nan")) == b.CLI_INVALID_ARGUMENT
    assert grad(workspace=None) == b.CLI_INVALID_ARGUMENT
    assert grad(workspace_bytes=100) == b.CLI_INVALID_ARGUMENT
    assert grad(workspace=A * 10 + 128) == b.CLI_INVALID_ARGUMENT


def test_rotary_table_refusals(b):
    def call(**over):
        args = dict(positions=100, rotary_dim=64, base=10000.0, scaling=0, factor=1.0, trained_positions=0,
                    table=A, stream=None)
        args.update(over)
        return b.lib.rotary_table(ctypes.byref(b.RotaryTableArgs(**args)))
    assert call(table=None) == b.CLI_INVALID_ARGUMENT and call(table=A + 8) == b.CLI_INVALID_ARGUMENT
    assert call(positions=0) == b.CLI_SHAPE_MISMATCH and call(rotary_dim=7) == b.CLI_SHAPE_MISMATCH
    assert call(rotary_dim=258) == b.CLI_UNSUPPORTED and call(scaling=4) == b.CLI_UNSUPPORTED
    assert call(base=1.0) == b.CLI_INVALID_ARGUMENT and call(factor=0.5) == b.CLI_INVALID_ARGUMENT
    assert call(base=float("nan")) == b.CLI_INVALID_ARGUMENT and call(factor=float("inf")) == b.CLI_INVALID_ARGUMENT
    assert call(scaling=3) == b.CLI_INVALID_ARGUMENT          # YARN without its trained length
    assert call(scaling=2, rotary_dim=2) == b.CLI_SHAPE_MISMATCH


def attention_args(b, **over):
    hq, hk, d = over.get("query_heads", 8), over.get("key_heads", 2), over.get("head_dim", 64)
    args = dict(dtype=0, items=4, query_rows=100, key_rows=1000, query_offsets=A * 1, key_offsets=A * 2,
                max_query_rows=100, max_key_rows=1000, query_heads=hq, key_heads=hk, head_dim=d, scale=0.125,
                key_mask=None, q=heads(b, 3, 100, hq, d), k=heads(b, 4, 1000, hk, d), v=heads(b, 5, 1000, hk, d),
                output=heads(b, 6, 100, hq, d), lse=A * 7, d_output=heads(b, 8, 100, hq, d),
                d_q=heads(b, 9, 100, hq, d), d_k=heads(b, 10, 1000, hk, d), d_v=heads(b, 11, 1000, hk, d),
                workspace=A * 12, workspace_bytes=1 << 34, device_status=A * 13, stream=None)
    args.update(over)
    return b.AttentionArgs(**args)


@pytest.mark.parametrize("over, status", [
    (dict(dtype=2), "CLI_UNSUPPORTED"), (dict(items=0), "CLI_SHAPE_MISMATCH"),
    (dict(query_rows=1 << 31), "CLI_SHAPE_MISMATCH"), (dict(key_rows=1 << 31), "CLI_SHAPE_MISMATCH"),
    (dict(head_dim=68), "CLI_SHAPE_MISMATCH"), (dict(head_dim=136), "CLI_UNSUPPORTED"),
    (dict(query_heads=7), "CLI_SHAPE_MISMATCH"), (dict(query_heads=0), "CLI_SHAPE_MISMATCH"),
    (dict(query_heads=258, key_heads=2), "CLI_UNSUPPORTED"), (dict(key_offsets=None), "CLI_INVALID_ARGUMENT"),
    (dict(query_offsets=None, items=1 << 30), "CLI_SHAPE_MISMATCH"),
    (dict(scale=float("nan")), "CLI_INVALID_ARGUMENT"), (dict(device_status=None), "CLI_INVALID_ARGUMENT"),
    (dict(key_offsets=A * 2 + 4), "CLI_INVALID_ARGUMENT"),
])
def test_attention_refusals(b, over, status):
    for verb in ("cross_attention", "cross_attention_backward"):
        assert getattr(b.lib, verb)(ctypes.byref(attention_args(b, **over))) == getattr(b, status), verb


def test_attention_refuses_bad_matrices(b):
    H = b.HeadsArgs
    fwd = lambda **o: b.lib.cross_attention(ctypes.byref(attention_args(b, **o)))  # noqa: E731
    bwd = lambda **o: b.lib.cross_attention_backward(ctypes.byref(attention_args(b, **o)))  # noqa: E731
    for call in (fwd, bwd):
        assert call(q=H(None, 512, 64)) == b.CLI_INVALID_ARGUMENT
        assert call(k=H(A * 4 + 8, 128, 64)) == b.CLI_INVALID_ARGUMENT
        assert call(v=H(A * 5, 132, 64)) == b.CLI_SHAPE_MISMATCH
        assert call(k=H(A * 4, 0, 64)) == b.CLI_SHAPE_MISMATCH              # broadcast rows
    assert fwd(output=H(A * 3, 512, 64)) == b.CLI_INVALID_ARGUMENT          # output over the queries
    assert fwd(output=H(A * 6, 256, 64)) == b.CLI_SHAPE_MISMATCH            # rows that overlap
    assert bwd(lse=None) == b.CLI_INVALID_ARGUMENT
    assert bwd(d_k=H(A * 11, 128, 64)) == b.CLI_INVALID_ARGUMENT            # dK over dV
    assert bwd(d_q=H(A * 6, 512, 64)) == b.CLI_INVALID_ARGUMENT             # dQ over the output it reads
    assert b.lib.cross_attention(None) == b.CLI_INVALID_ARGUMENT
    assert b.lib.cross_attention_workspace_bytes(None) == 0


def test_binding_refuses_host_memory(b):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(b.InvalidArgumentError):
        b.rotary_heads(x, torch.zeros(8, 32, 2))
    with pytest.raises(b.InvalidArgumentError):
        b.cross_attention(x, None, x, x, torch.zeros(2, dtype=torch.int64))
