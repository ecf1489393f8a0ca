"""What the token-state verbs refuse on the host, past tests/test_states_reference.py: no CUDA call is made."""

import ctypes

import pytest

from test_states_reference import A, attention_args, heads, rotary_args
from test_states_reference import b as _b

b = _b   # the fixture


@pytest.mark.parametrize("over", [
    # one CTA for four units of (item, key head): 2^34 of them
    dict(items=1 << 30, query_heads=64, key_heads=64, max_query_rows=1, max_key_rows=32),
    # items cut along their states: 2^35 rows to join, eight a CTA; items * heads is 2^32
    dict(items=1 << 30, query_heads=4, key_heads=4, max_query_rows=8, max_key_rows=1000, key_rows=(1 << 31) - 5000),
])
def test_attention_refuses_more_blocks_than_a_grid_has(b, over):
    args = attention_args(b, **over)
    assert b.lib.cross_attention(ctypes.byref(args)) == b.CLI_SHAPE_MISMATCH
    assert b.lib.cross_attention_workspace_bytes(ctypes.byref(args)) == 0


def test_attention_sizes_below_that_are_taken(b):
    args = attention_args(b, items=1 << 26, query_heads=64, key_heads=64, max_query_rows=1, max_key_rows=32)
    assert b.lib.cross_attention(ctypes.byref(args)) != b.CLI_SHAPE_MISMATCH


def test_matrices_past_the_address_space_are_refused(b):
    """Strides and spans that wrap in 64 bits: the overlap checks would look at another place."""
    H = b.HeadsArgs
    for rows, row, head in ((1 << 30, 1 << 38, 64), (100, (1 << 63) + 256, 64), (100, 256, (1 << 63) + 64)):
        part = dict(rows=rows, x=H(A * 4, row, head), y=heads(b, 5, rows, 4, 64))
        assert b.lib.rotary_heads(ctypes.byref(rotary_args(b, part=part))) == b.CLI_SHAPE_MISMATCH
        args = attention_args(b, key_rows=rows, max_key_rows=300, k=H(A * 4, row, head))
        assert b.lib.cross_attention(ctypes.byref(args)) == b.CLI_SHAPE_MISMATCH


@pytest.mark.parametrize("field", ["gain", "d_gain", "positions"])
def test_misaligned_vectors_are_refused(b, field):
    """32-bit values at an odd address: the kernel's access would fault."""
    for off in (1, 2, 3):
        part = {field: A * 20 + off}
        args = rotary_args(b, part=part)
        assert b.lib.norm_rotary_heads_backward(ctypes.byref(args)) == b.CLI_INVALID_ARGUMENT


def test_misaligned_attention_vectors_are_refused(b):
    for name, off in (("lse", 2), ("key_offsets", 4), ("query_offsets", 4), ("device_status", 2)):
        for verb in ("cross_attention", "cross_attention_backward"):
            args = attention_args(b, **{name: A * 20 + off})
            assert getattr(b.lib, verb)(ctypes.byref(args)) == b.CLI_INVALID_ARGUMENT, name
