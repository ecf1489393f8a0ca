"""What the token-state verbs refuse on the host, past tests/test_states_reference.py: no CUDA call is made."""

import ctypes

import pytest

from test_states_reference import A, attention_args, heads
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
