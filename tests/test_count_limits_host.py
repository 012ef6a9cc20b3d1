"""Sizes whose tiles of keys cannot be counted in 32 bits are refused through the C ABI before
anything is looked up or launched (the few-row kernel counts them so)."""
import pytest

from test_prefix_host import args_of as prefix_args, calls as prefix_calls, lib as prefix_lib  # noqa: F401
from test_q4_host import args_of as q4_args, lib as q4_lib  # noqa: F401

# 65536 (request, KV head) pairs, tables for 2^29 positions each; and 128 of 2^28 with 4096 rows
WIDE = [dict(batch=4096, num_q_heads=16, num_kv_heads=16, max_pages=1 << 25, num_pages=64),
        dict(batch=16, num_q_heads=8, num_kv_heads=8, max_pages=1 << 24, num_pages=64, q_len=4096),
        dict(batch=2**31 - 1, num_q_heads=1 << 20, num_kv_heads=1 << 20, num_pages=64, q_len=1 << 29)]


@pytest.mark.parametrize("shape", WIDE)
def test_prefix(prefix_lib, shape):  # noqa: F811
    a, s = prefix_args(dict(shape=shape))
    assert list(prefix_calls(prefix_lib, a, s)) == [2] * 3


@pytest.mark.parametrize("shape", WIDE)
def test_4_bit_decode(q4_lib, shape):  # noqa: F811
    a, s = q4_args(dict(shape=shape))
    assert q4_lib.pa_decode_q4(*[a[k] for k in ("q", "k", "v", "bt", "cl", "ps", "scale", "causal", "out")], s,
                               a["mcl"], a["ws"], a["wsb"], None) == 2
