"""Queries and keys side by side in each head: layouts whose rows meet are refused by the
C entry, before any CUDA work.  (Those that do not are turned in tests on the GPU.)"""
import pytest

kda = pytest.importorskip("kda_gated_delta_chunked_gb300", reason="libkda.so not built (run __graft_entry__.build())")
from test_cache_rotary_host import rot  # noqa: E402
from test_operators_host import BAD, P  # noqa: E402


def side_by_side(at, heads=4, kheads=4, head=136, khead=136, token=544, ktoken=544, width=64, kwidth=64, **kw):
    """Queries [10, heads, width] in place at P[0], keys `at` channels behind them."""
    a = dict(heads=heads, width=width, offset=width - 64, token_stride=token, head_stride=head, out_token_stride=token, out_head_stride=head)
    b = dict(heads=kheads, width=kwidth, offset=kwidth - 64, token_stride=ktoken, head_stride=khead, out_token_stride=ktoken, out_head_stride=khead)
    return rot(out=P[0], key=P[0] + 2 * at, key_out=P[0] + 2 * at, part=a, key_part=b, **kw)


def test_rows_that_meet_within_heads():
    assert side_by_side(63) == BAD and side_by_side(73) == BAD and side_by_side(136 * 4 + 73) == BAD
    assert side_by_side(64, width=66) == BAD and side_by_side(72, kwidth=65) == BAD
    # heads outermost
    out = dict(head=1360, khead=1360, token=136, ktoken=136)
    assert side_by_side(63, **out) == BAD and side_by_side(73, **out) == BAD and side_by_side(1360 + 73, **out) == BAD
    # other heads or tokens a stride
    assert side_by_side(60, heads=2, head=272) == BAD and side_by_side(68, kheads=3, khead=150, ktoken=544) == BAD
    assert side_by_side(73, tokens=1) == BAD and side_by_side(63, tokens=1, kheads=1) == BAD
