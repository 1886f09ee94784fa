"""Calls of more work than a launch may have threads for, and bounds that the
binding fills in, on the host."""
import pytest

from tests.test_serve_abi import APPEND, ATTN, INVALID, call


@pytest.mark.parametrize("kw", [
    dict(B=1 << 22, T=1 << 22, heads=8, kv=8, max_new=1),           # 2^25 workgroups of a row block
    dict(B=1 << 14, T=1 << 15, heads=8, kv=4, max_new=1 << 14),     # 128 rows each
])
def test_attention_of_more_workgroups_than_a_launch_has_is_refused(kw):
    assert call("q4_attention", ATTN, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(B=1 << 21, T=1 << 21, max_new=1), dict(T=1 << 27, max_new=1)])
def test_an_append_of_more_workgroups_than_a_launch_has_is_refused(kw):
    # (more pages of a sequence than that come in several launches)
    assert call("q4_kv_append", APPEND, **kw) == INVALID
