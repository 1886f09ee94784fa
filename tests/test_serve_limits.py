"""Calls of more work than a launch may have threads for, and bounds that the
binding fills in."""
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu
from tests.serve_util import Batch, random_cache
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


@pytest.mark.gpu
def test_the_default_max_len_of_a_long_table():
    """A table that reaches past 2^31 positions: lengths are int32, so that is
    where the default bound ends."""
    need_gpu()
    b = Batch([1, 2], [300, 70], 128, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    q = torch.randn((3, 4, 64), device="cuda")
    table, cu, ln = b.device()
    far = torch.full((2, (1 << 31) // 128 + 5), -1, dtype=torch.int32, device="cuda")
    far[:, :table.shape[1]] = table
    want = q4.attention(q, *caches, table, cu, ln)
    got = q4.attention(q, *caches, far, cu, ln)
    assert torch.allclose(got, want, rtol=1e-5, atol=1e-6)
