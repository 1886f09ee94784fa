"""Attention with bounds below what the sequences bring: queries past max_new
are not computed and their outputs stay as they are, in every kernel and with
one split of the keys or several; the others are right."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import serve_oracle as orc
from tests.gpu_util import need_gpu
from tests.serve_util import Batch, random_cache, rounded
from tests.test_attention_gpu import FILL, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("new,lengths,heads,kv_heads,max_new,max_len", [
    ([5, 1, 3], [60, 9, 3], 2, 2, 1, 60),             # a row of 16, one split
    ([5, 1, 3], [60, 9, 3], 8, 2, 2, 60),
    ([5, 2], [3000, 700], 2, 2, 1, 3000),             # few splits
    ([7, 2], [9000, 90], 4, 1, 3, 9000),              # many
    ([50, 1, 90] + FILL, [300, 80, 90] + FILL, 4, 2, 40, 300),    # rows that share keys
    ([60, 70, 3], [30000, 900, 3], 8, 2, 50, 30000),              # and splits of them
])
def test_queries_past_max_new_are_left_alone(new, lengths, heads, kv_heads, max_new, max_len, dtype):
    need_gpu()
    b = Batch(new, lengths, 64, 3)
    k, v, ks, vs = random_cache(b, kv_heads, 64, 4)
    qt, q = rounded(np.random.default_rng(5).normal(0, 1.5, (b.T, heads, 64)), dtype)
    print(f"[attention] new={new[:3]} max_new={max_new} max_len={max_len} {dtype}", flush=True)
    out = torch.full((b.T, heads, 64), 7.0, dtype=qt.dtype, device="cuda")
    q4.attention(qt.cuda(), *[torch.from_numpy(x).cuda() for x in (k, v, ks, vs)], *b.device(), max_new=max_new,
                 max_len=max_len, out=out)
    got = out.double().cpu().numpy()
    ref, bound = orc.attention(q, k, v, ks, vs, b.table, b.cu, b.len)
    tol = tolerance(ref, bound, dtype, 64 ** -0.5, max_len, 64, 1.0)
    i = np.concatenate([np.arange(n) for n in new])
    assert (got[i >= max_new] == 7.0).all()
    assert (np.abs(got - ref) <= tol)[i < max_new].all()
