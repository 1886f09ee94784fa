"""Scales that are none: a negative one stands for NaN in every operator, -0
for 0, whatever the page size and the number of rows (an imported cache may
hold them; the append never makes them).  And infinite ones, which the append
makes of infinite elements: no query that sees one has a finite output."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu
from tests.serve_util import Batch, random_cache
from tests.test_attention_gpu import FILL, check, run

pytestmark = pytest.mark.gpu


def shows_where_it_is_seen(which, value, page, new, fill, dtype="f32", window=0):
    """Sequence 0's second page has the scale `value`; earlier queries of the
    same call do not see it, nor do those whose window has left it."""
    lengths = [3 * page + 20, 300] + fill

    def edit(b, k, v, ks, vs):
        (ks if which == "k" else vs)[b.table[0, 1]] = value
    with np.errstate(invalid="ignore"):
        got, ref, tol = run([new, 1] + fill, lengths, 4, 2, 64, page, dtype, edit=edit, seed=14, window=window)
    pos = np.arange(lengths[0] - new, lengths[0])
    sees = (pos >= page) & ((pos - window + 1 < 2 * page) if window else True)
    sees = np.concatenate([sees, np.zeros(1 + len(fill), bool)])
    assert (~np.isfinite(got[sees])).all()
    assert np.isfinite(got[~sees]).all()
    assert (np.abs(got[~sees] - ref[~sees]) <= tol[~sees]).all()


MANY = [(1, 16, []), (1, 64, []), (3, 128, []), (250, 64, []), (70, 32, FILL), (170, 64, FILL), (400, 128, FILL)]


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [-0.02, -1e-30, -np.inf])
@pytest.mark.parametrize("new,page,fill", MANY)
def test_a_negative_scale_shows_where_it_is_seen(which, value, new, page, fill):
    shows_where_it_is_seen(which, value, page, new, fill)
    shows_where_it_is_seen(which, value, page, new, fill, dtype="bf16", window=page)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("new,page,fill", MANY)
def test_an_infinite_scale_shows_where_it_is_seen(which, new, page, fill):
    shows_where_it_is_seen(which, np.inf, page, new, fill)
    shows_where_it_is_seen(which, np.inf, page, new, fill, dtype="f16", window=page)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_an_appended_key_that_is_not_finite_shows(value, page):
    """The first token of a page, its key infinite in one channel, under
    queries of either sign there."""
    need_gpu()
    caches = q4.new_cache(3, 2, 64, page)
    n = page + 1
    k, q = torch.randn((n, 2, 64), device="cuda"), torch.randn((n, 4, 64), device="cuda")
    k[page, 0, 9] = value
    q[page, :2, 9] = torch.tensor([3.0, -3.0], device="cuda")
    args = [*caches, i32([[2, 0]]), i32([0, n]), i32([n])]
    q4.kv_append(k, k.nan_to_num(0.0, 0.0, 0.0), *args)
    out = q4.attention(q, *args)
    assert out[page, :2].isnan().all() and out[:page].isfinite().all() and out[page, 2:].isfinite().all()


@pytest.mark.parametrize("new,page,fill", MANY)
def test_minus_zero_is_a_scale_of_zero(new, page, fill):
    def edit(b, k, v, ks, vs):
        for p in b.used[::2]:
            ks[p] = vs[p] = -0.0
    check([new, 5] + fill, [3 * page + 20, 70] + fill, 4, 2, 64, page, "f32", edit=edit, seed=13)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("value", [-0.02, -float("inf"), float("nan")])
def test_an_append_to_a_page_without_a_scale(value):
    """What it held is not known: not finite until the page starts anew."""
    need_gpu()
    caches = q4.new_cache(2, 2, 64, 16)
    for c in caches[:2]:
        c.fill_(100)
    for c in caches[2:]:
        c.fill_(1.0)
        c[1, 1] = value
    k = torch.randn((2, 2, 64), device="cuda")
    q4.kv_append(k, k, *caches, i32([[1]]), i32([0, 2]), i32([7]))
    for got in q4.kv_dequant(*caches):
        assert got[0].isfinite().all() and got[1, 0].isfinite().all() and got[1, 1].isnan().all()
    q4.kv_append(k, k, *caches, i32([[1]]), i32([0, 2]), i32([2]))
    for got in q4.kv_dequant(*caches):
        assert got.isfinite().all()
        assert ((got[1, :, :2] - k.transpose(0, 1)).abs() <= 0.51 * k.abs().amax((0, 2))[:, None, None] / 127).all()


def test_an_append_to_a_page_of_scale_minus_zero():
    need_gpu()
    caches = q4.new_cache(1, 1, 64, 16)
    for c in caches[2:]:
        c.fill_(-0.0)
    k = torch.randn((1, 1, 64), device="cuda")
    q4.kv_append(k, -k, *caches, i32([[0]]), i32([0, 1]), i32([3]))
    for got, want in zip(q4.kv_dequant(*caches), (k, -k)):
        assert ((got[0, 0, 2] - want[0, 0]).abs() <= 0.51 * k.abs().max() / 127).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_values_of_a_page_without_a_scale(dtype):
    need_gpu()
    b = Batch([1], [40], 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    for c in caches[2:]:
        c.fill_(0.5)
        c[1, 0] = -0.5
    for got in q4.kv_dequant(*caches, dtype=dtype):
        assert got[1, 0].isnan().all() and got[1, 1].isfinite().all() and got[[0, 2]].isfinite().all()
