"""Attention over the paged 8-bit cache against the fp64 oracle.

Bound of an output element, from the kernel's arithmetic (h: half a step of
the digits; V the largest |value| a query sees, s its largest |score|):
  * a query's digits: step 2^-22 of its largest element (three digits; 2^-14
    for two), so a score is off by at most  e_q = scale max|q| sum|k| h_q,
    h_q = 2^-23 or 2^-15; fp32 steps of the score, its maximum's subtraction
    and the exponential: e_s = 10 2^-24 (max|s| + 1);
    probabilities and their sum: 2 (e_q + e_s) V;
  * probabilities' digits: half a step h_p = 2^-24 or 2^-16 of a tile's
    largest, 64 tokens, and a tile's largest is at most its sum: 64 h_p V.
    Where a tile mixes pages, the digits are relative to its largest
    p * scale, so V times the largest ratio of scales (spread);
  * sums over tiles and waves in fp32: (tiles + 32) 2^-24 V;
  * the output's rounding, finfo.eps / 2 |out|.
"""
import math

import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import serve_oracle as orc
from tests.gpu_util import need_gpu
from tests.serve_util import TORCH, Batch, random_cache, rounded, strided

pytestmark = pytest.mark.gpu


def tolerance(out, bound, dtype, scale, max_len, page, spread):
    h_q, h_p = (2.0 ** -23, 2.0 ** -24) if dtype == "f32" else (2.0 ** -15, 2.0 ** -16)
    s, V, k1, q = (bound[..., i:i + 1] for i in range(4))
    mix = math.exp(2 * spread) if page < 64 else 1.0
    tiles = max_len / 64 + 2
    return (V * (2 * (scale * q * k1 * h_q + 10 * 2.0 ** -24 * (s + 1)) + 64 * h_p * mix
                 + (tiles + 32) * 2.0 ** -24) + torch.finfo(TORCH[dtype]).eps / 2 * np.abs(out))


def run(new, lengths, heads, kv_heads, dim, page, dtype, *, window=0, seed=0, layout="packed",
        scale=None, spread=1.0, q_gain=1.5, bounds=True, edit=None, max_len=None):
    need_gpu()
    b = Batch(new, lengths, page, seed)
    k, v, ks, vs = random_cache(b, kv_heads, dim, seed + 1, spread)
    g = np.random.default_rng(seed + 2)
    qt, q = rounded(g.normal(0, q_gain, (b.T, heads, dim)), dtype)
    if edit:
        edit(b, k, v, ks, vs)
    print(f"[attention] new={b.new[:6]} len={b.lengths[:6]} heads={heads}/{kv_heads} dim={dim} "
          f"page={page} {dtype} window={window} {layout}", flush=True)
    table, cu, ln = b.device()
    out = strided(torch.full((b.T, heads, dim), float("nan"), dtype=TORCH[dtype]), layout)
    caches = [torch.from_numpy(x).cuda() for x in (k, v, ks, vs)]
    kw = dict(max_new=max(b.new + [1]), max_len=max_len or max(b.lengths + [0])) if bounds else {}
    got = q4.attention(strided(qt, layout), *caches, table, cu, ln, softmax_scale=scale,
                       window=window, out=out, **kw)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    got = got.double().cpu().numpy()
    ref, bound = orc.attention(q, k, v, ks, vs, b.table, b.cu, b.len, scale=scale, window=window)
    tol = tolerance(ref, bound, dtype, dim ** -0.5 if scale is None else abs(scale),
                    max(b.lengths + [0]), page, spread)
    return got, ref, tol


def check(*args, **kw):
    got, ref, tol = run(*args, **kw)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()) if got.size else 0.0
    print(f"            worst error / bound {worst:.3f}", flush=True)
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_lengths_around_pages_and_tiles(page, dtype):
    lengths = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 257, 320]
    check([1] * len(lengths), lengths, 8, 2, 64, page, dtype, seed=page)


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_sizes(dim, dtype):
    check([1, 3, 1], [70, 150, 5], 6, 2, dim, 32, dtype, seed=dim)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (7, 1), (32, 8), (15, 5), (16, 1), (17, 1),
                                            (40, 2), (64, 1)])
def test_head_groups(heads, kv_heads):
    check([1, 2, 5], [90, 40, 130], heads, kv_heads, 64, 16, "f32", seed=heads)


@pytest.mark.parametrize("layout", ["packed", "fused", "heads_first", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_strides(layout, dtype):
    check([1, 6, 2], [100, 66, 3], 8, 4, 80, 32, dtype, layout=layout, seed=5)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [1, 7, 64, 65, 100, 1000])
def test_windows(window, page):
    check([1, 4, 9, 20], [300, 129, 9, 77], 4, 2, 64, page, "f32", window=window, seed=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 64])
def test_many_new_tokens(page, dtype):
    check([130, 1, 64, 37], [130, 500, 300, 38], 8, 2, 64, page, dtype, seed=11)
    check([97, 200], [600, 201], 4, 1, 128, page, dtype, seed=12, window=150)


# sequences that make the rows many enough for the kernel that shares keys between them
FILL = [1] * 75


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 128, 144, 192, 256])
@pytest.mark.parametrize("page,dtype", [(16, "f32"), (64, "f16"), (128, "f32"), (32, "bf16")])
def test_chunks_of_all_head_sizes(dim, page, dtype):
    check([33, 70, 1] + FILL, [33, 400, 90] + FILL, 4, 2, dim, page, dtype, seed=dim, layout="fused")


@pytest.mark.parametrize("window", [1, 40, 64, 129, 1000])
@pytest.mark.parametrize("page", [16, 64])
def test_chunks_under_windows(window, page):
    check([150, 64, 3, 0] + FILL, [700, 64, 200, 10] + FILL, 3, 1, 64, page, "f32", window=window, seed=window)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 1), (32, 8), (130, 1)])
def test_chunks_of_head_groups(heads, kv_heads):
    check([65, 129, 2] + FILL, [80, 300, 2] + FILL, heads, kv_heads, 32, 64, "f16", seed=heads)


def test_chunks_over_long_contexts_are_split():
    check([40, 7] + FILL, [5000, 2100] + FILL, 8, 2, 128, 64, "bf16", seed=1)
    check([40, 7] + FILL, [5000, 2100] + FILL, 8, 2, 64, 16, "f32", seed=2, window=3000)
    check([40, 5] + FILL, [60, 2100] + FILL, 8, 2, 64, 16, "f32", seed=3, max_len=100000)


@pytest.mark.parametrize("new,lengths,heads,kv_heads,dim,page,dtype,window", [
    ([70, 5], [17000, 900], 8, 2, 64, 64, "bf16", 0),
    ([70, 5], [17000, 900], 8, 2, 128, 16, "f32", 0),
    ([40, 33, 0], [14000, 33, 50], 16, 16, 32, 64, "f16", 0),
    ([9, 9, 1] + [9] * 9, [20000, 19, 1] + [700] * 9, 8, 2, 80, 128, "f32", 0),
    ([70, 66, 3], [30000, 29000, 3], 8, 2, 64, 32, "bf16", 20000),
])
def test_chunks_of_few_sequences_over_long_contexts(new, lengths, heads, kv_heads, dim, page, dtype, window):
    """Few rows, so that rows times keys make the choice of the shared keys."""
    check(new, lengths, heads, kv_heads, dim, page, dtype, window=window, seed=dim)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_blocks_of_chunks(dtype):
    """More than 512 workgroups of 128 rows by the bounds."""
    check([130] + [3] * 120, [600] + [9] * 120, 16, 4, 64, 64, dtype, seed=5)


def test_chunks_with_scores_and_scales_far_apart():
    for kw in (dict(q_gain=40.0, seed=8), dict(scale=0.0, seed=9), dict(scale=-0.3, seed=10), dict(spread=3.0, seed=12),
               dict(q_gain=3e5, seed=13)):
        for page in (16, 64, 128):
            check([100, 30] + FILL, [400, 170] + FILL, 4, 2, 64, page, "f32", **kw)
    check([100, 30] + FILL, [400, 170] + FILL, 4, 2, 64, 64, "bf16", q_gain=40.0, seed=8)


def test_empty_sequences_and_queries_before_the_start():
    # length 0 (queries see nothing), no new tokens, more new tokens than the length
    got, ref, tol = run([1, 0, 3, 2, 0], [0, 50, 2, 40, 0], 4, 2, 64, 16, "f32")
    assert (np.abs(got - ref) <= tol).all()
    assert (got[0] == 0).all() and (got[1] == 0).all()  # the second: pos = -1


def test_nothing_to_do():
    need_gpu()
    b = Batch([0, 0], [5, 9], 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 0)]
    q = torch.empty((0, 4, 64), device="cuda")
    assert q4.attention(q, *caches, *b.device()).shape == (0, 4, 64)


@pytest.mark.parametrize("lengths,kv_heads", [([5000], 1), ([9000, 30, 2500], 2), ([20011], 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_axis_split_over_workgroups(lengths, kv_heads, dtype):
    check([1] * len(lengths), lengths, 4 * kv_heads, kv_heads, 64, 64, dtype, seed=3)


# a generous max_len: the kernel for long contexts on short ones too
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_short_contexts_among_long_ones(page, dtype):
    lengths = [0, 1, 2, 63, 64, 65, 0, 127, 128, 129, 300, 700, 2100, 17]
    check([1] * len(lengths), lengths, 8, 2, 64, page, dtype, seed=page, max_len=4096)
    check([0, 1, 1, 0], [70, 0, 400, 90], 4, 4, 128, page, dtype, seed=page, max_len=1 << 20)


@pytest.mark.parametrize("heads,kv_heads,new", [(16, 1, [1, 2, 2, 1]), (6, 2, [5, 1, 10, 0]), (32, 1, [1, 1, 1, 1]),
                                                (7, 1, [3, 4, 2, 1])])
@pytest.mark.parametrize("window", [0, 100, 2500])
def test_several_rows_over_long_contexts(heads, kv_heads, new, window):
    check(new, [2300, 4, 130, 900], heads, kv_heads, 96, 32, "f32", window=window, seed=heads, max_len=9000)


@pytest.mark.parametrize("dim", [16, 48, 80, 128, 176, 256])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_head_sizes_over_long_contexts(dim, dtype):
    check([1, 1], [2500, 200], 4, 2, dim, 64, dtype, seed=dim)


def test_many_sequences():
    g = np.random.default_rng(0)
    lengths = [int(x) for x in g.integers(0, 150, 600)]
    lengths[77] = 2200
    check([1] * 600, lengths, 2, 1, 32, 16, "f32", seed=1)


def test_default_bounds_match_exact_ones():
    a = run([1, 3], [200, 90], 8, 2, 64, 16, "f32", bounds=True)[0]
    b, ref, tol = run([1, 3], [200, 90], 8, 2, 64, 16, "f32", bounds=False)
    assert (np.abs(b - ref) <= tol).all() and (np.abs(a - ref) <= tol).all()


def test_scores_far_apart_and_all_equal():
    check([1, 2], [400, 70], 4, 2, 64, 64, "f32", q_gain=40.0, seed=8)
    check([1, 2], [400, 70], 4, 2, 64, 16, "f32", scale=0.0, seed=9)
    check([1, 2], [400, 70], 4, 2, 64, 16, "f32", scale=-0.3, seed=10)


@pytest.mark.parametrize("page", [16, 64])
def test_page_scales_far_apart(page):
    check([1, 3, 18], [500, 130, 260], 4, 2, 64, page, "f32", spread=3.0, seed=21)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_zero_scales(page):
    def edit(b, k, v, ks, vs):
        for p in b.used[::2]:
            ks[p] = 0
            vs[p] = 0
            k[p] = 0
            v[p] = 0
    check([1, 5], [400, 70], 4, 2, 64, page, "f32", edit=edit, seed=13)


# (an infinite key scale is left out: a score of -inf is no weight at all)
@pytest.mark.parametrize("which,value", [("k", np.nan), ("v", np.nan), ("v", np.inf)])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("new,fill", [(40, []), (60, FILL)])
def test_a_page_that_is_not_finite_shows_only_where_it_is_seen(which, value, page, new, fill):
    """Sequence 0's second page; earlier queries of the same call do not see it."""
    lengths = [page + 20, 300] + fill

    def edit(b, k, v, ks, vs):
        (ks if which == "k" else vs)[b.table[0, 1]] = value
    with np.errstate(invalid="ignore"):
        got, ref, tol = run([new, 1] + fill, lengths, 4, 2, 64, page, "f32", edit=edit, seed=14)
    sees = np.array([lengths[0] - new + i >= page for i in range(new)] + [False] * (1 + len(fill)))
    assert (~np.isfinite(got[sees])).all(axis=2).all()
    assert np.isfinite(got[~sees]).all()
    assert (np.abs(got[~sees] - ref[~sees]) <= tol[~sees]).all()


def test_bad_pages_in_chunks():
    need_gpu()
    b = Batch([90] + FILL, [200] + FILL, 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    q = torch.randn((b.T, 4, 64), device="cuda")
    table, cu, ln = b.device()
    clean = q4.attention(q, *caches, table, cu, ln, max_new=90)
    table[0, 9] = b.pages  # positions 144 .. 159; the new tokens are at 110 .. 199
    got = q4.attention(q, *caches, table, cu, ln, max_new=90)
    assert clean.isfinite().all() and got[34:90].isnan().all()
    assert torch.allclose(got[:34], clean[:34], rtol=1e-5, atol=1e-6) and torch.equal(got[90:], clean[90:])


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite_stay_in_their_row(value):
    need_gpu()
    b = Batch([1, 4], [200, 70], 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    q = torch.randn((5, 4, 64), device="cuda")
    clean = q4.attention(q, *caches, *b.device())
    q[2, 1, 7] = value
    got = q4.attention(q, *caches, *b.device())
    assert got[2, 1].isnan().all()
    keep = torch.ones((5, 4), dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])


def test_bad_pages_give_nan_where_they_are_seen():
    """Page numbers outside the cache and a table that is too short: the
    kernel's own checks (covered on the CPU by test_serve_index.py)."""
    need_gpu()
    b = Batch([1, 1, 2, 1], [200, 200, 200, 40], 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    q = torch.randn((5, 4, 64), device="cuda")
    table, cu, ln = b.device()
    clean = q4.attention(q, *caches, table, cu, ln)
    assert clean.isfinite().all()
    bad = table.clone()
    bad[0, 3] = b.pages          # one past the cache
    bad[1, 12] = -1              # the last page
    got = q4.attention(q, *caches, bad, cu, ln)
    assert got[:2].isnan().all() and torch.equal(got[2:], clean[2:])
    # only 12 columns: positions 192 .. 199 have no entry; windows that skip bad pages are fine
    got = q4.attention(q, *caches, table[:, :12].contiguous(), cu, ln, max_len=200)
    assert got[:4].isnan().all() and torch.equal(got[4:], clean[4:])
    windowed = q4.attention(q, *caches, bad, cu, ln, window=100)
    assert windowed[0].isfinite().all() and windowed[1].isnan().all()


def test_results_repeat_and_replay():
    """Bit-identical again, and from a graph replayed with other lengths."""
    need_gpu()
    b = Batch([1, 1, 1], [3000, 70, 900], 64, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 128, 1)]
    q = torch.randn((3, 8, 128), device="cuda")
    table, cu, ln = b.device()
    out = torch.empty_like(q)
    ws = torch.empty(q4.attention_workspace_bytes(3, 3, 8, 2, 128, page=64, max_new=1, max_len=3000),
                     dtype=torch.uint8, device="cuda")
    call = lambda: q4.attention(q, *caches, table, cu, ln, max_new=1, max_len=3000, out=out,  # noqa: E731
                                workspace=ws)
    first = call().clone()
    assert torch.equal(call(), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ([3000, 70, 900], [64, 1, 2999], [5, 3, 1], [3000, 70, 900]):
        ln.copy_(torch.tensor(lengths, dtype=torch.int32))
        table2, _, _ = b.device()
        valid = min(lengths)  # the table names pages for the first lengths only
        eager = q4.attention(q, *caches, table2, cu, ln, max_new=1, max_len=3000).clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert valid > 0 and torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(eager, 7.0))


def test_on_a_stream_of_its_own():
    need_gpu()
    b = Batch([1, 2], [700, 70], 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    q = torch.randn((3, 4, 64), device="cuda")
    args = b.device()
    want = q4.attention(q, *caches, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = q4.attention(q, *caches, *args)
    s.synchronize()
    assert torch.equal(got, want)
