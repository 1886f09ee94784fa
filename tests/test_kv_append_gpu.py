"""The cache append against the fp64 oracle: a code is right if it is within
half a step of the exact quotient, plus what fp32 can move the quotient by.

Slack of a quotient (at most 127): the turned element is off by at most
4 2^-24 of the pair's magnitude (cosine and sine 2^-23 each way, two products
and a sum), at most sqrt(2) of the page's largest element; the scale and the
division add 3 2^-24: 127 (6 + 3) 2^-24 < 1e-4.
"""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import serve_oracle as orc
from tests.gpu_util import need_gpu
from tests.serve_util import TORCH, Batch, random_cache, rounded, strided

pytestmark = pytest.mark.gpu

SLACK = 1e-4
SCALE_TOL = 8 * 2.0 ** -24


def freqs(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


def check(new, lengths, heads, kv_heads, dim, page, dtype, *, rot=None, interleaved=False, seed=0,
          layout="packed", gain=1.0, in_place=False, bound=True):
    need_gpu()
    rot = dim if rot is None else rot
    b = Batch(new, lengths, page, seed)
    k, v, ks, vs = random_cache(b, kv_heads, dim, seed + 1)
    g = np.random.default_rng(seed + 2)
    kt, kx = rounded(g.normal(0, gain, (b.T, kv_heads, dim)), dtype)
    vt, vx = rounded(g.normal(0, gain, (b.T, kv_heads, dim)), dtype)
    qt, qx = rounded(g.normal(0, gain, (b.T, heads, dim)), dtype)
    f = freqs(rot)
    print(f"[append] new={b.new[:6]} len={b.lengths[:6]} heads={heads}/{kv_heads} dim={dim} "
          f"page={page} {dtype} rot={rot} {layout}", flush=True)
    caches = [torch.from_numpy(x).cuda() for x in (k, v, ks, vs)]
    table, cu, ln = b.device()
    qd = strided(qt, layout)
    got_q = q4.kv_append(strided(kt, layout), strided(vt, layout), *caches, table, cu, ln, q=qd,
                         q_out=qd if in_place else None,
                         inv_freq=torch.from_numpy(f).cuda() if rot else None,
                         interleaved=interleaved, max_new=max(b.new + [1]) if bound else None)
    torch.cuda.synchronize()
    if in_place:
        assert got_q.data_ptr() == qd.data_ptr()
    gk, gv, gks, gvs = (x.cpu().numpy() for x in caches)
    rk, rv, rks, rvs, touched = orc.append(kx, vx, k, v, ks, vs, b.table, b.cu, b.len, f, interleaved)
    gv_t, v_t = np.swapaxes(gv, 2, 3), np.swapaxes(v, 2, 3)
    pages = {p for p, _ in touched}
    for p in range(b.pages):
        if p not in pages:  # untouched pages are bit for bit what they were
            assert np.array_equal(gk[p], k[p]) and np.array_equal(gv[p], v[p])
            assert np.array_equal(gks[p], ks[p], equal_nan=True)
            assert np.array_equal(gvs[p], vs[p], equal_nan=True)
    for p, used in touched:
        assert np.allclose(gks[p], rks[p], rtol=SCALE_TOL, atol=0)
        assert np.allclose(gvs[p], rvs[p], rtol=SCALE_TOL, atol=0)
        for got, ref in ((gk, rk), (gv_t, rv)):
            off = np.abs(got[p, :, :used].astype(np.float64) - ref[p, :, :used])
            assert off.max() <= 0.5 + SLACK, (p, off.max())
    # queries: products of fp32 and one rounding
    want = np.stack([np.stack([orc.rotate(qx[t, h], pos0 + t - t0, f, interleaved) for h in range(heads)])
                     for t0, n, pos0 in orc.spans(b.cu, b.len) for t in range(t0, t0 + n)]) \
        if b.T else np.zeros((0, heads, dim))
    # half a step is relative down to the smallest normal number, and constant below it
    info = torch.finfo(TORCH[dtype])
    half = info.eps / 2 * np.maximum(np.abs(want), info.smallest_normal)
    err = np.abs(got_q.double().cpu().numpy() - want)
    assert (err <= half + 6 * 2.0 ** -24 * np.abs(qx).max()).all()
    return caches, b


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens(page, dtype):
    lengths = [1, 2, 16, 17, 18, 33, 64, 65, 100, 127, 128, 129]
    check([1] * len(lengths), lengths, 4, 2, 64, page, dtype, seed=page)
    check([1] * len(lengths), lengths, 4, 2, 64, page, dtype, seed=page, gain=0.01)  # no scale grows
    check([1] * len(lengths), lengths, 4, 2, 64, page, dtype, seed=page, gain=9.0)   # every scale grows


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_chunks_that_start_and_end_inside_pages(page):
    new = [1, 5, 15, 16, 17, 33, 64, 100, 130, 200]
    before = [0, 3, 16, 7, 0, 31, 64, 60, 1, 128]
    check(new, [a + n for a, n in zip(before, new)], 4, 2, 64, page, "f32", seed=3)


@pytest.mark.parametrize("dim", [16, 48, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes_and_partial_turns(dim, interleaved):
    for rot in sorted({0, 2, dim // 2, dim}):
        check([3, 1, 20], [3, 40, 25], 6, 3, dim, 16, "f32", rot=rot, interleaved=interleaved, seed=dim)
    check([130], [135], 2, 1, dim, 128, "bf16", interleaved=interleaved, seed=1)


@pytest.mark.parametrize("layout", ["packed", "fused", "heads_first", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_in_place(layout, dtype):
    check([1, 6, 20], [100, 66, 20], 8, 4, 80, 32, dtype, layout=layout, in_place=True)
    check([1, 6, 20], [100, 66, 20], 8, 4, 80, 32, dtype, layout=layout, bound=False)


def test_far_positions_keep_their_angle():
    need_gpu()
    for pos in (1 << 20, (1 << 24) + 3, (1 << 30) + 12345):
        f = freqs(64, 500000.0)
        g = np.random.default_rng(pos)
        kt, kx = rounded(g.normal(0, 1, (1, 1, 64)), "f32")
        caches = q4.new_cache(1, 1, 64, 16)
        table = torch.full((1, pos // 16 + 1), -1, dtype=torch.int32, device="cuda")
        table[0, pos // 16] = 0
        # queries in the place of keys: they are not coded
        got = q4.kv_append(kt.cuda(), kt.cuda(), *caches, table,
                           torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                           torch.tensor([pos + 1], dtype=torch.int32, device="cuda"), q=kt.cuda(),
                           inv_freq=torch.from_numpy(f).cuda())
        want = orc.rotate(kx[0, 0], pos, f)
        # fp64 angle: pos 2^-53 revolutions at most, below 2^-22; then fp32
        assert np.abs(got[0, 0].cpu().numpy() - want).max() <= (6 * 2.0 ** -24 + 2.0 ** -20) * np.abs(kx).max()


def test_a_page_filled_token_by_token():
    """Each step against the state the last one left: growth after growth."""
    need_gpu()
    dim, page, g = 64, 16, np.random.default_rng(0)
    caches = q4.new_cache(2, 1, dim, page)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    f = freqs(dim)
    for pos in range(20):
        kt, kx = rounded(g.normal(0, 1 + pos % 7, (1, 1, dim)), "f32")
        vt, vx = rounded(g.normal(0, 1 + pos % 5, (1, 1, dim)), "f32")
        before = [x.cpu().numpy().copy() for x in caches]
        ln = torch.tensor([pos + 1], dtype=torch.int32, device="cuda")
        q4.kv_append(kt.cuda(), vt.cuda(), *caches, table, cu, ln, inv_freq=torch.from_numpy(f).cuda())
        after = [x.cpu().numpy() for x in caches]
        rk, rv, rks, rvs, touched = orc.append(kx, vx, *before, table.cpu().numpy(), cu.cpu().numpy(),
                                               ln.cpu().numpy(), f)
        (p, used), = touched
        assert np.abs(after[0][p, 0, :used] - rk[p, 0, :used]).max() <= 0.5 + SLACK
        assert np.abs(after[1][p, 0, :, :used].T - rv[p, 0, :used]).max() <= 0.5 + SLACK
        assert np.allclose(after[2], rks, rtol=SCALE_TOL) and np.allclose(after[3], rvs, rtol=SCALE_TOL)


def test_a_page_that_starts_anew_forgets_what_it_held():
    need_gpu()
    caches = q4.new_cache(1, 1, 64, 16)
    caches[0].fill_(99)
    caches[1].fill_(-99)
    caches[2].fill_(float("nan"))
    caches[3].fill_(float("inf"))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.randn((3, 1, 64), device="cuda")
    q4.kv_append(k, 2 * k, *caches, i32([[0]]), i32([0, 3]), i32([3]))
    assert torch.allclose(caches[2], k.abs().max() / 127) and torch.allclose(caches[3], 2 * k.abs().max() / 127)
    assert (caches[0][0, 0, 3:] == 0).all() and (caches[1][0, 0, :, 3:] == 0).all()


def test_zeros_and_values_that_are_not_finite():
    need_gpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (float("nan"), float("inf"), -float("inf")):
        caches = q4.new_cache(2, 2, 64, 16)
        k = torch.zeros((2, 2, 64), device="cuda")
        v = k.clone()
        v[1, 1, 5] = bad
        q4.kv_append(k, v, *caches, i32([[1]]), i32([0, 2]), i32([2]))
        assert (caches[2] == 0).all() and (caches[0] == 0).all()
        assert caches[3][1, 0] == 0 and not caches[3][1, 1].isfinite()
        dk, dv = q4.kv_dequant(*caches)
        assert (dk == 0).all() and (dv[1, 0] == 0).all() and not dv[1, 1, :2].isfinite().any()
    # the smallest normal and subnormal magnitudes
    for x in (2.0 ** -126, 2.0 ** -140, 3e38):
        caches = q4.new_cache(1, 1, 64, 16)
        k = torch.full((1, 1, 64), x, device="cuda")
        q4.kv_append(k, -k, *caches, i32([[0]]), i32([0, 1]), i32([1]))
        dk, dv = q4.kv_dequant(*caches)
        assert ((dk[0, 0, 0] - x).abs() <= x / 200 + 2.0 ** -149 * 64).all(), x
        assert torch.equal(dk, -dv)


def test_tokens_without_a_place_are_not_stored():
    """Bad pages, a table that is too short, more new tokens than the length
    (checked on the CPU by test_serve_index.py first)."""
    need_gpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    caches = q4.new_cache(3, 1, 64, 16)
    k = torch.randn((8, 1, 64), device="cuda")
    q = torch.randn((8, 2, 64), device="cuda")
    # sequence 0: page 3 does not exist; 1: page -1; 2: position 32 is past the table; 3: three of four have a place
    out = q4.kv_append(k, k, *caches, i32([[3, 0], [-1, 0], [0, 0], [2, 2]]), i32([0, 1, 3, 4, 8]),
                       i32([5, 2, 33, 3]), q=q)
    torch.cuda.synchronize()
    assert torch.equal(out, q)
    assert (caches[0][:2] == 0).all() and (caches[2][:2] == 0).all()
    assert torch.allclose(caches[2][2, 0], k[5:8].abs().max() / 127)
    assert (caches[0][2, 0, :3].abs().amax(1) > 0).all() and (caches[0][2, 0, 3:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page,dim", [(16, 16), (32, 80), (64, 128), (128, 256)])
def test_dequant(page, dim, dtype):
    need_gpu()
    b = Batch([1, 1], [page + 3, 5], page, 0)
    k, v, ks, vs = random_cache(b, 3, dim, 1)
    dk, dv = q4.kv_dequant(*[torch.from_numpy(x).cuda() for x in (k, v, ks, vs)], dtype=TORCH[dtype])
    for got, codes, s in ((dk, k, ks), (dv, np.swapaxes(v, 2, 3), vs)):
        want = (torch.from_numpy(codes.astype(np.float32)) * torch.from_numpy(s)[:, :, None, None]).to(TORCH[dtype])
        assert torch.equal(torch.nan_to_num(got.cpu(), 9.0), torch.nan_to_num(want, 9.0))
