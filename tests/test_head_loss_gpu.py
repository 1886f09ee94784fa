"""The packed head's cross entropy and its gradient on the GPU against the fp64
oracle.  Bounds (products as in experts_util.py): with ez the largest error of a
row's logits, lse is off by ez and 2^-20 (1 + |lse|) for exponentials and sums
(relative errors of 2^-21 each in a logarithm), a probability by p (ez + else +
2^-20), its product with the scale by the type's kept bits."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import GIVEN, HALF_STEP, KEPT, TORCH, assert_within, packed, product_bound, rounded, strided, sums

pytestmark = pytest.mark.gpu


def check(M, V, K, group, dtype, order="high_first", layout="packed", seed=0, gain=2.5, targets=None):
    rng = np.random.default_rng(seed)
    codes, scales = packed(rng, (), V, K, group)
    scales = (gain * scales).astype(np.float32)
    w = oracle.matrix(codes, scales, group, order == "high_first")
    x, xv = rounded(rng.normal(size=(M, K)), dtype)
    if targets is None:
        targets = rng.integers(0, V, M)
        targets[rng.random(M) < 0.2] = -1
    g = rng.normal(size=M).astype(np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales, targets)]
    kw = dict(group_size=group, nibble_order=order)
    xd = strided(x, layout)
    r = q4.head_cross_entropy(xd, *dev, **kw)
    loss, lse = oracle.cross_entropy(xv, w, targets)
    ez = product_bound(xv, 0 * xv, w, GIVEN[dtype])
    elz = ez.max(1)
    elp = elz + 2.0 ** -20 * (1 + np.abs(lse))
    assert_within(r.lse, lse, elp, "lse")
    assert_within(r.loss, loss, elp + elz + 2.0 ** -20 * (1 + np.abs(lse)) + 2.0 ** -23 * np.abs(np.nan_to_num(loss)), "loss")
    out = strided(torch.zeros_like(x), layout)
    # with the exact lse in fp32
    lse32 = torch.from_numpy(lse).float()
    dx = q4.head_cross_entropy_backward(xd, *dev, lse32.cuda(), torch.from_numpy(g).cuda(), dx=out, **kw)
    assert dx.data_ptr() == out.data_ptr() and dx.dtype == TORCH[dtype]
    want = oracle.cross_entropy_grad(xv, w, targets, g.astype(np.float64))
    z = xv @ w.T
    p = np.exp(z - lse[:, None])
    # (the largest element of a row bounds the kept bits' absolute floor, 2^-39 of it)
    ed = np.abs(g)[:, None] * (p * (ez + elz[:, None] + 2.0 ** -20 * (1 + np.abs(z)) + 2.0 ** -23 * np.abs(lse)[:, None])
                               + 2.0 ** -23 * (np.arange(V)[None] == targets[:, None]) + 2.0 ** -39)
    ed[targets < 0] = 0
    hot = (np.arange(V)[None] == targets[:, None]).astype(float)
    d = np.abs((p - hot) * g[:, None])
    d[targets < 0] = 0
    a = np.abs(w)
    bound = ed @ a + (KEPT[dtype] + 2.0 ** -24 + sums(V)) * (d @ a)
    assert_within(dx, want, bound + HALF_STEP[dtype] * (np.abs(want) + bound) + 2.0 ** -25, "dx")
    return out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M,V,K", [(1, 1, 8), (1, 1003, 256), (3, 129, 72), (65, 640, 264), (200, 300, 136)])
def test_parity(M, V, K, group, dtype):
    check(M, V, K, group, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_vocabularies_of_several_pieces_and_low_first(dtype):
    check(300, 5000, 64, 32, dtype, order="low_first")
    check(2, 70000, 40, 0, dtype, order="low_first")


@pytest.mark.parametrize("layout", ["wide", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_strides(layout, dtype):
    out = check(70, 300, 104, 64, dtype, layout=layout)
    if layout == "wide":
        assert out._base[:, :8].isnan().all() and out._base[:, 112:].isnan().all()


def test_far_logits_and_targets():
    """Sharp rows (logits of some hundreds), every target none, targets past the vocabulary."""
    check(20, 200, 128, 0, "f32", gain=100.0)
    check(20, 200, 128, 0, "f32", targets=np.full(20, -5))
    t = np.arange(20)
    t[3], t[7] = 200, 1 << 40
    check(20, 200, 128, 32, "bf16", targets=t)


def test_infinities_stay_in_their_row():
    M, V, K = 70, 500, 64
    codes, scales = packed(np.random.default_rng(0), (), V, K, 32)
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales)]
    x = torch.randn(M, K).cuda()
    t = torch.randint(0, V, (M,)).cuda()
    g = torch.randn(M).cuda()
    a = q4.head_cross_entropy(x, *dev, t, group_size=32)
    da = q4.head_cross_entropy_backward(x, *dev, t, a.lse, g, group_size=32)
    x[4, 3], x[9, 1] = float("inf"), float("nan")
    b = q4.head_cross_entropy(x, *dev, t, group_size=32)
    db = q4.head_cross_entropy_backward(x, *dev, t, b.lse, g, group_size=32)
    rest = torch.ones(M, dtype=torch.bool)
    rest[[4, 9]] = False
    assert b.loss[[4, 9]].isnan().all() and db[[4, 9]].isnan().all()
    assert torch.equal(a.loss[rest], b.loss[rest]) and torch.equal(da[rest], db[rest])


@pytest.mark.parametrize("M", [5, 300])
def test_gradient_scale_and_zero(M):
    codes, scales = packed(np.random.default_rng(0), (), 700, 64, 0)
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales)]
    x, t, g = torch.randn(M, 64).cuda(), torch.randint(0, 700, (M,)).cuda(), torch.randn(M).cuda()
    lse = q4.head_cross_entropy(x, *dev, t, group_size=0).lse
    f = lambda v: q4.head_cross_entropy_backward(x, *dev, t, lse, v, group_size=0)  # noqa: E731
    assert torch.equal(f(g * 2.0 ** -100), f(g) * 2.0 ** -100)
    assert (f(torch.zeros_like(g)) == 0).all()


def test_agrees_with_the_layer_and_token_logprobs():
    """The same head through linear, token_logprobs and linear_backward, in fp32 throughout."""
    M, V, K = 7, 2001, 256
    codes, scales = packed(np.random.default_rng(0), (), V, K, 0)
    qw, s = torch.from_numpy(codes).cuda(), torch.from_numpy(2.5 * scales).cuda()
    x, t, g = torch.randn(M, K).cuda(), torch.randint(0, V, (M,)).cuda(), torch.randn(M).cuda()
    logits = q4.linear(x, qw, s, group_size=0, math="f32")
    r = q4.token_logprobs(logits, t)
    d = q4.token_logprobs_backward(logits, t, r.lse, r.entropy, -g)
    want = q4.linear_backward(d, qw, s, K=K, group_size=0, math="f32")
    h = q4.head_cross_entropy(x, qw, s, t, group_size=0)
    dx = q4.head_cross_entropy_backward(x, qw, s, t, h.lse, g, group_size=0)
    assert torch.allclose(h.loss, -r.logprob, rtol=0, atol=1e-4) and torch.allclose(h.lse, r.lse, rtol=0, atol=1e-4)
    assert torch.allclose(dx, want, rtol=0, atol=1e-4 * want.abs().max().item())


def test_captured_graph_and_many_rows():
    M, V, K = 8300, 300, 64  # more rows than are taken at a time
    codes, scales = packed(np.random.default_rng(0), (), V, K, 32)
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales)]
    x, g = torch.randn(M, K).cuda(), torch.randn(M).cuda()
    t = torch.randint(0, V, (M,)).cuda()

    def step():
        r = q4.head_cross_entropy(x, *dev, t, group_size=32)
        return r.loss, q4.head_cross_entropy_backward(x, *dev, t, r.lse, g, group_size=32)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(3):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        want = [o.clone() for o in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    # rows of the last part alone
    part = q4.head_cross_entropy(x[8192:], *dev, t[8192:], group_size=32)
    assert torch.allclose(part.loss, outs[0][8192:], rtol=0, atol=1e-4)


def test_no_rows():
    codes, scales = packed(np.random.default_rng(0), (), 10, 64, 32)
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales)]
    x, t = torch.empty(0, 64).cuda(), torch.empty(0, dtype=torch.int64).cuda()
    r = q4.head_cross_entropy(x, *dev, t, group_size=32)
    assert r.loss.shape == (0,)
    assert q4.head_cross_entropy_backward(x, *dev, t, r.lse, r.loss, group_size=32).shape == (0, 64)
