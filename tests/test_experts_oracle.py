"""Pins of oracle/experts_oracle.py: hand-computed values, torch's autograd in
fp64, and mistakes planted in the oracle that the comparison has to notice."""
import math

import numpy as np
import pytest
import torch

from oracle import experts_oracle as o
from oracle import q4_oracle

RNG = np.random.default_rng(0)


@pytest.mark.parametrize("high", [False, True])
@pytest.mark.parametrize("group", [0, 32])
def test_matrix_is_the_layers(group, high):
    codes = RNG.integers(0, 256, (5, 32)).astype(np.uint8)
    scales = RNG.random(5 if group == 0 else (2, 5)).astype(np.float32)
    x = RNG.normal(size=(3, 64)).astype(np.float32)
    want, _ = q4_oracle.linear(x, codes, scales, None, K=64, group_size=group, order="high_first" if high else "low_first")
    assert np.allclose(x.astype(np.float64) @ o.matrix(codes, scales, group, high).T, want, rtol=1e-12, atol=1e-12)


def test_route_by_hand():
    z = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    ids, w = o.route(z, 2)
    assert ids.tolist() == [1, 2] and np.allclose(w, [4 / 6, 2 / 6])
    ids, w = o.route(z, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [1.0, 0.5])
    ids, w = o.route(z, 2, bias=[0.5, 0, 0, 0])  # scores 1/8 4/8 2/8 1/8
    assert ids.tolist() == [0, 1] and np.allclose(w, [1 / 5, 4 / 5])
    # groups (0, 1) and (2, 3): the first by its best, the second by the sum of two with a bias
    assert o.route(z, 2, groups=2, top_groups=1)[0].tolist() == [1, 0]
    assert o.route(z, 2, bias=[-0.4, 0, 0.1, 0.1], groups=2, top_groups=1)[0].tolist() == [2, 3]
    assert o.route([-math.inf, 0.0, -math.inf], 2)[0].tolist() == [1, -1]
    assert o.route([0.0, 0.0, 0.0], 2)[0].tolist() == [0, 1]
    assert np.allclose(o.route([0.0, 1.0], 1, "sigmoid", renormalize=False)[1], [1 / (1 + math.exp(-1))])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_is_autograds(kind, renormalize):
    z = torch.randn(9, dtype=torch.float64, requires_grad=True)
    g = np.array([0.3, -1.0, 2.0])
    ids = np.array([4, 0, 7])
    s = (torch.softmax(z, 0) if kind == "softmax" else torch.sigmoid(z))[torch.from_numpy(ids)]
    w = 1.5 * (s / s.sum() if renormalize else s)
    want, = torch.autograd.grad((w * torch.from_numpy(g)).sum(), z)
    assert np.allclose(o.route_grad(z.detach().numpy(), ids, g, kind, renormalize, 1.5), want.numpy(), atol=1e-14)


def test_experts_and_gradients_are_autograds():
    E, H, W, T, k = 3, 8, 6, 5, 2
    gu, dn = RNG.normal(size=(E, 2 * W, H)), RNG.normal(size=(E, H, W))
    ids = np.array([[0, 1], [2, -1], [1, 1], [-1, -1], [2, 0]])
    x = torch.randn(T, H, dtype=torch.float64, requires_grad=True)
    w = torch.rand(T, k, dtype=torch.float64, requires_grad=True)
    out = torch.zeros(T, H, dtype=torch.float64)
    pre = np.zeros((T, k, 2 * W))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                z = torch.from_numpy(gu[e]) @ x[t]
                pre[t, j] = z.detach().numpy()
                h = torch.nn.functional.silu(z[:W]) * z[W:]
                out = out.index_add(0, torch.tensor([t]), (w[t, j] * (torch.from_numpy(dn[e]) @ h))[None])
    xn, wn = x.detach().numpy(), w.detach().numpy()
    assert np.allclose(o.experts(xn, ids, wn, gu, dn), out.detach().numpy(), atol=1e-12)
    d = RNG.normal(size=(T, H))
    dx, dw = torch.autograd.grad(out, (x, w), torch.from_numpy(d))
    ox, ow = o.experts_grad(d, ids, wn, pre, gu, dn)
    assert np.allclose(ox, dx.numpy(), atol=1e-12) and np.allclose(ow, dw.numpy(), atol=1e-12)


def test_cross_entropy_is_torchs():
    x = torch.randn(6, 8, dtype=torch.float64, requires_grad=True)
    w = torch.randn(20, 8, dtype=torch.float64)
    t = torch.tensor([3, -1, 0, 19, 7, 7])
    loss = torch.nn.functional.cross_entropy(x @ w.t(), t, ignore_index=-1, reduction="none")
    g = torch.randn(6, dtype=torch.float64)
    dx, = torch.autograd.grad((loss * g).sum(), x)
    xn, wn, tn = x.detach().numpy(), w.numpy(), t.numpy()
    ol, olse = o.cross_entropy(xn, wn, tn)
    assert np.allclose(ol, loss.detach().numpy(), atol=1e-12)
    assert np.allclose(olse, torch.logsumexp(x @ w.t(), 1).detach().numpy(), atol=1e-12)
    assert np.allclose(o.cross_entropy_grad(xn, wn, tn, g.numpy()), dx.numpy(), atol=1e-12)
    assert math.isnan(o.cross_entropy(xn, wn, np.array([20] * 6))[0][0])


@pytest.mark.parametrize("mistake", ["swap gate and up", "no weight", "renormalised twice", "wrong nibble", "shifted target"])
def test_planted_mistakes_are_seen(mistake):
    """What the tests' bounds must be able to tell apart."""
    x = RNG.normal(size=(2, 16))
    gu, dn = RNG.normal(size=(1, 8, 16)), RNG.normal(size=(1, 16, 4))
    ids, w = np.zeros((2, 1), dtype=int), np.full((2, 1), 0.5)
    right = o.experts(x, ids, w, gu, dn)
    if mistake == "swap gate and up":
        other = o.experts(x, ids, w, np.concatenate([gu[:, 4:], gu[:, :4]], 1), dn)
    elif mistake == "no weight":
        other = o.experts(x, ids, 2 * w, gu, dn)
    elif mistake == "renormalised twice":
        right, other = o.route(x[0], 3, renormalize=False)[1], o.route(x[0], 3)[1]
    elif mistake == "wrong nibble":
        codes, s = RNG.integers(0, 256, (3, 8)).astype(np.uint8), np.ones(3, np.float32)
        right, other = o.matrix(codes, s, 0), o.matrix(codes, s, 0, True)
    else:
        head = RNG.normal(size=(9, 16))
        right, other = o.cross_entropy(x, head, [1, 2])[0], o.cross_entropy(x, head, [2, 3])[0]
    assert np.abs(right - other).max() > 1e-3
