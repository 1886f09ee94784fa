"""Routing and its gradient on the GPU against the fp64 oracle.

Choices have to be equal: values are distinct fp32 or 16-bit numbers, equal
ones go to the lowest index, and with a bias the kernel forms the sums in 64
bits as the oracle does.  Weights: exponentials and the division are each good
to 2 or 3 units in the last place and a sum of up to 512 terms in 6 + 8 steps
to 14 half units: 32 * 2^-24 of the value.  Gradients: the differences g - mean
and ds - mean cancel, so their bound is relative to the terms, 64 * 2^-24 of
s (|g| + sum |g| s), plus the type's rounding."""
import math

import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import HALF_STEP, TORCH, rounded

pytestmark = pytest.mark.gpu
WAYS = [dict(), dict(kind="sigmoid"), dict(renormalize=False), dict(kind="sigmoid", renormalize=False, scale=2.5),
        dict(bias=True), dict(kind="sigmoid", bias=True, scale=0.5), dict(groups=4, top_groups=2),
        dict(kind="sigmoid", bias=True, groups=4, top_groups=3), dict(kind="softmax", bias=True, groups=2, top_groups=1)]


def own(way):
    d = {k: v for k, v in way.items() if k not in ("kind", "bias")}
    return dict(score=way.get("kind", "softmax"), **d)


def logits(T, E, dtype, seed, holes=0.0):
    rng = np.random.default_rng(seed)
    z = 2.0 * rng.normal(size=(T, E))
    z[rng.random((T, E)) < holes] = -math.inf
    return rounded(z, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (5, 60, 4), (3, 64, 8), (9, 128, 5), (2, 256, 8), (3, 384, 10), (2, 1000, 32)])
@pytest.mark.parametrize("way", WAYS)
def test_choice_and_gradient(T, E, k, dtype, way):
    rng = np.random.default_rng(E)
    z, zv = logits(T, E, dtype, E + k)
    bias = 0.3 * rng.normal(size=E).astype(np.float32) if way.get("bias") else None
    if k > E // way.get("groups", 1) * way.get("top_groups", 1):
        pytest.skip("more experts than the groups hold")
    kw = own(way)
    args = {**way, "bias": bias}
    r = q4.route(z.cuda(), k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    g = rng.normal(size=(T, k)).astype(np.float32)
    kw2 = {n: v for n, v in kw.items() if n in ("score", "renormalize", "scale")}
    dz = q4.route_backward(z.cuda(), r.ids, torch.from_numpy(g).cuda(), **kw2)
    for t in range(T):
        ids, w = oracle.route(zv[t], k, **args)
        assert r.ids[t].tolist() == ids.tolist()
        got = r.weights[t].double().cpu().numpy()
        assert (np.abs(got - w) <= 32 * 2.0 ** -24 * np.abs(w)).all()
        gw = {n: v for n, v in args.items() if n in ("kind", "renormalize", "scale")}
        want = oracle.route_grad(zv[t], ids, g[t].astype(np.float64), **gw)
        s = oracle.scores(zv[t], args.get("kind", "softmax"))
        part = s / s[ids].sum() if args.get("renormalize", True) else s
        terms = part * (np.abs(g[t]).max() + (np.abs(g[t]) * part[ids]).sum()) * abs(args.get("scale", 1.0))
        bound = 64 * 2.0 ** -24 * terms + HALF_STEP[dtype] * np.abs(want) + 2.0 ** -25  # fp16 subnormals
        assert (np.abs(dz[t].double().cpu().numpy() - want) <= bound).all()
    assert dz.dtype == TORCH[dtype]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(kind, renormalize):
    rng = np.random.default_rng(3)
    z, ids, g = rng.normal(size=24), np.array([3, 17, 8]), rng.normal(size=3)

    def f(v):
        s = oracle.scores(v, kind)[ids]
        return np.dot(g, s / s.sum() if renormalize else s)

    step = 1e-5
    want = np.array([(f(z + step * e) - f(z - step * e)) / (2 * step) for e in np.eye(24)])
    got = q4.route_backward(torch.from_numpy(z).float()[None].cuda(), torch.tensor([ids.tolist()], dtype=torch.int32).cuda(),
                            torch.from_numpy(g).float()[None].cuda(), score=kind, renormalize=renormalize)
    # differences of values near 1: 1e-16 / 1e-5 and a third derivative's 1e-10; the kernel's 64 * 2^-24 of terms below 4
    assert np.abs(got[0].double().cpu().numpy() - want).max() <= 2e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way", [dict(), dict(kind="sigmoid", bias=True), dict(groups=5, top_groups=3),
                                 dict(bias=True, groups=5, top_groups=2)])
def test_masked_experts(dtype, way):
    T, E, k = 40, 20, 8
    z, zv = logits(T, E, dtype, 1, holes=0.6)
    z[0], zv[0] = -math.inf, -math.inf  # nothing is left
    z[1], zv[1] = -math.inf, -math.inf
    z[1, 7], zv[1, 7] = 1.0, 1.0
    bias = np.linspace(3, -3, E).astype(np.float32) if way.get("bias") else None
    r = q4.route(z.cuda(), k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **own(way))
    dz = q4.route_backward(z.cuda(), r.ids, torch.ones(T, k).cuda(), score=way.get("kind", "softmax"))
    for t in range(T):
        ids, w = oracle.route(zv[t], k, **{**way, "bias": bias})
        assert r.ids[t].tolist() == ids.tolist()
        assert (np.abs(r.weights[t].double().cpu().numpy() - w) <= 32 * 2.0 ** -24 * w).all()
    assert torch.isfinite(dz).all() and (dz[0] == 0).all()


def test_ties_go_to_the_lowest_index():
    z = torch.zeros(3, 96).cuda()
    z[1, 50] = z[1, 20] = 1.0
    z[2] = -0.0
    z[2, 90] = 0.0
    for kw in (dict(), dict(bias=torch.zeros(96).cuda()), dict(groups=8, top_groups=2)):
        ids = q4.route(z, 5, **kw).ids.tolist()
        assert ids[0] == [0, 1, 2, 3, 4] and ids[2] == [0, 1, 2, 3, 4]
        assert ids[1][:2] == [20, 50]


def test_nan_and_infinity_reach_the_weights():
    z = torch.randn(4, 70).cuda()
    z[1, 3] = float("nan")
    z[2, 5] = float("inf")
    z[3] = float("nan")
    for bias in (None, torch.zeros(70).cuda()):
        r = q4.route(z, 4, bias=bias)
        assert torch.isfinite(r.weights[0]).all() and r.weights[1:].isnan().all()
        assert (r.ids >= 0).all() and r.ids[2, 0] == 5 and r.ids[3].tolist() == [0, 1, 2, 3]
        s = q4.route(z, 4, bias=bias, score="sigmoid")
        assert s.weights[1].isnan().all() and torch.isfinite(s.weights[2]).all() and s.ids[2, 0] == 5
        g = torch.ones(4, 4).cuda()
        d = q4.route_backward(z, r.ids, g)
        assert torch.isfinite(d[0]).all() and d[1:].isnan().all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_apart_logits(score):
    """Chosen scores far below the largest keep their shares; scores of 0 give weights of 0."""
    z = torch.full((2, 8), -90.0).cuda()
    z[0, 0] = 80.0
    z[1] = -3e38
    r = q4.route(z, 3, score=score, bias=torch.tensor([-9.0] + [0.0] * 7).cuda())
    assert torch.isfinite(r.weights).all()
    want = oracle.route(z[0].cpu().numpy(), 3, score, [-9.0] + [0.0] * 7)
    assert r.ids[0].tolist() == want[0].tolist()
    if score == "softmax":
        assert np.allclose(r.weights[0].cpu().numpy(), 1 / 3)
    d = q4.route_backward(z, r.ids, torch.randn(2, 3).cuda(), score=score)
    assert torch.isfinite(d).all()


def test_strides_in_place_and_bad_ids():
    z = torch.randn(6, 50)
    wide = torch.full((6, 61), float("nan")).cuda()
    wide[:, 3:53] = z.cuda()
    a, b = q4.route(wide[:, 3:53], 4), q4.route(z.cuda(), 4)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.weights, b.weights)
    g = torch.randn(6, 4).cuda()
    ids = b.ids.clone()
    ids[2, 1] = 50  # names no expert
    ids[3, 1] = -1
    want = q4.route_backward(z.cuda(), ids, g)
    assert want[2].isnan().all() and torch.isfinite(want[[0, 1, 3, 4, 5]]).all()
    got = q4.route_backward(wide[:, 3:53], ids, g, dlogits=wide[:, 3:53])
    assert got.data_ptr() == wide[:, 3:53].data_ptr()
    assert torch.equal(got[3:], want[3:]) and wide[:, :3].isnan().all() and wide[:, 53:].isnan().all()


def test_no_tokens():
    r = q4.route(torch.empty(0, 8).cuda(), 2)
    assert r.ids.shape == (0, 2)
    assert q4.route_backward(torch.empty(0, 8).cuda(), r.ids, r.weights).shape == (0, 8)


@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 64, 10, 8), (128, 64, 5, 7), (256, 16, 3, 10), (160, 8, 3, 6),
                                                   (96, 8, 4, 8), (512, 32, 6, 32), (1024, 2, 1, 5), (1024, 512, 9, 4), (48, 3, 2, 9)])
@pytest.mark.parametrize("way", [dict(), dict(bias=True), dict(kind="sigmoid", bias=True)])
def test_groups_of_any_size(E, groups, top_groups, k, way):
    """Groups of whole lanes and others, with equal and masked logits among them."""
    z, zv = logits(33, E, "bf16", E + groups, holes=0.2)
    z[5] = z[6] = 0.5
    zv[5] = zv[6] = 0.5
    bias = np.random.default_rng(1).normal(size=E).astype(np.float32) if way.get("bias") else None
    if bias is not None:
        bias[: E // 2] = bias[0]
    r = q4.route(z.cuda(), k, bias=None if bias is None else torch.from_numpy(bias).cuda(), groups=groups,
                 top_groups=top_groups, score=way.get("kind", "softmax"))
    for t in range(33):
        ids, w = oracle.route(zv[t], k, **{**way, "bias": bias}, groups=groups, top_groups=top_groups)
        assert r.ids[t].tolist() == ids.tolist()
        assert (np.abs(r.weights[t].double().cpu().numpy() - w) <= 32 * 2.0 ** -24 * w).all()
