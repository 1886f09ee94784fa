"""Sigmoid scores too small for fp32 keep their shares where they are divided by
their sum.  Bounds as in test_route_gpu.py."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import HALF_STEP, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("low,high", [(-130.0, -95.0), (-600.0, -590.0), (-89.0, -85.0), (-3.0, 3.0), (30.0, 90.0)])
def test_shares_of_small_scores(low, high, bias, dtype):
    T, E, k = 9, 40, 5
    rng = np.random.default_rng(3)
    z, zv = rounded(rng.uniform(low, high, (T, E)), dtype)
    b = rng.normal(size=E).astype(np.float32) if bias else None
    r = q4.route(z.cuda(), k, score="sigmoid", bias=None if b is None else torch.from_numpy(b).cuda(), scale=1.5)
    g = rng.normal(size=(T, k)).astype(np.float32)
    dz = q4.route_backward(z.cuda(), r.ids, torch.from_numpy(g).cuda(), score="sigmoid", scale=1.5)
    for t in range(T):
        ids, w = oracle.route(zv[t], k, "sigmoid", b, scale=1.5)
        assert r.ids[t].tolist() == ids.tolist()
        assert (np.abs(r.weights[t].double().cpu().numpy() - w) <= 32 * 2.0 ** -24 * w).all()
        want = oracle.route_grad(zv[t], ids, g[t].astype(np.float64), "sigmoid", True, 1.5)
        s = oracle.scores(zv[t], "sigmoid")
        part = np.zeros(E)
        part[ids] = s[ids] / s[ids].sum()
        terms = 1.5 * part * (np.abs(g[t]).max() + (np.abs(g[t]) * part[ids]).sum())
        bound = 64 * 2.0 ** -24 * terms + HALF_STEP[dtype] * np.abs(want) + 2.0 ** -25
        assert (np.abs(dz[t].double().cpu().numpy() - want) <= bound).all()
