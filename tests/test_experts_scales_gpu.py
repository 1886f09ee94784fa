"""Gradients where a matrix's groups have scales far apart: a column's bits are
those of its own group.  Bounds as in experts_util.py."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import GIVEN, HALF_STEP, KEPT, assert_within, expert_grad_bounds, packed, product_bound, rounded, sums
from tests.test_experts_gpu import Layer

pytestmark = pytest.mark.gpu


def far(groups):
    """Factors of the groups: every other one far below the rest."""
    return np.where(np.arange(groups) % 2 == 0, 2.0 ** -24, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 192])
@pytest.mark.parametrize("T,E", [(3, 4), (150, 2), (700, 2)])
def test_experts(T, E, group, dtype):
    layer = Layer(E, 392, 264, group)
    for scales, at in ((layer.gus, 1), (layer.dns, 3)):
        scales *= far(scales.shape[1])[None, :, None].astype(np.float32)
        layer.dev[at] = torch.from_numpy(scales).cuda()
    layer.gate_up = [oracle.matrix(layer.gu[e], layer.gus[e], group) for e in range(E)]
    layer.down = [oracle.matrix(layer.dn[e], layer.dns[e], group) for e in range(E)]
    rng = np.random.default_rng(1)
    d, dv = rounded(rng.normal(size=(T, layer.H)), dtype)
    pre = rng.normal(size=(T, 2, 2 * layer.W)).astype(np.float32)
    ids, w = layer.slots(T, 2, 1)
    dx, dw = q4.experts_backward(d.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(),
                                 torch.from_numpy(pre).cuda(), *layer.dev, **layer.kw)
    pick = np.unique(np.linspace(0, T - 1, min(T, 20)).astype(int))
    at = torch.from_numpy(pick).cuda()
    args = (dv[pick], ids[pick], w[pick].astype(np.float64), pre[pick].astype(np.float64), layer.gate_up, layer.down)
    dxw, dww = oracle.experts_grad(*args)
    edx, edw = expert_grad_bounds(*args, dtype, oracle.sigmoid)
    # (without a floor: the type's smallest step is far below the smallest group's gradients)
    assert_within(dx[at], dxw, edx + HALF_STEP[dtype] * (np.abs(dxw) + edx), "dx")
    assert_within(dw[at], dww, edw + 2.0 ** -24 * np.abs(dww), "dweights")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 192])
@pytest.mark.parametrize("M", [3, 300])
def test_head(M, group, dtype):
    V, K = 333, 264
    rng = np.random.default_rng(M)
    codes, scales = packed(rng, (), V, K, group)
    scales = (3 * scales * far(len(scales))[:, None]).astype(np.float32)
    w = oracle.matrix(codes, scales, group)
    x, xv = rounded(rng.normal(size=(M, K)), dtype)
    targets, g = rng.integers(0, V, M), rng.normal(size=M).astype(np.float32)
    lse = oracle.cross_entropy(xv, w, targets)[1]
    dx = q4.head_cross_entropy_backward(
        x.cuda(), *(torch.from_numpy(a).cuda() for a in (codes, scales, targets)), torch.from_numpy(lse).float().cuda(),
        torch.from_numpy(g).cuda(), group_size=group)
    want = oracle.cross_entropy_grad(xv, w, targets, g.astype(np.float64))
    z = xv @ w.T
    p = np.exp(z - lse[:, None])
    ez = product_bound(xv, 0 * xv, w, GIVEN[dtype])
    hot = np.arange(V)[None] == targets[:, None]
    ed = np.abs(g)[:, None] * (p * (ez + ez.max(1)[:, None] + 2.0 ** -20 * (1 + np.abs(z)) + 2.0 ** -23 * np.abs(lse)[:, None])
                               + 2.0 ** -23 * hot + 2.0 ** -39)
    a = np.abs(w)
    bound = ed @ a + (KEPT[dtype] + 2.0 ** -24 + sums(V)) * (np.abs((p - hot) * g[:, None]) @ a)
    assert_within(dx, want, bound + HALF_STEP[dtype] * (np.abs(want) + bound), "dx")
