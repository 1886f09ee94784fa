"""16-bit types lose nothing between the products: what is computed on the way
(the gated rows, gradients, probabilities) is held to 22 bits whatever the
activations' type, so only the output's own rounding is the type's.

Bounds are those of experts_util.py with 2^-22 for the kept values of every
type.  Few terms a sum, so that its roundings do not cover those of 11 bits:
2^-12 of single terms against sums(64) = 28 * 2^-23 of all of them."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests import experts_util as u
from tests.experts_util import HALF_STEP, assert_within, rounded
from tests.test_experts_gpu import Layer
from tests.test_head_loss_gpu import check as check_head

pytestmark = pytest.mark.gpu
WAYS = [(1, 8, 2), (9, 8, 2), (40, 8, 2), (130, 8, 2), (1400, 2, 1)]  # T, experts, top_k


@pytest.fixture(autouse=True)
def kept(monkeypatch):
    for t in ("f16", "bf16"):
        monkeypatch.setitem(u.KEPT, t, 2.0 ** -22)


def inputs(layer, T, k, dtype, seed=1):
    x, xv = rounded(np.random.default_rng(seed).normal(size=(T, layer.H)), dtype)
    ids, w = layer.slots(T, k, seed)
    pick = np.unique(np.linspace(0, T - 1, min(T, 40)).astype(int))
    return x.cuda(), xv[pick], ids, w, pick


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T,E,k", WAYS)
def test_gated_rows(T, E, k, group, dtype):
    layer = Layer(E, 128, 64, group)
    x, xv, ids, w, pick = inputs(layer, T, k, dtype)
    got = q4.experts(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *layer.dev, **layer.kw)
    want = oracle.experts(xv, ids[pick], w[pick].astype(np.float64), layer.gate_up, layer.down)
    e = u.expert_bounds(xv, ids[pick], w[pick], layer.gate_up, layer.down, dtype, oracle.sigmoid)[2]
    assert_within(got[torch.from_numpy(pick).cuda()], want, e + HALF_STEP[dtype] * (np.abs(want) + e) + 2.0 ** -25, "out")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T,E,k", WAYS)
def test_gradients_of_gate_and_up(T, E, k, group, dtype):
    layer = Layer(E, 128, 32, group)
    d, dv, ids, w, pick = inputs(layer, T, k, dtype)
    pre = np.random.default_rng(2).normal(size=(T, k, 64)).astype(np.float32)
    dx, _ = q4.experts_backward(d, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(),
                                torch.from_numpy(pre).cuda(), *layer.dev, **layer.kw)
    args = (dv, ids[pick], w[pick].astype(np.float64), pre[pick].astype(np.float64), layer.gate_up, layer.down)
    want = oracle.experts_grad(*args)[0]
    e = u.expert_grad_bounds(*args, dtype, oracle.sigmoid)[0]
    assert_within(dx[torch.from_numpy(pick).cuda()], want, e + HALF_STEP[dtype] * (np.abs(want) + e) + 2.0 ** -25, "dx")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("M,V", [(3, 129), (70, 200), (400, 136)])
def test_heads_gradient(M, V, group, dtype):
    check_head(M, V, 72, group, dtype)
