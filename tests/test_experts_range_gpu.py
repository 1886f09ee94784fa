"""Magnitudes between the products' steps: sums of activations times codes that
pass fp32's range before their scale brings them back, and gradients before the
gate's slope does.  Bounds as in experts_util.py."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import HALF_STEP, assert_within, expert_bounds, expert_grad_bounds, rounded
from tests.test_experts_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T", [1, 9, 40, 130])
@pytest.mark.parametrize("x_up,gate_down,down_down", [(123, 119, 0), (61.5, 0, 119)])
def test_sums_past_the_range_before_their_scale(T, group, dtype, x_up, gate_down, down_down):
    """Rows of 2^123 times scales of 2^-119 (of the gate and up, or of down behind rows of 2^61.5)."""
    layer = Layer(8, 128, 64, group)
    layer.gate_up = [m * 2.0 ** -gate_down for m in layer.gate_up]
    layer.down = [m * 2.0 ** -down_down for m in layer.down]
    for i, by in ((1, gate_down), (3, down_down)):
        layer.dev[i] = layer.dev[i] * 2.0 ** -by
    x, xv = rounded(np.random.default_rng(1).normal(size=(T, layer.H)) * 2.0 ** x_up, dtype)
    ids, w = layer.slots(T, 2, 1)
    got, pre = q4.experts(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), *layer.dev, **layer.kw,
                          keep=True)
    want = oracle.experts(xv, ids, w.astype(np.float64), layer.gate_up, layer.down)
    pre_want, epre, e = expert_bounds(xv, ids, w, layer.gate_up, layer.down, dtype, oracle.sigmoid)
    assert torch.isfinite(got).all()
    assert_within(pre, pre_want, epre, "pre")
    assert_within(got, want, e + HALF_STEP[dtype] * (np.abs(want) + e) + 2.0 ** -25, "out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 150])
def test_gradients_of_closed_gates(T, dtype):
    """The output's gradient times a large up passes the range where the gate's slope brings it back."""
    layer = Layer(8, 64, 32, 32)
    rng = np.random.default_rng(2)
    d, dv = rounded(rng.normal(size=(T, layer.H)) * 1e18, dtype)
    pre = np.concatenate([rng.uniform(-75, -60, (T, 2, layer.W)), 1e24 * rng.normal(size=(T, 2, layer.W))], 2).astype(np.float32)
    ids, w = layer.slots(T, 2, 1)
    dx, dw = q4.experts_backward(d.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(),
                                 torch.from_numpy(pre).cuda(), *layer.dev, **layer.kw)
    args = (dv, ids, w.astype(np.float64), pre.astype(np.float64), layer.gate_up, layer.down)
    dxw, dww = oracle.experts_grad(*args)
    edx, edw = expert_grad_bounds(*args, dtype, oracle.sigmoid)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert_within(dx, dxw, edx + HALF_STEP[dtype] * (np.abs(dxw) + edx), "dx")
    assert_within(dw, dww, edw + 2.0 ** -24 * np.abs(dww), "dweights")
