"""The head's loss and gradient in several pieces of the vocabulary and several
parts of the rows, against fp64.  Bounds as in
test_head_loss_gpu.py, for some of the rows."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import GIVEN, HALF_STEP, KEPT, TORCH, assert_within, packed, product_bound, rounded, sums

pytestmark = pytest.mark.gpu


def check(M, V, K, group, dtype, some, order="low_first"):
    """`some`: the rows compared.  Returns the call's tensors."""
    rng = np.random.default_rng(M + V)
    codes, scales = packed(rng, (), V, K, group)
    scales = (2.5 * scales).astype(np.float32)
    x, xv = rounded(rng.normal(size=(M, K)), dtype)
    targets = rng.integers(0, V, M)
    targets[some] = np.linspace(0, V - 1, len(some)).astype(int)  # in every piece, the first and the last column
    targets[some[1]] = -1
    g = rng.normal(size=M).astype(np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (codes, scales, targets)]
    kw = dict(group_size=group, nibble_order=order)
    xd, gd = x.cuda(), torch.from_numpy(g).cuda()
    r = q4.head_cross_entropy(xd, *dev, **kw)
    dx = q4.head_cross_entropy_backward(xd, *dev, r.lse, gd, **kw)
    w, ts, gs, xs = oracle.matrix(codes, scales, group, order == "high_first"), targets[some], g[some], xv[some]
    loss, lse = oracle.cross_entropy(xs, w, ts)
    ez = product_bound(xs, 0 * xs, w, GIVEN[dtype])
    elz = ez.max(1)
    at = torch.from_numpy(some).cuda()
    elp = elz + 2.0 ** -20 * (1 + np.abs(lse))
    assert_within(r.lse[at], lse, elp, "lse")
    assert_within(r.loss[at], loss, elp + elz + 2.0 ** -20 * (1 + np.abs(lse)), "loss")
    want = oracle.cross_entropy_grad(xs, w, ts, gs.astype(np.float64))
    z = xs @ w.T
    p = np.exp(z - lse[:, None])
    hot = np.arange(V)[None] == ts[:, None]
    # (with the kernel's own lse: its error elp beside the logits')
    ed = np.abs(gs)[:, None] * (p * (ez + elp[:, None] + 2.0 ** -20 * (1 + np.abs(z)) + 2.0 ** -23 * np.abs(lse)[:, None])
                                + 2.0 ** -23 * hot + 2.0 ** -39)
    d = np.abs((p - hot) * gs[:, None])
    ed[ts < 0] = d[ts < 0] = 0
    a = np.abs(w)
    bound = ed @ a + (KEPT[dtype] + 2.0 ** -24 + sums(V)) * (d @ a)
    assert_within(dx[at], want, bound + HALF_STEP[dtype] * (np.abs(want) + bound) + 2.0 ** -25, "dx")
    return xd, dev, gd, r, dx, kw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V,K,group", [(2048, 70001, 64, 0), (2048, 70001, 64, 32), (1999, 40007, 72, 0), (1100, 129000, 136, 128)])
def test_pieces_of_the_vocabulary(M, V, K, group, dtype):
    # the workspace has fp32 room for one piece's gradient of the logits: less than all of them, so there are several
    assert q4.head_cross_entropy_backward_workspace_bytes(M, V, K, group_size=group, dtype=TORCH[dtype]) < 4 * M * V
    check(M, V, K, group, dtype, np.array([0, 1, 63, 64, 127, 128, 777, M - 2, M - 1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("M,V", [(8300, 300), (16500, 9001)])
def test_rows_in_several_parts(M, V, group, dtype):
    some = np.array([0, 1, 4000, 8190, 8191, 8192, 8193, 8250, M - 2, M - 1])
    x, (qw, s, t), g, r, dx, kw = check(M, V, 64, group, dtype, some)
    last = M // 8192 * 8192
    part = q4.head_cross_entropy(x[last:], qw, s, t[last:], **kw)
    assert torch.allclose(part.loss, r.loss[last:], rtol=0, atol=1e-4)
    dpart = q4.head_cross_entropy_backward(x[last:], qw, s, t[last:], r.lse[last:], g[last:], **kw)
    # two roundings to the type, and products that differ by their bound, far below 2^-11 of the largest
    top = dx[last:].double().abs().amax(1, keepdim=True)
    over = (dpart.double() - dx[last:].double()).abs() - 2 * HALF_STEP[dtype] * dx[last:].double().abs() - 2.0 ** -11 * top
    assert over.max().item() <= 0
