"""Packed experts in every way their kernels divide the work (by depth, number
of experts and rows of an expert), and a step of routing, experts and head with
all its gradients.  Bounds as in experts_util.py, for a few of the tokens."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import HALF_STEP, TORCH, assert_within, expert_bounds, expert_grad_bounds, packed, rounded
from tests.test_experts_gpu import Layer
from tests.test_experts_gpu import check as check_layer

pytestmark = pytest.mark.gpu


class Matrices:
    """One expert's matrix in fp64 when it is asked for."""

    def __init__(self, codes, scales, group):
        self.codes, self.scales, self.group = codes, scales, group

    def __getitem__(self, e):
        return oracle.matrix(self.codes[e], self.scales[e], self.group, False)


def check(E, H, W, group, T, k, dtype, some=5, backward=True, spread=0):
    """ids of a few experts more often than the others where spread > 0."""
    rng = np.random.default_rng(E + H + W + T)
    gu, gus = packed(rng, (E,), 2 * W, H, group)
    dn, dns = packed(rng, (E,), H, W, group)
    dev = [torch.from_numpy(a).cuda() for a in (gu, gus, dn, dns)]
    x, xv = rounded(rng.normal(size=(T, H)), dtype)
    d, dv = rounded(rng.normal(size=(T, H)), dtype)
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)], dtype=np.int32)
    if spread:
        ids[::2] %= spread
    w = rng.random((T, k)).astype(np.float32)
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    got, pre = q4.experts(x.cuda(), it, wt, *dev, group_size=group, keep=True)
    pick = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, some)]))
    gate_up, down = Matrices(gu, gus, group), Matrices(dn, dns, group)
    xs, ds, ip, wp = xv[pick], dv[pick], ids[pick], w[pick]

    def one(m):  # the first 2 * W rows alone tell the width
        return [m[e] if e in ip else m[0] if e == 0 else None for e in range(E)]

    mg, md = one(gate_up), one(down)
    pre_want, epre, eout = expert_bounds(xs, ip, wp, mg, md, dtype, oracle.sigmoid)
    want = oracle.experts(xs, ip, wp.astype(np.float64), mg, md)
    at = torch.from_numpy(pick).cuda()
    assert_within(pre[at], pre_want, epre, "pre")
    assert_within(got[at], want, eout + HALF_STEP[dtype] * (np.abs(want) + eout) + 2.0 ** -25, "out")
    if not backward:
        return
    pre32 = pre.clone()
    pre32[at] = torch.from_numpy(pre_want).float().cuda()
    pv = pre32[at].double().cpu().numpy()
    dx, dw = q4.experts_backward(d.cuda(), it, wt, pre32, *dev, group_size=group)
    dxw, dww = oracle.experts_grad(ds, ip, wp.astype(np.float64), pv, mg, md)
    edx, edw = expert_grad_bounds(ds, ip, wp, pv, mg, md, dtype, oracle.sigmoid)
    assert_within(dx[at], dxw, edx + HALF_STEP[dtype] * (np.abs(dxw) + edx) + 2.0 ** -25, "dx")
    assert_within(dw[at], dww, edw + 2.0 ** -24 * np.abs(dww), "dweights")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 64, 128])
@pytest.mark.parametrize("E,H,W,T", [(140, 32, 512, 70), (140, 1024, 32, 70), (64, 2080, 1024, 96), (64, 2048, 2080, 96)])
def test_workgroups_of_several_column_blocks(E, H, W, T, group, dtype):
    check(E, H, W, group, T, 2, dtype, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T,E", [(2, 4), (7, 4), (30, 3)])
@pytest.mark.parametrize("H,W", [(2056, 24), (24, 2056), (2080, 32), (4640, 32), (32, 4640), (8232, 16), (16, 8232)])
def test_depths(H, W, T, E, group, dtype):
    check(E, H, W, group, T, 2, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("E,T,k", [(2, 700, 1), (1, 1100, 1), (3, 1100, 3)])
def test_experts_of_many_rows(E, T, k, group, dtype):
    check(E, 136, 72, group, T, k, dtype, some=24)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 250, 900])
def test_uneven_experts(T, dtype):
    check(24, 264, 200, 64, T, 2, dtype, some=24, spread=3)


class Step:
    """Rows through the choice of experts, the experts and the head; all gradients."""

    def __init__(self, M, E, H, W, V, k, group, seed=0):
        rng = np.random.default_rng(seed)
        self.k, self.group = k, group
        self.gu, self.gus = packed(rng, (E,), 2 * W, H, group)
        self.dn, self.dns = packed(rng, (E,), H, W, group)
        self.hw, self.hs = packed(rng, (), V, H, 0)
        self.x = rng.normal(size=(M, H)).astype(np.float32)
        self.z = rng.normal(size=(M, E)).astype(np.float32)
        self.targets = rng.integers(0, V, M)
        self.targets[::5] = -1
        self.g = np.full(M, 1.0 / M, dtype=np.float32)
        self.dev = {n: torch.from_numpy(getattr(self, n)).cuda()
                    for n in ("gu", "gus", "dn", "dns", "hw", "hs", "x", "z", "targets", "g")}

    def run(self, workspace=None):
        t, kw = self.dev, dict(group_size=self.group, nibble_order="low_first", workspace=workspace)
        head = dict(group_size=0, nibble_order="low_first", workspace=workspace)
        mats = (t["gu"], t["gus"], t["dn"], t["dns"])
        r = q4.route(t["z"], self.k)
        y, pre = q4.experts(t["x"], r.ids, r.weights, *mats, keep=True, **kw)
        hidden = t["x"] + y
        loss = q4.head_cross_entropy(hidden, t["hw"], t["hs"], t["targets"], **head)
        dh = q4.head_cross_entropy_backward(hidden, t["hw"], t["hs"], t["targets"], loss.lse, t["g"], **head)
        dx, dw = q4.experts_backward(dh, r.ids, r.weights, pre, *mats, **kw)
        dz = q4.route_backward(t["z"], r.ids, dw)
        return loss.loss, dh + dx, dw, dz, r.ids

    def want(self, ids):
        E, x, z = self.gu.shape[0], self.x.astype(np.float64), self.z.astype(np.float64)
        gate_up = [oracle.matrix(self.gu[e], self.gus[e], self.group, False) for e in range(E)]
        down = [oracle.matrix(self.dn[e], self.dns[e], self.group, False) for e in range(E)]
        head = oracle.matrix(self.hw, self.hs, 0, False)
        w = np.exp(np.take_along_axis(z, ids.astype(np.int64), 1))
        w /= w.sum(1, keepdims=True)
        hidden = x + oracle.experts(x, ids, w, gate_up, down)
        loss, _ = oracle.cross_entropy(hidden, head, self.targets)
        dh = oracle.cross_entropy_grad(hidden, head, self.targets, self.g.astype(np.float64))
        pre = np.array([[gate_up[e] @ x[t] for e in ids[t]] for t in range(len(x))])
        dx, dw = oracle.experts_grad(dh, ids, w, pre, gate_up, down)
        dz = np.array([oracle.route_grad(z[t], ids[t], dw[t]) for t in range(len(x))])
        return loss, dh + dx, dw, dz


@pytest.mark.parametrize("M,E,k,group", [(1, 4, 2, 32), (5, 8, 3, 64), (40, 6, 2, 0), (300, 5, 2, 128)])
def test_step_of_router_experts_and_head(M, E, k, group):
    s = Step(M, E, 64, 40, 203, k, group)
    got = s.run()
    want = s.want(got[4].cpu().numpy())
    # six products in turn, each off by sums(203) + 2^-22 = 5.7e-6 of its terms; the terms of a sum of
    # up to 203 are on average 0.8 of the largest and their sum about 14 times the result's size:
    # 6 * 14 * 0.8 * 5.7e-6 = 4e-4; s (dw - mean) is off by at most twice what dw is
    sizes = [np.abs(b).max() for b in want]
    sizes[3] = 2 * sizes[2]
    for a, b, size, what in zip(got, want, sizes, ("loss", "dx", "dweights", "dlogits")):
        assert np.abs(a.double().cpu().numpy() - b).max() <= 4e-4 * size, what


@pytest.mark.parametrize("M", [4, 200])
def test_steps_at_once_and_captured(M):
    """Two steps on two streams at the same time; two graphs that share a workspace, replayed in turn."""
    steps = [Step(M, 6, 128, 72, 1003, 2, 32, seed) for seed in (0, 1)]
    eager = [[t.clone() for t in s.run()] for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                outs.append(s.run())
        torch.cuda.synchronize()
        for got, want in zip(outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    n = max(q4.experts_workspace_bytes(M, 128, 72, 6, 2, group_size=32),
            q4.experts_backward_workspace_bytes(M, 128, 72, 6, 2, group_size=32),
            q4.head_cross_entropy_workspace_bytes(M, 1003, 128, group_size=0),
            q4.head_cross_entropy_backward_workspace_bytes(M, 1003, 128, group_size=0))
    workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, held = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(s.run(workspace))
        graphs.append(g)
    for turn in range(3):
        for s in steps:
            for n in ("x", "z"):
                s.dev[n].normal_(generator=torch.Generator(device="cuda").manual_seed(turn))
        want = [[t.clone() for t in s.run()] for s in steps]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got, w in zip(held, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 6), (3, 2), (11, 4)])
def test_few_slots_of_many_experts(T, k, dtype):
    """Slots that look for their expert's other rows themselves: spread, all of
    one expert, one expert several times in a token, empty ones."""
    layer = Layer(48, 264, 72, 32)
    ids = np.random.default_rng(T).integers(0, 48, (T, k)).astype(np.int32)
    check_layer(layer, T, k, dtype, ids=ids)
    check_layer(layer, T, k, dtype, ids=np.full((T, k), 47, dtype=np.int32))
    check_layer(layer, T, k, dtype, ids=(ids % 2).astype(np.int32))
    check_layer(layer, T, k, dtype, empty=0.6)
    check_layer(layer, T, k, dtype, ids=np.full((T, k), -1, dtype=np.int32), layout="wide")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_few_slots_with_bad_ids_and_rows(dtype):
    layer = Layer(40, 264, 72, 64)
    ids, w = layer.slots(6, 3, 0)
    x = torch.randn(6, 264).to(TORCH[dtype]).cuda()
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    it[3] = it[0]
    good, pre = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True)
    order = torch.tensor([4, 0, 5, 2, 1, 3]).cuda()
    again, pre2 = q4.experts(x[order], it[order], wt[order], *layer.dev, **layer.kw, keep=True)
    assert torch.equal(again, good[order]) and torch.equal(pre2, pre[order])
    rest = torch.arange(6) != 1
    it2, x2 = it.clone(), x.clone()
    it2[1, 2] = 40
    assert torch.equal(q4.experts(x, it2, wt, *layer.dev, **layer.kw)[rest], good[rest])
    assert q4.experts(x, it2, wt, *layer.dev, **layer.kw)[1].isnan().all()
    x2[1, 100] = float("inf")
    bad = q4.experts(x2, it, wt, *layer.dev, **layer.kw)
    assert torch.equal(bad[rest], good[rest]) and not torch.isfinite(bad[1]).any()
