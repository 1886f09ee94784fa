"""Packed experts and their gradients on the GPU against the fp64 oracle; the
bounds are derived in experts_util.py."""
import math

import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import experts_oracle as oracle
from tests.experts_util import (HALF_STEP, TORCH, assert_within, expert_bounds, expert_grad_bounds, packed,
                                rounded, strided)

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, E, H, W, group, seed=0, order="low_first", spread=0.5):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.W, self.group, self.order = E, H, W, group, order
        self.gu, self.gus = packed(rng, (E,), 2 * W, H, group, spread)
        self.dn, self.dns = packed(rng, (E,), H, W, group, spread)
        high = order == "high_first"
        self.gate_up = [oracle.matrix(self.gu[e], self.gus[e], group, high) for e in range(E)]
        self.down = [oracle.matrix(self.dn[e], self.dns[e], group, high) for e in range(E)]
        self.dev = [torch.from_numpy(a).cuda() for a in (self.gu, self.gus, self.dn, self.dns)]
        self.kw = dict(group_size=group, nibble_order=order)

    def slots(self, T, k, seed, empty=0.0):
        rng = np.random.default_rng(seed)
        ids = np.array([rng.permutation(self.E)[:k] if k <= self.E else rng.integers(0, self.E, k)
                        for _ in range(T)], dtype=np.int32)
        ids[rng.random(ids.shape) < empty] = -1
        return ids, rng.random((T, k)).astype(np.float32)


def check(layer, T, k, dtype, seed=1, empty=0.0, layout="packed", ids=None):
    rng = np.random.default_rng(seed)
    x, xv = rounded(rng.normal(size=(T, layer.H)), dtype)
    d, dv = rounded(rng.normal(size=(T, layer.H)), dtype)
    own, w = layer.slots(T, k, seed, empty)
    ids = own if ids is None else ids
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    xd, dd = strided(x, layout), strided(d, layout)
    out = strided(torch.zeros_like(x), layout)
    got, pre = q4.experts(xd, it, wt, *layer.dev, **layer.kw, keep=True, out=out)
    assert got.data_ptr() == out.data_ptr() and got.dtype == TORCH[dtype]
    want = oracle.experts(xv, ids, w.astype(np.float64), layer.gate_up, layer.down)
    pre_want, epre, eout = expert_bounds(xv, ids, w, layer.gate_up, layer.down, dtype, oracle.sigmoid)
    used = ids >= 0
    assert_within(pre[torch.from_numpy(used).cuda()], pre_want[used], epre[used], "pre")
    assert_within(got, want, eout + HALF_STEP[dtype] * (np.abs(want) + eout) + 2.0 ** -25, "out")
    # the gradients at fp32 values of the gate and up
    pre32 = torch.from_numpy(pre_want).float()
    dx, dw = q4.experts_backward(dd, it, wt, pre32.cuda(), *layer.dev, **layer.kw, dx=out)
    dxw, dww = oracle.experts_grad(dv, ids, w.astype(np.float64), pre32.double().numpy(), layer.gate_up, layer.down)
    edx, edw = expert_grad_bounds(dv, ids, w, pre32.double().numpy(), layer.gate_up, layer.down, dtype, oracle.sigmoid)
    assert_within(dx, dxw, edx + HALF_STEP[dtype] * (np.abs(dxw) + edx) + 2.0 ** -25, "dx")
    assert_within(dw, dww, edw + 2.0 ** -24 * np.abs(dww), "dweights")
    if layout == "wide":
        assert out._base[:, :8].isnan().all() and out._base[:, 8 + layer.H:].isnan().all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 192])
@pytest.mark.parametrize("T", [1, 2, 9, 40, 130])
def test_parity(T, group, dtype):
    """Few rows found by the workgroups, few rows listed, and tiles of many rows."""
    check(Layer(8, 256, 136, group), T, 2, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,W,group", [(8, 8, 0), (40, 24, 32), (264, 72, 64), (520, 200, 128), (96, 1032, 32), (1096, 16, 128)])
@pytest.mark.parametrize("T,E,k", [(3, 3, 2), (33, 2, 1), (150, 5, 3)])
def test_odd_sizes(H, W, group, T, E, k, dtype):
    check(Layer(E, H, W, group, order="high_first"), T, k, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("T,E", [(2, 4), (90, 3)])
def test_deep_rows(T, E, dtype):
    """Depths of several rounds of a wave's chunks."""
    check(Layer(E, 4616, 24, 128), T, 2, dtype)
    check(Layer(E, 24, 4616, 32), T, 2, dtype)


@pytest.mark.parametrize("layout", ["wide", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 120])
def test_strides(T, dtype, layout):
    check(Layer(6, 264, 72, 32), T, 2, dtype, layout=layout)


@pytest.mark.parametrize("T", [6, 400, 1500])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_experts_and_listed_rows(T, dtype):
    check(Layer(100, 64, 32, 32), T, 4, dtype)


@pytest.mark.parametrize("T", [4, 60, 300])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_empty_slots(T, dtype):
    check(Layer(8, 128, 64, 32), T, 3, dtype, empty=0.7)
    layer = Layer(8, 128, 64, 32)
    ids = np.full((T, 3), -1, dtype=np.int32)
    check(layer, T, 3, dtype, ids=ids)
    ids[T // 2, 1] = 7
    check(layer, T, 3, dtype, ids=ids)


@pytest.mark.parametrize("T", [3, 50, 300])
def test_one_expert_takes_all_and_twice(T):
    layer = Layer(5, 128, 64, 64)
    check(layer, T, 2, "f32", ids=np.full((T, 2), 3, dtype=np.int32))
    ids = np.tile(np.array([[4, 0, 4, 4]], dtype=np.int32), (T, 1))
    check(layer, T, 4, "bf16", ids=ids)


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_ids_make_their_tokens_nan(T, dtype):
    layer = Layer(4, 64, 32, 32)
    ids, w = layer.slots(T, 2, 0)
    x = torch.randn(T, 64).to(TORCH[dtype]).cuda()
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    good, pre = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True)
    gdx, gdw = q4.experts_backward(x, it, wt, pre, *layer.dev, **layer.kw)
    for bad in (4, 1 << 30):
        it2 = it.clone()
        it2[1, 0] = bad
        out = q4.experts(x, it2, wt, *layer.dev, **layer.kw)
        dx, dw = q4.experts_backward(x, it2, wt, pre, *layer.dev, **layer.kw)
        rest = torch.arange(T) != 1
        assert out[1].isnan().all() and torch.equal(out[rest], good[rest])
        assert dx[1].isnan().all() and torch.equal(dx[rest], gdx[rest])
        assert dw[1, 0].isnan() and dw[1, 1] == gdw[1, 1] and torch.equal(dw[rest], gdw[rest])


@pytest.mark.parametrize("T", [4, 40, 400])
def test_rows_do_not_depend_on_their_neighbours(T):
    """The same tokens among others, and in another order: the same bits; infinities and NaN stay in their row."""
    layer = Layer(6, 264, 136, 64)
    ids, w = layer.slots(T, 2, 3)
    x = torch.randn(T, 264).cuda()
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    out, pre = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True)
    dx, dw = q4.experts_backward(x, it, wt, pre, *layer.dev, **layer.kw)
    order = torch.randperm(T, generator=torch.Generator().manual_seed(0)).cuda()
    again, pre2 = q4.experts(x[order], it[order], wt[order], *layer.dev, **layer.kw, keep=True)
    dx2, dw2 = q4.experts_backward(x[order], it[order], wt[order], pre2, *layer.dev, **layer.kw)
    assert torch.equal(again, out[order]) and torch.equal(pre2, pre[order])
    assert torch.equal(dx2, dx[order]) and torch.equal(dw2, dw[order])
    x[0, 5], x[2, 7] = float("inf"), float("nan")
    bad, pre3 = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True)
    dx3, dw3 = q4.experts_backward(x, it, wt, pre3, *layer.dev, **layer.kw)
    rest = torch.ones(T, dtype=torch.bool)
    rest[[0, 2]] = False
    assert not torch.isfinite(bad[0]).any() and bad[2].isnan().all() and dx3[2].isnan().all() and dw3[2].isnan().all()
    assert torch.equal(bad[rest], out[rest]) and torch.equal(dx3[rest], dx[rest]) and torch.equal(dw3[rest], dw[rest])


@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e15])
def test_magnitudes(T, size):
    """Rows of any size: gradients scale with dout, gate and up with x."""
    layer = Layer(6, 128, 64, 32)
    ids, w = layer.slots(T, 2, 3)
    d = torch.randn(T, 128).cuda()
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    two = 2.0 ** round(math.log2(size))
    x = 0.1 * d
    _, pre = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True)
    _, scaled = q4.experts(x * two, it, wt, *layer.dev, **layer.kw, keep=True)
    assert torch.equal(scaled, pre * two)
    dx, dw = q4.experts_backward(d, it, wt, pre, *layer.dev, **layer.kw)
    dx2, dw2 = q4.experts_backward(d * two, it, wt, pre, *layer.dev, **layer.kw)
    assert torch.equal(dx2, dx * two) and torch.equal(dw2, dw * two)


@pytest.mark.parametrize("T", [4, 300])
def test_outlier_channels_and_scales(T):
    """One channel 1000 times the others, scales over six orders of magnitude: bounds relative to the terms hold."""
    layer = Layer(6, 256, 128, 32, spread=7.0)
    rng = np.random.default_rng(0)
    x = rng.normal(size=(T, 256))
    x[:, 17] *= 1000
    x, xv = rounded(x, "f32")
    ids, w = layer.slots(T, 2, 3)
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    got, pre = q4.experts(x.cuda(), it, wt, *layer.dev, **layer.kw, keep=True)
    want, epre, eout = expert_bounds(xv, ids, w, layer.gate_up, layer.down, "f32", oracle.sigmoid)
    assert_within(pre, want, epre, "pre")
    assert_within(got, oracle.experts(xv, ids, w.astype(np.float64), layer.gate_up, layer.down), 1.01 * eout, "out")


def test_gradient_against_differences():
    layer = Layer(3, 32, 16, 32)
    rng = np.random.default_rng(5)
    T, k = 2, 2
    x, g = rng.normal(size=(T, 32)), rng.normal(size=(T, 32))
    ids, w = layer.slots(T, k, 7)
    x32, g32 = torch.from_numpy(x).float().cuda(), torch.from_numpy(g).float().cuda()
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    _, pre = q4.experts(x32, it, wt, *layer.dev, **layer.kw, keep=True)
    dx, dw = q4.experts_backward(g32, it, wt, pre, *layer.dev, **layer.kw)
    f = lambda xx, ww: (g * oracle.experts(xx, ids, ww, layer.gate_up, layer.down)).sum()  # noqa: E731
    x, w, h = x32.double().cpu().numpy(), w.astype(np.float64), 1e-5
    for at in np.ndindex(T, 32):
        step = np.zeros((T, 32))
        step[at] = h
        want = (f(x + step, w) - f(x - step, w)) / (2 * h)
        # values of order 10: 1e-15 * 10 / 1e-5, third derivatives 1e-10, the kernels' 1e-5 of the terms
        assert abs(dx[at].item() - want) <= 1e-4
    for at in np.ndindex(T, k):
        step = np.zeros((T, k))
        step[at] = h
        assert abs(dw[at].item() - (f(x, w + step) - f(x, w - step)) / (2 * h)) <= 1e-4


@pytest.mark.parametrize("T", [2, 30, 300])
def test_workspace_streams_and_repeats(T):
    """A caller's workspace full of NaN, another stream than the default, the same bits each time."""
    layer = Layer(8, 256, 128, 128)
    ids, w = layer.slots(T, 2, 1)
    it, wt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    x = torch.randn(T, 256).cuda()
    out, pre = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True)
    dx, dw = q4.experts_backward(x, it, wt, pre, *layer.dev, **layer.kw)
    n = max(q4.experts_workspace_bytes(T, 256, 128, 8, 2, group_size=128),
            q4.experts_backward_workspace_bytes(T, 256, 128, 8, 2, group_size=128))
    ws = torch.full((n // 4 + 4,), float("nan")).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, p2 = q4.experts(x, it, wt, *layer.dev, **layer.kw, keep=True, workspace=ws)
        dx2, dw2 = q4.experts_backward(x, it, wt, p2, *layer.dev, **layer.kw, workspace=ws)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(pre, p2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(q4.Q4Error) as e:
        q4.experts(x, it, wt, *layer.dev, **layer.kw, workspace=small)
    assert e.value.status == 3
    with pytest.raises(q4.Q4Error) as e:
        q4.experts(x, it, wt, *layer.dev, **layer.kw, out=x)
    assert e.value.status == 2


@pytest.mark.parametrize("T", [3, 64, 300])
def test_captured_graph_follows_its_inputs(T):
    layer = Layer(8, 256, 128, 32)
    x = torch.randn(T, 256).cuda()
    z = torch.randn(T, 8).cuda()
    d = torch.randn(T, 256).cuda()

    def step():
        r = q4.route(z, 2)
        out, pre = q4.experts(x, r.ids, r.weights, *layer.dev, **layer.kw, keep=True)
        dx, dw = q4.experts_backward(d, r.ids, r.weights, pre, *layer.dev, **layer.kw)
        return r.ids, out, dx, dw, q4.route_backward(z, r.ids, dw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, z, d):
            t.normal_(generator=g)
        want = [o.clone() for o in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_no_tokens():
    layer = Layer(2, 64, 32, 32)
    e = torch.empty
    out, pre = q4.experts(e(0, 64).cuda(), e(0, 2, dtype=torch.int32).cuda(), e(0, 2).cuda(), *layer.dev, **layer.kw, keep=True)
    assert out.shape == (0, 64) and pre.shape == (0, 2, 64)
    dx, dw = q4.experts_backward(out, e(0, 2, dtype=torch.int32).cuda(), e(0, 2).cuda(), pre, *layer.dev, **layer.kw)
    assert dx.shape == (0, 64) and dw.shape == (0, 2)


def test_weights_past_4_gib():
    """The last experts of arrays of more than 2^32 bytes give what they give alone."""
    E, H, W = 520, 4096, 2048
    g = torch.Generator(device="cuda").manual_seed(0)
    gu = torch.randint(0, 256, (E, 2 * W, H // 2), generator=g, dtype=torch.uint8, device="cuda")
    dn = torch.randint(0, 256, (E, H, W // 2), generator=g, dtype=torch.uint8, device="cuda")
    gus = torch.rand((E, 2 * W), generator=g, device="cuda") * 0.005
    dns = torch.rand((E, H), generator=g, device="cuda") * 0.005
    last = [t[-2:].clone() for t in (gu, gus, dn, dns)]
    for T in (2, 40):
        x = torch.randn((T, H), generator=g, device="cuda")
        w = torch.rand((T, 2), generator=g, device="cuda")
        ids = torch.tensor([[1, 0]] * T, dtype=torch.int32).cuda()
        a, pa = q4.experts(x, ids + (E - 2), w, gu, gus, dn, dns, group_size=0, keep=True)
        b, pb = q4.experts(x, ids, w, *last, group_size=0, keep=True)
        assert torch.isfinite(a).all()
        # tiles of another shape may sum in another order
        assert (a - b).abs().max() <= 1e-4 * b.abs().max() and (pa - pb).abs().max() <= 1e-4 * pb.abs().max()
        da, wa = q4.experts_backward(x, ids + (E - 2), w, pb, gu, gus, dn, dns, group_size=0)
        db, wb = q4.experts_backward(x, ids, w, pb, *last, group_size=0)
        assert (da - db).abs().max() <= 1e-4 * db.abs().max() and (wa - wb).abs().max() <= 1e-4 * wb.abs().max()
