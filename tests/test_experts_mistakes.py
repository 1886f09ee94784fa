"""Mistakes planted in the oracle are past the bounds that the GPU tests compare
with (experts_util.py), at their sizes, types and groups; the oracle rounded to
the type is within them."""
import numpy as np
import pytest
import torch

from oracle import experts_oracle as o
from tests.experts_util import (GIVEN, HALF_STEP, KEPT, TORCH, assert_within, expert_bounds, expert_grad_bounds, packed,
                                product_bound, rounded, sums)

DTYPES = ["f32", "f16", "bf16"]


class Case:
    """Five tokens over four experts of 256 x 136, two slots each."""

    def __init__(self, dtype, group):
        rng = np.random.default_rng(group)
        self.T, self.k, self.E, self.H, self.W = 5, 2, 4, 256, 136
        self.dtype, self.group = dtype, group
        self.gu, self.gus = packed(rng, (self.E,), 2 * self.W, self.H, group)
        self.dn, self.dns = packed(rng, (self.E,), self.H, self.W, group)
        self.x, self.d = (rounded(rng.normal(size=(self.T, self.H)), dtype)[1] for _ in range(2))
        self.ids = np.array([rng.permutation(self.E)[:self.k] for _ in range(self.T)])
        self.ids[1, 0] = -1
        self.w = rng.random((self.T, self.k))
        self.gate_up, self.down = self.matrices()
        self.pre, self.epre, self.eout = expert_bounds(self.x, self.ids, self.w, self.gate_up, self.down, dtype, o.sigmoid)

    def matrices(self, high=False, late=0):
        """late: groups are taken so many places further on."""
        roll = lambda s: np.roll(s, -late, 0) if late and s.ndim == 2 else s  # noqa: E731
        return ([o.matrix(c[e], roll(s[e]), self.group, high) for e in range(self.E)]
                for c, s in ((self.gu, self.gus), (self.dn, self.dns)))

    def swap(self):
        return [np.concatenate([m[self.W:], m[:self.W]]) for m in self.gate_up]


def compare(got, want, bound, dtype, last=True):
    """As the GPU tests: rounded to the type, within the bound and half a step."""
    t = torch.from_numpy(np.ascontiguousarray(got)).to(TORCH[dtype] if last else torch.float32)
    assert_within(t, want, bound + (HALF_STEP[dtype] if last else 2.0 ** -24) * (np.abs(want) + bound) + 2.0 ** -25, "")


def outputs(c, mistake):
    gu, dn, ids, w = c.gate_up, c.down, c.ids, c.w
    if mistake == "gate and up change places":
        gu = c.swap()
    elif mistake == "a weight left out":
        w = np.where(np.arange(c.k) == 1, 1.0, w)
    elif mistake == "slots' weights change places":
        w = w[:, ::-1]
    elif mistake == "wrong nibble":
        gu, _ = c.matrices(high=True)
    elif mistake == "wrong nibble of down":
        _, dn = c.matrices(high=True)
    elif mistake == "the next group's scales":
        gu, dn = c.matrices(late=1)
    elif mistake == "a slot left out":
        ids = np.where(np.arange(c.k) == 1, -1, ids)
    elif mistake == "the neighbouring expert":
        ids = np.where(ids >= 0, (ids + 1) % c.E, ids)
    elif mistake == "the last columns left out":
        x = c.x.copy()
        x[:, -8:] = 0
        return o.experts(x, ids, w, gu, dn)
    elif mistake == "one code off by one":
        gu = [m.copy() for m in gu]
        for e in range(c.E):  # a column of 256, in half of the rows
            gu[e][::2, 3] += np.abs(c.gus[e].reshape(-1, 2 * c.W)[0, ::2])
    return o.experts(c.x, ids, w, gu, dn)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("mistake", [None, "gate and up change places", "a weight left out", "slots' weights change places",
                                     "wrong nibble", "wrong nibble of down", "the next group's scales", "a slot left out",
                                     "the neighbouring expert", "the last columns left out", "one code off by one"])
def test_outputs(mistake, group, dtype):
    if mistake == "the next group's scales" and group == 0:
        pytest.skip("one group")
    c = Case(dtype, group)
    want = outputs(c, None)
    if mistake is None:
        compare(want, want, c.eout, dtype)
        return
    with pytest.raises(AssertionError):
        compare(outputs(c, mistake), want, c.eout, dtype)


def gradients(c, pre, mistake):
    """(dx, dweights) from their definition, with one step of it wrong."""
    dx, dw = np.zeros(c.d.shape), np.zeros(c.w.shape)
    for t in range(c.T):
        for j, e in enumerate(c.ids[t]):
            if e < 0:
                continue
            g, u = pre[t, j, :c.W], pre[t, j, c.W:]
            s = o.sigmoid(g)
            r = c.d[t] @ c.down[e]
            dw[t, j] = np.dot(g * s * u, r) * (c.w[t, j] if mistake == "the weight in its own gradient" else 1)
            if mistake == "up left out of dweights":
                dw[t, j] = np.dot(g * s, r)
            dh = r * (1 if mistake == "the weight left out of dx" else c.w[t, j])
            slope = s if mistake == "1 - sigmoid left out" else s * (1 + g * (1 - s))
            parts = [dh * u * slope, dh * g * s]
            if mistake == "dg and du change places":
                parts = parts[::-1]
            dx[t] += np.concatenate(parts) @ c.gate_up[e]
    if mistake == "one slot's dx":
        last = c.w.copy()
        last[:, 1] = 0
        dx = o.experts_grad(c.d, c.ids, last, pre, c.gate_up, c.down)[0]
    return dx, dw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("mistake", [None, "1 - sigmoid left out", "the weight left out of dx", "the weight in its own gradient",
                                     "up left out of dweights", "dg and du change places", "one slot's dx"])
def test_gradients(mistake, group, dtype):
    c = Case(dtype, group)
    pre = c.pre.astype(np.float32).astype(np.float64)
    want, dww = o.experts_grad(c.d, c.ids, c.w, pre, c.gate_up, c.down)
    edx, edw = expert_grad_bounds(c.d, c.ids, c.w, pre, c.gate_up, c.down, dtype, o.sigmoid)
    dx, dw = gradients(c, pre, mistake)
    of_weights = mistake in ("the weight in its own gradient", "up left out of dweights")
    for wrong, args in ((mistake is not None and not of_weights, (dx, want, edx, dtype)),
                        (of_weights, (dw, dww, edw, dtype, False))):
        if wrong:
            with pytest.raises(AssertionError):
                compare(*args)
        else:
            compare(*args)


def head(x, w, targets, g, mistake):
    """(loss, lse, dx) with one step wrong."""
    t = targets.copy()
    if mistake == "the next target":
        t = np.where(t >= 0, (t + 1) % w.shape[0], t)
    if mistake == "a column left out":  # of every row's likelier ones
        odd = int(np.argsort(np.where(np.isin(np.arange(len(w)), t), -np.inf, (x @ w.T).min(0)))[-1])
        w, t = np.delete(w, odd, 0), t - (t > odd)
    loss, lse = o.cross_entropy(x, w, t)
    if mistake == "an empty row's loss":
        loss[1] = lse[1]
    dx = o.cross_entropy_grad(x, w, t, g)
    z = x @ w.T
    p = np.exp(z - lse[:, None])
    if mistake == "the onehot left out":
        dx = np.where((t < 0)[:, None], 0, (p * g[:, None]) @ w)
    if mistake == "g of the mean":
        dx = o.cross_entropy_grad(x, w, t, g / len(t))
    if mistake == "an empty row's gradient":
        dx[1] = (p[1] * g[1]) @ w
    return loss, lse, dx


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("mistake,of", [(None, ""), ("the next target", "loss dx"), ("a column left out", "lse loss dx"),
                                        ("an empty row's loss", "loss"), ("the onehot left out", "dx"), ("g of the mean", "dx"),
                                        ("an empty row's gradient", "dx")])
def test_head(mistake, of, group, dtype):
    """One of the sizes of test_head_loss_gpu.py, with its bounds."""
    M, V, K = 3, 129, 72
    rng = np.random.default_rng(1)
    codes, scales = packed(rng, (), V, K, group)
    w = o.matrix(codes, (2.5 * scales).astype(np.float32), group)
    x = rounded(rng.normal(size=(M, K)), dtype)[1]
    targets, g = np.array([V - 2, -1, 17]), rng.normal(size=M)
    loss, lse, dx = head(x, w, targets, g, None)
    ez = product_bound(x, 0 * x, w, GIVEN[dtype])
    elz = ez.max(1)
    elp = elz + 2.0 ** -20 * (1 + np.abs(lse))
    z = x @ w.T
    p, hot = np.exp(z - lse[:, None]), np.arange(V)[None] == targets[:, None]
    ed = np.abs(g)[:, None] * (p * (ez + elz[:, None] + 2.0 ** -20 * (1 + np.abs(z)) + 2.0 ** -23 * np.abs(lse)[:, None])
                               + 2.0 ** -23 * hot + 2.0 ** -39)
    d = np.abs((p - hot) * g[:, None])
    ed[targets < 0] = d[targets < 0] = 0
    bound = ed @ np.abs(w) + (KEPT[dtype] + 2.0 ** -24 + sums(V)) * (d @ np.abs(w))
    got = dict(zip(("loss", "lse", "dx"), head(x, w, targets, g, mistake)))
    for name, args in (("loss", (loss, elp + elz + 2.0 ** -20 * (1 + np.abs(lse)), dtype, False)), ("lse", (lse, elp, dtype, False)),
                       ("dx", (dx, bound, dtype))):
        if name in of.split():
            with pytest.raises(AssertionError):
                compare(got[name], *args)
        else:
            compare(got[name], *args)
