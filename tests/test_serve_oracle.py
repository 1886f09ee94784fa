"""What pins the fp64 oracle of the decode-side operators: hand-made values,
dense torch in fp64, and gradients by differences; and that planted mistakes in
it are seen by the same comparisons."""
import math

import numpy as np
import torch

from oracle import serve_oracle as orc
from tests.serve_util import Batch, random_cache


def test_rotation_by_hand():
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0, 6.0])
    f = [0.5, 0.25]
    y = orc.rotate(x, 2, f)
    assert np.allclose(y[[0, 2]], [math.cos(1) - 3 * math.sin(1), math.sin(1) + 3 * math.cos(1)])
    assert np.allclose(y[[1, 3]], [2 * math.cos(.5) - 4 * math.sin(.5), 2 * math.sin(.5) + 4 * math.cos(.5)])
    assert np.array_equal(y[4:], x[4:])
    z = orc.rotate(x, 2, f, interleaved=True)
    assert np.allclose(z[:2], [math.cos(1) - 2 * math.sin(1), math.sin(1) + 2 * math.cos(1)])
    assert np.allclose(np.linalg.norm(y), np.linalg.norm(x)) and np.allclose(np.linalg.norm(z), np.linalg.norm(x))
    # the product of two turned vectors depends on the distance alone
    a, b = np.random.default_rng(0).normal(size=(2, 6))
    d = [orc.rotate(a, p + 3, f) @ orc.rotate(b, p, f) for p in (0, 5, 1000)]
    assert np.allclose(d, d[0])


def test_append_by_hand():
    k = np.zeros((3, 1, 16))
    k[0], k[1], k[2] = 127.0, 254.0, -63.5
    cache = [np.zeros((2, 1, 16, 16), np.int8), np.zeros((2, 1, 16, 16), np.int8),
             np.zeros((2, 1), np.float32), np.zeros((2, 1), np.float32)]
    kq, vq, ks, vs, touched = orc.append(k, -k, *cache, np.array([[1, 0]]), [0, 3], [17])
    # positions 14, 15 in page 1 (not fresh, scale 0 before), 16 in page 0
    assert touched == [(1, 16), (0, 1)]
    assert ks[1, 0] == 2.0 and ks[0, 0] == 0.5 and np.array_equal(ks, vs)
    assert (kq[1, 0, 14] == 63.5).all() and (kq[1, 0, 15] == 127).all() and (kq[0, 0, 0] == -127).all()
    assert np.array_equal(vq, -kq)
    # growth: codes already there shrink
    cache[0][1, 0, :2] = 100
    cache[2][1] = 1.0
    kq, _, ks, _, _ = orc.append(k[1:2], k[1:2], *cache, np.array([[1, 0]]), [0, 1], [3])
    assert ks[1, 0] == 2.0 and (kq[1, 0, :2] == 50).all() and (kq[1, 0, 2] == 127).all()


def dense(q, k, v, ks, vs, table, cu, lens, window=0):
    T, Hq, D = q.shape
    H = k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0:
            continue
        ids = torch.from_numpy(table[b, :-(-L // k.shape[2])].astype(np.int64))
        kk = (torch.from_numpy(k)[ids].double() * torch.from_numpy(ks)[ids][..., None, None].double())
        vv = (torch.from_numpy(v)[ids].double() * torch.from_numpy(vs)[ids][..., None, None].double()).transpose(2, 3)
        kk, vv = (x.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :L] for x in (kk, vv))
        kk, vv = (x.repeat_interleave(Hq // H, 0) for x in (kk, vv))
        qq = torch.from_numpy(q[cu[b]:cu[b + 1]]).double().transpose(0, 1)
        i, j = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
        mask = (j <= i) & ((j > i - window) if window else torch.ones_like(j <= i))
        s = (qq @ kk.transpose(1, 2) / math.sqrt(D)).masked_fill(~mask, -math.inf)
        out[cu[b]:cu[b + 1]] = (torch.softmax(s, -1) @ vv).transpose(0, 1)
    return out.numpy()


def test_attention_against_dense_torch():
    for window in (0, 9):
        b = Batch([1, 4, 30], [37, 20, 30], 16, 2)
        k, v, ks, vs = random_cache(b, 2, 32, 3)
        q = np.random.default_rng(1).normal(size=(b.T, 6, 32))
        out, bound = orc.attention(q, k, v, ks, vs, b.table, b.cu, b.len, window=window)
        want = dense(q, k, v, ks, vs, b.table, b.cu, b.len, window)
        assert np.abs(out - want).max() < 1e-12
        assert (np.abs(out) <= bound[..., 1:2] + 1e-12).all()
        # planted: a page out of place, a scale of another head, a mask one off
        t = b.table.copy()
        t[0, [1, 2]] = t[0, [2, 1]]
        assert np.abs(orc.attention(q, k, v, ks, vs, t, b.cu, b.len, window=5)[0][0] -
                      dense(q, k, v, ks, vs, b.table, b.cu, b.len, 5)[0]).max() > 1e-3
        assert np.abs(orc.attention(q, k, v, ks, vs[:, ::-1], b.table, b.cu, b.len, window=window)[0] - want).max() > 1e-3
        assert np.abs(orc.attention(q, k, v, ks, vs, b.table, b.cu, b.len, window=8)[0] - want).max() > 1e-3


def test_attention_without_keys_and_with_bad_pages():
    b = Batch([2, 1], [1, 20], 16, 0)
    k, v, ks, vs = random_cache(b, 1, 16, 0)
    q = np.random.default_rng(0).normal(size=(3, 2, 16))
    out, _ = orc.attention(q, k, v, ks, vs, b.table, b.cu, b.len)
    assert (out[0] == 0).all() and np.isfinite(out).all()
    t = b.table.copy()
    t[1, 1] = 99
    out, _ = orc.attention(q, k, v, ks, vs, t, b.cu, b.len)
    assert np.isnan(out[2]).all() and np.isfinite(out[:2]).all()


def test_logprobs_against_torch():
    x = np.random.default_rng(0).normal(0, 3, (4, 50))
    x[1, 5:] = -np.inf
    t = np.array([3, 2, 49, -1])
    lp, ent, lse, ids, top = orc.logprobs(x, t, 3)
    z = torch.log_softmax(torch.from_numpy(x), 1)
    assert np.allclose(lp[:3], z[range(3), t[:3]]) and lp[3] == 0
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(x), 1))
    assert np.allclose(ent, torch.distributions.Categorical(logits=torch.from_numpy(x).clamp(min=-1e300)).entropy())
    want = torch.topk(z, 3, 1)
    assert np.array_equal(ids, want.indices.numpy()) and np.allclose(top, want.values)
    ids = orc.logprobs(np.array([[1.0, 2, 2, 0, 2]]), None, 4)[3]
    assert ids.tolist() == [[1, 2, 4, 0]]
    lp, ent, lse, _, top = orc.logprobs(np.full((1, 4), -np.inf), np.array([1]), 2)
    assert lp[0] == lse[0] == -np.inf and ent[0] == 0 and (top == -np.inf).all()


def test_gradient_against_differences_and_autograd():
    g0 = np.random.default_rng(2)
    x = g0.normal(0, 2, (3, 12))
    t, g, h = np.array([4, -1, 0]), g0.normal(size=3), g0.normal(size=3)
    lp, ent, lse, _, _ = orc.logprobs(x, t)
    d = orc.logprobs_grad(x, t, lse, ent, g, h)

    def loss(z):
        a, b, _, _, _ = orc.logprobs(z, t)
        return (g * np.where(t >= 0, a, 0) + h * b).sum()
    for m in range(3):
        for v in range(12):
            z = x.copy()
            z[m, v] += 1e-6
            y = x.copy()
            y[m, v] -= 1e-6
            assert abs((loss(z) - loss(y)) / 2e-6 - d[m, v]) < 1e-7
    # planted: a missing entropy term, a sign
    assert np.abs(orc.logprobs_grad(x, t, lse, 0 * ent, g, h) - d).max() > 1e-2
    assert np.abs(orc.logprobs_grad(x, t, lse, ent, -g, h) - d).max() > 1e-2
