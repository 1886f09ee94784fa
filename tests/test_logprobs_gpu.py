"""Token log probabilities and their gradient against the fp64 oracle.

Bounds, from the kernel's arithmetic, with y = x - m and E = sum p |y|:
  * e^y: 2^-23 (its unit's rounding) + |y| 2^-23 (the difference and the
    change of base), relative; sums of n terms in a row: n 2^-24, relative,
    n = vocab / 256 + 64 (a thread's, then the joins');
  * lse: (n + 16) 2^-24 + 2^-23 (1 + E) + 2^-22 |lse|, and a log
    probability, |x - m| 2^-24 more;
  * entropy = log S - W / S: the same for log S; W's terms are off by their
    relative errors: E ((n + 16) 2^-24) + 2^-22 (E + sum p y^2 + H).
"""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import serve_oracle as orc
from tests.gpu_util import need_gpu
from tests.serve_util import TORCH

pytestmark = pytest.mark.gpu


def logits_of(M, V, dtype, seed, pad=0, gain=3.0):
    g = np.random.default_rng(seed)
    t = torch.from_numpy(g.normal(0, gain, (M, V))).to(TORCH[dtype])
    buf = torch.full((M, V + pad), float("nan"), dtype=TORCH[dtype], device="cuda")
    buf[:, :V] = t.cuda()
    return buf[:, :V], t.double().numpy(), torch.from_numpy(g.integers(0, V, M))


def check(x, xd, targets, k, top_lp_slack=0.0):
    M, V = x.shape
    r = q4.token_logprobs(xd, targets.cuda(), top_k=k)
    torch.cuda.synchronize()
    lp, ent, lse, ids, top = orc.logprobs(x, targets.numpy(), k)
    with np.errstate(invalid="ignore"):
        m = x.max(1, keepdims=True)
        y = x - m
        p = np.exp(x - lse[:, None])
        E = np.where(p > 0, p * np.abs(y), 0).sum(1)
        Q = np.where(p > 0, p * y * y, 0).sum(1)
    n = V / 256 + 64
    t_lse = (n + 16) * 2.0 ** -24 + 2.0 ** -23 * (1 + E) + 2.0 ** -22 * np.abs(lse)
    t_ent = t_lse + E * (n + 16) * 2.0 ** -24 + 2.0 ** -22 * (E + Q + ent)
    err = lambda a, b: np.abs(a.double().cpu().numpy() - b)  # noqa: E731
    assert (err(r.lse, lse) <= t_lse).all()
    assert (err(r.entropy, ent) <= t_ent).all()
    assert (err(r.logprob, lp) <= t_lse + 2.0 ** -23 * np.abs(lp)).all()
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    assert (err(r.top_logprobs, top) <= t_lse[:, None] + 2.0 ** -23 * np.abs(top)).all()
    return r


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 63, 64, 255, 1000, 1025, 4097, 8192, 20011])
def test_vocabularies(V, dtype):
    need_gpu()
    for pad, k in ((0, 0), (3, 1), (1, 5)):
        xd, x, t = logits_of(5, V, dtype, V + pad, pad)
        print(f"[logprobs] V={V} {dtype} pad={pad} k={k}", flush=True)
        check(x, xd, t, min(k, V))


@pytest.mark.parametrize("M,V", [(1, 128257), (4, 128257), (40, 32003), (300, 3001), (1100, 500)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_and_parts(M, V, dtype):
    need_gpu()
    xd, x, t = logits_of(M, V, dtype, M)
    check(x, xd, t, 20)


@pytest.mark.parametrize("M,V", [(300, 32767), (300, 32768), (280, 40003), (1030, 33000)])
@pytest.mark.parametrize("dtype,k", [("f32", 0), ("f32", 32), ("bf16", 7)])
def test_long_rows_without_parts(M, V, dtype, k):
    need_gpu()
    xd, x, t = logits_of(M, V, dtype, M)
    check(x, xd, t, k)


@pytest.mark.parametrize("k", [1, 2, 3, 19, 31, 32])
def test_ties_go_to_the_lowest_index(k):
    need_gpu()
    g = np.random.default_rng(k)
    for V in (40, 3000, 20000):
        x = torch.from_numpy(g.integers(0, 6, (6, V))).float()
        x[0] = 1.25          # nothing but ties
        x[1, ::2] = -0.0     # equal to 0
        x[1, 1::2] = 0.0
        check(x.double().numpy(), x.cuda(), torch.zeros(6, dtype=torch.int64), k)


@pytest.mark.parametrize("order", ["ascending", "descending"])
def test_sorted_logits(order):
    need_gpu()
    x = torch.linspace(-8, 8, 12345)[None].repeat(2, 1)
    x = x.flip(1) if order == "descending" else x
    check(x.double().numpy(), x.cuda().contiguous(), torch.tensor([0, 12344]), 32)


def test_masked_logits():
    need_gpu()
    x = torch.randn((8, 5000)) * 3
    x[0, 1:] = -float("inf")               # one token left
    x[1] = -float("inf")                   # none
    x[2] = torch.finfo(torch.float32).min  # all at the type's lowest value
    x[3, 7:] = torch.finfo(torch.float32).min
    x[4, ::3] = -float("inf")
    x[5, :4990] = -float("inf")
    x[6] += 1e4
    t = torch.tensor([0, 3, 5, 2, 3, 10, 8, -1])
    r = q4.token_logprobs(x.cuda(), t.cuda(), top_k=20)
    lp, ent, lse, ids, top = orc.logprobs(x.double().numpy(), t.numpy(), 20)
    tol = dict(rtol=2e-6, atol=2e-5)
    assert np.allclose(r.lse.cpu(), lse, **tol) and np.allclose(r.entropy.cpu(), ent, **tol)
    got = r.logprob.cpu().numpy()
    ok = [0, 1, 2, 3, 4, 5, 7]
    assert np.allclose(got[ok], lp[ok], **tol)
    assert abs(got[6] - lp[6]) < 2e-3  # logits of 1e4 have steps of 2^-10
    assert got[4] == -np.inf and got[5] == -np.inf and got[1] == -np.inf and got[7] == 0
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    assert r.entropy[1] == 0 and r.lse[1] == -float("inf") and (r.top_logprobs[1] == -float("inf")).all()


def test_rows_that_are_not_finite_and_targets_out_of_range():
    need_gpu()
    x = torch.randn((6, 3000))
    x[0, 17] = float("nan")
    x[1, 2900] = float("inf")
    x[2] = float("nan")
    t = torch.tensor([1, 1, 1, 3000, -5, 4])
    clean = q4.token_logprobs(x[3:].cuda(), t[3:].cuda(), top_k=4)
    r = q4.token_logprobs(x.cuda(), t.cuda(), top_k=4)
    for row in range(3):
        assert r.lse[row].isnan() and r.entropy[row].isnan() and r.logprob[row].isnan()
        assert r.top_logprobs[row].isnan().all()
    want = torch.topk(torch.nan_to_num(x[0], -9e9), 4).indices
    assert torch.equal(r.top_ids[0].cpu(), want) and r.top_ids[1, 0] == 2900 and (r.top_ids[2] == -1).all()
    assert torch.equal(r.lse[3:], clean.lse) and torch.equal(r.top_ids[3:], clean.top_ids)
    assert r.logprob[3].isnan() and r.logprob[4] == 0 and r.logprob[5].isfinite()
    assert q4.token_logprobs(x.cuda()).logprob is None


def grad_case(M, V, dtype, seed, pad=0):
    xd, x, t = logits_of(M, V, dtype, seed, pad)
    g = np.random.default_rng(seed + 9)
    _, ent, lse, _, _ = orc.logprobs(x, t.numpy())
    f = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32))  # noqa: E731
    return xd, x, t, f(lse), f(ent), f(g.normal(0, 1, M)), f(g.normal(0, 0.3, M))


def grad_tolerance(x, lse, ent, g, h, want, dtype):
    l = x - lse.numpy()[:, None].astype(np.float64)
    p = np.exp(l)
    g, h, ent = (np.abs(np.zeros(len(x)) if a is None else a.numpy().astype(np.float64))[:, None] for a in (g, h, ent))
    l = np.where(p > 0, np.abs(l), 0)
    return p * 2.0 ** -22 * (2 + l) * (g + h * (l + ent)) + 2.0 ** -24 * g + \
        torch.finfo(TORCH[dtype]).eps / 2 * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 3, 8, 65, 1000, 5003])
def test_gradient(V, dtype):
    need_gpu()
    for pad, terms in ((0, "gh"), (1, "g"), (5, "h")):
        xd, x, t, lse, ent, g, h = grad_case(4, V, dtype, V, pad)
        t[1] = -1
        g, h = g if "g" in terms else None, h if "h" in terms else None
        c = lambda a: None if a is None else a.cuda()  # noqa: E731
        got = q4.token_logprobs_backward(xd, t.cuda(), lse.cuda(), ent.cuda(), c(g), c(h))
        want = orc.logprobs_grad(x, t.numpy(), lse.numpy(), ent.numpy(), None if g is None else g.numpy(),
                                 None if h is None else h.numpy())
        err = np.abs(got.double().cpu().numpy() - want)
        gg = None if g is None else torch.where(t >= 0, g, 0)
        assert (err <= grad_tolerance(x, lse, ent, gg, h, want, dtype)).all(), (pad, terms)


def test_gradient_in_place_and_into_a_padded_buffer():
    need_gpu()
    xd, x, t, lse, ent, g, h = grad_case(3, 1001, "f32", 0, 7)
    args = [a.cuda() for a in (t, lse, ent, g, h)]
    want = q4.token_logprobs_backward(xd, *args)
    buf = torch.full((3, 1010), 5.0, device="cuda")
    q4.token_logprobs_backward(xd, *args, dlogits=buf[:, 3:1004])
    assert torch.equal(buf[:, 3:1004], want) and (buf[:, :3] == 5).all() and (buf[:, 1004:] == 5).all()
    q4.token_logprobs_backward(xd, *args, dlogits=xd)
    assert torch.equal(xd, want)


def test_gradient_against_differences():
    """sum(g logprob) + sum(h entropy) from the kernel's own forward, along
    random directions: a central difference of fp32 results, step e = 0.05,
    is off by e^2 / 6 of the third derivative (of order 1 here, at most the
    direction's cube) and by the forward's rounding over e."""
    need_gpu()
    xd, x, t, _, _, g, h = grad_case(6, 257, "f32", 4)
    c = [a.cuda() for a in (t, g, h)]
    f = q4.token_logprobs(xd, c[0])
    grad = q4.token_logprobs_backward(xd, c[0], f.lse, f.entropy, c[1], c[2])

    def value(z):
        r = q4.token_logprobs(z, c[0])
        return (c[1] * r.logprob + c[2] * r.entropy).double()
    for seed in range(4):
        d = torch.randn(xd.shape, generator=torch.Generator().manual_seed(seed)).cuda()
        e = 0.05
        slope = (value(xd + e * d) - value(xd - e * d)) / (2 * e)
        want = (grad.double() * d.double()).sum(1)
        assert ((slope - want).abs() <= 0.02 * (1 + c[1].abs() + c[2].abs())).all()


def test_gradient_of_masked_rows():
    need_gpu()
    x = torch.randn((6, 2000)) * 3
    x[0, 1:] = -float("inf")
    x[1] = -float("inf")
    x[2, 5:] = torch.finfo(torch.float32).min
    x[3, 0] = float("nan")
    t = torch.tensor([0, 3, 2, 1, 2000, -1])
    r = q4.token_logprobs(x.cuda(), t.cuda())
    g, h = torch.full((6,), 2.0).cuda(), torch.full((6,), 3.0).cuda()
    got = q4.token_logprobs_backward(x.cuda(), t.cuda(), r.lse, r.entropy, g, h).cpu()
    assert (got[1] == 0).all() and got[[0, 2, 5]].isfinite().all()
    assert (got[0, 1:] == 0).all() and abs(got[0, 0]) < 1e-5 and (got[2, 5:] == 0).all()
    assert got[3].isnan().all() and got[4].isnan().all()
    assert abs(got[5].double().sum()) < 1e-4


def test_logprobs_replay_in_a_graph():
    need_gpu()
    x = torch.randn((3, 50000), device="cuda")
    t = torch.tensor([5, 6, 7], device="cuda")
    q4.token_logprobs(x, t, top_k=8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = q4.token_logprobs(x, t, top_k=8)
        d = q4.token_logprobs_backward(x, t, r.lse, r.entropy, r.entropy)
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        e = q4.token_logprobs(x, t, top_k=8)
        ed = q4.token_logprobs_backward(x, t, e.lse, e.entropy, e.entropy)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, e)) and torch.equal(d, ed)


@pytest.mark.parametrize("V", [5000, 40003, 128257])
@pytest.mark.parametrize("M", [1, 300])
def test_rows_that_one_logit_fills(M, V):
    """Log probability and entropy next to 0, to a part of themselves.

    The other terms sum to r = S - 1, about 10^-5 here.  ln S = log1p(r): the
    largest logit's thread adds 1 to its step's sum in at most 5 additions that
    round by 2^-24 each (the later ones keep what they round off), and each term
    2^y errs by |y| 2^-23 + 2^-22 of itself with y to 2^5."""
    need_gpu()
    if M * V > 20_000_000:
        V = 66_000
    g = np.random.default_rng(V)
    t = torch.from_numpy(g.normal(0, 0.5, (M, V))).float()
    where = torch.from_numpy(g.integers(0, V, M))
    t[torch.arange(M), where] = float(np.log(V) + 11.5)
    x = t.double()
    big = x.max(1, keepdim=True).values
    e = torch.exp(x - big)
    e[torch.arange(M), where] = 0.0
    rest = e.sum(1)
    lp = -torch.log1p(rest)
    ent = -lp - (e * (x - big)).sum(1) / (1 + rest)
    r = q4.token_logprobs(t.cuda(), where.cuda(), top_k=1)
    tol = 5 * 2.0 ** -24 + 2.0 ** -17 * rest
    assert ((r.logprob.double().cpu() - lp).abs() <= tol).all()
    assert ((r.top_logprobs[:, 0].double().cpu() - lp).abs() <= tol).all()
    assert ((r.entropy.double().cpu() - ent).abs() <= 5 * 2.0 ** -24 + 2.0 ** -17 * 40 * rest).all()
