"""The example decoder with experts in its feed-forward parts and the loss
without logits: that it runs, and its gradients."""
import numpy as np
import pytest
import torch

from oracle import experts_oracle as oracle
from tests.gpu_util import need_gpu
from tests.test_decode_example_gpu import example

pytestmark = pytest.mark.gpu
SHAPE = dict(hidden=128, layers=2, heads=6, kv_heads=2, head_dim=32, vocab=1003, group=32, page=16, experts=6, top_k=2,
             expert_ffn=72)


def test_it_decodes_and_its_losses_agree():
    need_gpu()
    ex = example()
    shape = ex.Shape(**SHAPE)
    model = ex.Decoder(shape, pages=12, batch=2, max_pages=6)
    gen = torch.Generator().manual_seed(0)
    prompts = [torch.randint(0, shape.vocab, (n,), generator=gen).cuda() for n in (9, 33)]
    ids, logprobs, _ = ex.generate(model, prompts, 5)
    assert ids.shape == (2, 5) and torch.isfinite(logprobs).all()
    one = ex.Decoder(shape, pages=6, batch=1, max_pages=6)
    hidden = one.step(prompts[1][:-1], [32])
    r, dx = ex.score(one, hidden, prompts[1][1:], entropy_weight=0.0)
    mean, dh = ex.loss(one, hidden, prompts[1][1:])
    # the layer's binary16 products of 128 terms against two parts: 2^-11 of logits below 10, and 2e-3
    # of the gradient's terms as in the other example's test
    assert abs(mean + r.logprob.mean()) <= 1e-2
    assert (dh + dx).abs().max() <= 1e-2 * dh.abs().max()


def test_gradient_of_router_and_experts():
    need_gpu()
    ex = example()
    layer = ex.Experts(6, 2, 64, 40, 32, torch.Generator().manual_seed(3), "cuda")
    x, g = torch.randn(5, 64).cuda(), torch.randn(5, 64).cuda()
    trace = {}
    layer(x, trace)
    got = layer.backward(g, trace["logits"], trace["ids"], trace["weights"], trace["pre"])
    qw, sc = [m.cpu().numpy() for m in layer.mats[0::2]], [m.cpu().numpy() for m in layer.mats[1::2]]
    up, down = ([oracle.matrix(q, s, 32) for q, s in zip(qw[i], sc[i])] for i in (0, 1))
    R, ids = layer.router.double().cpu().numpy(), trace["ids"].cpu().numpy()

    def f(v):
        z = v @ R
        w = np.exp(np.take_along_axis(z, ids.astype(np.int64), 1))
        return (g.double().cpu().numpy() * oracle.experts(v, ids, w / w.sum(1, keepdims=True), up, down)).sum()

    at, h = x.double().cpu().numpy(), 1e-5
    for i in ((0, 0), (1, 17), (4, 63)):
        step = np.zeros(at.shape)
        step[i] = h
        # differences of values of order 100: 1e-14 * 100 / 1e-5; fp32 products of 64 and 80 terms
        assert abs(got[i].item() - (f(at + step) - f(at - step)) / (2 * h)) <= 1e-3
