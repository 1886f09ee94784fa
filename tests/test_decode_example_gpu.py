"""The example decoder at a small size: every operator is checked on the
tensors that the path gave it, as they were used together.

Bounds: the cache's codes and the attention's outputs as in
test_kv_append_gpu.py and test_attention_gpu.py; log probabilities as in
test_logprobs_gpu.py at this vocabulary (1e-5 covers them); the head's input
gradient is the binary16 path of linear_backward, 2e-3 of sum |dlogits w|.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from oracle import serve_oracle as orc
from tests.gpu_util import need_gpu
from tests.test_attention_gpu import tolerance
from tests.test_kv_append_gpu import SCALE_TOL, SLACK

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode.py")


def example():
    spec = importlib.util.spec_from_file_location("decode_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def check_layer(t, inv_freq):
    c = lambda x: x.detach().cpu().numpy()  # noqa: E731
    before, after = [c(x) for x in t["before"]], [c(x) for x in t["after"]]
    table, cu, ln = c(t["table"]), c(t["cu"]), c(t["lengths"])
    f = c(inv_freq)
    rk, rv, rks, rvs, touched = orc.append(c(t["k"]), c(t["v"]), *before, table, cu, ln, f)
    for p, used in touched:
        assert np.allclose(after[2][p], rks[p], rtol=SCALE_TOL) and np.allclose(after[3][p], rvs[p], rtol=SCALE_TOL)
        assert np.abs(after[0][p, :, :used] - rk[p, :, :used]).max() <= 0.5 + SLACK
        assert np.abs(np.swapaxes(after[1], 2, 3)[p, :, :used] - rv[p, :, :used]).max() <= 0.5 + SLACK
    q_in, q = c(t["q_in"]).astype(np.float64), c(t["q"])
    for t0, n, pos0 in orc.spans(cu, ln):
        for i in range(n):
            for h in range(q.shape[1]):
                want = orc.rotate(q_in[t0 + i, h], pos0 + i, f)
                assert np.abs(q[t0 + i, h] - want).max() <= 8 * 2.0 ** -24 * np.abs(want).max() + 2.0 ** -23 * np.abs(q_in).max()
    ref, bound = orc.attention(q, *after, table, cu, ln)
    ratio = after[3][after[3] > 0]
    tol = tolerance(ref, bound, "f32", q.shape[2] ** -0.5, int(ln.max()), after[0].shape[2],
                    float(np.log(ratio.max() / ratio.min())) / 2)
    assert (np.abs(c(t["out"]) - ref) <= tol).all()


def test_the_example_decodes_scores_and_differentiates():
    need_gpu()
    ex = example()
    shape = ex.Shape(hidden=128, layers=2, heads=6, kv_heads=2, head_dim=32, ffn=256, vocab=1003, group=32, page=16)
    model = ex.Decoder(shape, pages=30, batch=3, max_pages=6)
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, shape.vocab, (n,), generator=gen).cuda() for n in (5, 40, 16)]
    new = [len(p) for p in prompts]
    trace = []
    hidden = model.step(torch.cat(prompts), new, trace)
    for _ in range(3):
        logits = model.logits(hidden[ex.last_of(new, "cuda")])
        r = q4.token_logprobs(logits, top_k=3)
        want = torch.log_softmax(logits.double(), 1)
        assert torch.equal(r.top_ids[:, 0], logits.argmax(1))
        assert (r.top_logprobs.double() - want.topk(3, 1).values).abs().max() < 1e-5
        new = [1, 1, 1]
        hidden = model.step(r.top_ids[:, 0], new, trace)
    assert len(trace) == 8
    for t in trace:
        check_layer(t, model.inv_freq)

    hidden = torch.randn((37, shape.hidden), device="cuda")
    targets = torch.randint(0, shape.vocab, (37,), generator=gen).cuda()
    r, dx = ex.score(model, hidden, targets)
    w = q4.dequant(model.head.qw, model.head.scales, shape.hidden, 0).double().cpu().numpy()
    x = model.logits(hidden).double().cpu().numpy()
    lp, ent, lse, _, _ = orc.logprobs(x, targets.cpu().numpy())
    assert np.abs(r.logprob.cpu().numpy() - lp).max() < 1e-5 and np.abs(r.entropy.cpu().numpy() - ent).max() < 1e-5
    g = np.full(37, 1.0 / 37)
    d = orc.logprobs_grad(x, targets.cpu().numpy(), lse, ent, g, 0.01 * g)
    assert (np.abs(dx.cpu().numpy() - d @ w) <= 2e-3 * (np.abs(d) @ np.abs(w))).all()


def test_generate_runs_and_repeats():
    need_gpu()
    ex = example()
    shape = ex.Shape(hidden=128, layers=2, heads=6, kv_heads=2, head_dim=32, ffn=256, vocab=1003, group=32, page=16)
    runs = []
    for _ in range(2):
        model = ex.Decoder(shape, pages=30, batch=2, max_pages=6)
        gen = torch.Generator().manual_seed(3)
        prompts = [torch.randint(0, shape.vocab, (n,), generator=gen).cuda() for n in (9, 21)]
        runs.append(ex.generate(model, prompts, 12))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    assert runs[0][0].shape == (2, 12) and (runs[0][1] <= 0).all()
