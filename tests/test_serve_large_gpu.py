"""The decode-side operators where offsets pass 32 bits, and replayed in
graphs: results are bit for bit those of small arrays and of eager calls."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu
from tests.serve_util import Batch, random_cache

pytestmark = pytest.mark.gpu


def test_pages_past_four_gigabytes():
    need_gpu()
    H, D, S = 8, 128, 64
    P = (1 << 32) // (H * D * S) + 5000  # 4.6 GB each for keys and values
    b = Batch([1, 3, 70], [300, 130, 200], S, 0, spare_pages=0)
    small = [torch.from_numpy(x).cuda() for x in random_cache(b, H, D, 1)]
    big = [torch.zeros((P, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    place = P - 1 - 7 * torch.arange(b.pages)  # far pages, spread
    for s, g in zip(small, big):
        g[place.cuda()] = s
    table, cu, ln = b.device()
    far = torch.where((table >= 0) & (table < b.pages), place.to(torch.int32).cuda()[table.clamp(0, b.pages - 1).long()], -1)
    q, k, v = (torch.randn((b.T, h, D), device="cuda") for h in (32, H, H))
    f = (10000.0 ** (-torch.arange(0, D, 2) / D)).cuda()
    outs = []
    for caches, t in ((small, table), (big, far.to(torch.int32))):
        qo = q4.kv_append(k, v, *caches, t, cu, ln, q=q, inv_freq=f)
        outs.append((qo, q4.attention(qo, *caches, t, cu, ln, max_new=70, max_len=300)))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for s, g in zip(small, big):
        assert torch.equal(s, g[place.cuda()])
    assert int(big[0].count_nonzero()) == int(small[0].count_nonzero())  # nothing else was written


def test_logits_past_two_to_the_31():
    need_gpu()
    V = 128257
    M = (1 << 31) // V + 40
    x = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    x[-3:] = (3 * torch.randn((3, V), device="cuda")).bfloat16()
    t = torch.arange(M, device="cuda") % V
    whole = q4.token_logprobs(x, t, top_k=4)
    part = q4.token_logprobs(x[-3:], t[-3:], top_k=4)
    assert torch.equal(whole.top_ids[-3:], part.top_ids)
    assert torch.allclose(whole.lse[-3:], part.lse, rtol=1e-6) and torch.allclose(whole.logprob[-3:], part.logprob, rtol=1e-5)
    assert torch.equal(whole.top_ids[0], torch.arange(4, device="cuda"))
    g = torch.ones(M, device="cuda")
    want = q4.token_logprobs_backward(x[-3:], t[-3:], whole.lse[-3:], whole.entropy[-3:], g[-3:])
    got = q4.token_logprobs_backward(x, t, whole.lse, whole.entropy, g, dlogits=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(x[-3:], want)
    assert abs(float(x[0, 0]) - (1 - 1 / V)) < 0.01 and abs(float(x[1, 0]) + 1 / V) < 1e-7


def test_a_decode_loop_replays():
    """append + attention captured once; each replay takes the next token."""
    need_gpu()
    H, G, D, S, B = 2, 3, 64, 16, 3
    caches = [q4.new_cache(20, H, D, S) for _ in range(2)]  # replayed, eager
    table = torch.randperm(20, generator=torch.Generator().manual_seed(0))[:18].view(B, 6).to(torch.int32).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ln = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = torch.zeros((B, G * H + 2 * H, D), device="cuda")
    f = (10000.0 ** (-torch.arange(0, D, 2) / D)).cuda()
    out = torch.empty((B, G * H, D), device="cuda")
    need = q4.attention_workspace_bytes(B, B, G * H, H, D, page=S, max_new=1, max_len=96)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step(cache, rows, out=None):
        q, k, v = rows.split([G * H, H, H], 1)
        qo = q4.kv_append(k, v, *cache, table, cu, ln, q=q, inv_freq=f, max_new=1)
        return q4.attention(qo, *cache, table, cu, ln, max_new=1, max_len=96, out=out, workspace=ws if out is not None else None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(caches[0], rows, out)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for c in caches[0]:
        c.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], rows, out)
    for c in caches[0]:
        c.zero_()
    for i in range(40):
        ln.add_(torch.tensor([1, 2 if i else 1, 1], dtype=torch.int32, device="cuda") if i < 20 else 1)
        rows.copy_(torch.randn(rows.shape, generator=torch.Generator().manual_seed(i)))
        want = step(caches[1], rows)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0)), i
    assert all(torch.equal(a, b) for a, b in zip(*caches))


def test_operators_on_a_stream_of_their_own():
    need_gpu()
    b = Batch([2, 1], [100, 40], 16, 0)
    caches = [torch.from_numpy(x).cuda() for x in random_cache(b, 2, 64, 1)]
    copy = [c.clone() for c in caches]
    k = torch.randn((3, 2, 64), device="cuda")
    x = torch.randn((2, 70000), device="cuda")
    args = b.device()
    q4.kv_append(k, k, *caches, *args)
    want = q4.token_logprobs(x, top_k=3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q4.kv_append(k, k, *copy, *args)
        got = q4.token_logprobs(x, top_k=3)
        d = q4.kv_dequant(*copy)
    s.synchronize()
    assert all(torch.equal(a.nan_to_num(3.0) if a.is_floating_point() else a, c.nan_to_num(3.0) if c.is_floating_point() else c)
               for a, c in zip(caches, copy))
    assert torch.equal(got.lse, want.lse) and torch.equal(got.top_ids, want.top_ids) and d[0].shape[0] == b.pages
