"""Calls whose work would fill a launch of 2^32 threads and more: nothing is
left out."""
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,H,page", [(4200, 8, 16), (6000, 4, 16), (1300, 8, 16)])
def test_an_append_of_many_sequences_without_a_bound(B, H, page):
    """max_new defaults to T: B pages of workgroups for each sequence."""
    need_gpu()
    D = 16
    k, q = torch.randn((B, H, D), device="cuda"), torch.randn((B, H, D), device="cuda")
    table = torch.randperm(B, device="cuda").to(torch.int32)[:, None]
    args = table, i32(range(B + 1)), torch.randint(1, page + 1, (B,), dtype=torch.int32, device="cuda")
    caches = [q4.new_cache(B, H, D, page) for _ in range(2)]
    want = q4.kv_append(k, -k, *caches[0], *args, q=q, max_new=1)
    got = q4.kv_append(k, -k, *caches[1], *args, q=q)
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(*caches))


def test_an_append_of_a_long_prompt_among_many_sequences():
    """Pages of one sequence past what a launch has workgroups for."""
    need_gpu()
    B, H, D, page, long = 3000, 8, 16, 16, 3000
    new = [1] * B
    new[7], new[2999] = long, 40
    T = sum(new)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new).cumsum(0)
    cols = -(-(long + 9) // page)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    ids, at = torch.randperm(B + 2 * cols), 0
    lengths = [n + 9 for n in new]
    for b, n in enumerate(lengths):
        m = -(-n // page)
        table[b, :m] = ids[at:at + m].int()
        at += m
    k = torch.randn((T, H, D), device="cuda")
    caches = q4.new_cache(B + 2 * cols, H, D, page)
    q4.kv_append(k, -k, *caches, table.cuda(), cu.cuda(), i32(lengths))
    dk, dv = q4.kv_dequant(*caches)
    for b in (0, 7, 8, 1500, 2999):
        t = torch.arange(lengths[b])
        at = table[b].cuda().long()[t.cuda() // page], slice(None), t.cuda() % page
        want = k[cu[b]:cu[b + 1]]
        step = caches[2][at[0][9:]][:, :, None]
        for got, w in ((dk[at][9:], want), (dv[at][9:], -want)):
            assert ((got - w).abs() <= 0.51 * step).all()
        assert (dk[at][:9] == 0).all()


def test_values_of_a_cache_of_very_many_pages():
    need_gpu()
    H, D, page = 8, 16, 16
    P = (1 << 24) // H + 1000
    g = torch.Generator(device="cuda").manual_seed(0)
    caches = [torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device="cuda")
              for s in ((P, H, page, D), (P, H, D, page))]
    caches += [torch.rand((P, H), generator=g, device="cuda") for _ in range(2)]
    got = q4.kv_dequant(*caches, dtype=torch.bfloat16)
    for part in (slice(0, 50), slice(P // 2, P // 2 + 50), slice(P - 1100, P)):
        want = q4.kv_dequant(*[c[part].contiguous() for c in caches], dtype=torch.bfloat16)
        assert all(torch.equal(a[part], b) for a, b in zip(got, want))


def test_log_probabilities_of_very_many_rows():
    need_gpu()
    M = (1 << 24) + 1003
    x = torch.randn((M, 5), device="cuda")
    t = torch.randint(0, 5, (M,), device="cuda")
    r = q4.token_logprobs(x, t, top_k=2)
    g, h = torch.randn(M, device="cuda"), torch.randn(M, device="cuda")
    d = q4.token_logprobs_backward(x, t, r.lse, r.entropy, g, h)
    for part in (slice(0, 100), slice((1 << 23) - 50, (1 << 23) + 50), slice(M - 1100, M)):
        want = q4.token_logprobs(x[part], t[part], top_k=2)
        assert torch.equal(r.top_ids[part], want.top_ids)
        assert torch.allclose(r.lse[part], want.lse, rtol=1e-5, atol=1e-6)
        assert torch.allclose(r.logprob[part], want.logprob, rtol=1e-5, atol=1e-6)
        assert torch.equal(d[part], q4.token_logprobs_backward(x[part], t[part], r.lse[part], r.entropy[part], g[part], h[part]))
