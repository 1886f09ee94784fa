"""The head's loss and gradient over a vocabulary past 2^24, against fp64 on the
device."""
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.experts_util import HALF_STEP, KEPT, TORCH, sums

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,dtype", [(1, "f32"), (3, "bf16")])
def test_vocabularies_past_2_24(M, dtype):
    V, K = (1 << 24) + 777, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    qw = torch.randint(0, 256, (V, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand(V, generator=gen, device="cuda") * 0.05 + 0.01
    x = torch.randn(M, K, generator=gen, device="cuda").to(TORCH[dtype])
    t = torch.tensor([V - 1, 5, (1 << 24) + 2][:M], device="cuda")
    g = torch.randn(M, generator=gen, device="cuda")
    r = q4.head_cross_entropy(x, qw, scales, t, group_size=0)
    dx = q4.head_cross_entropy_backward(x, qw, scales, t, r.lse, g, group_size=0)
    w = torch.stack([(qw & 15).double(), (qw >> 4).double()], 2).view(V, K) - 8
    w *= scales[:, None].double()
    z = x.double() @ w.t()
    lse = torch.logsumexp(z, 1)
    # logits below 8: 2^-22 and sums(8) of them; exponentials and sums 2^-20 (1 + lse) as in test_head_loss_gpu.py
    e = 8 * K * (2.0 ** -22 + sums(K)) + 2.0 ** -20 * (1 + lse)
    assert ((r.lse.double() - lse).abs() <= e).all()
    assert ((r.loss.double() - (lse - z.gather(1, t[:, None])[:, 0])).abs() <= 2 * e).all()
    p = torch.exp(z - lse[:, None])
    p.scatter_add_(1, t[:, None], torch.full_like(p[:, :1], -1.0))
    d = p * g[:, None].double()
    want, terms = d @ w, d.abs() @ w.abs()
    # a probability's error is 2 e of it; the chain of V / 16 additions of 2^-23 each adds up like a walk, sqrt(2^20)
    # 2^-23 = 2^-13 of the terms, eight times that
    bound = (2 * e[:, None] + KEPT[dtype] + 2.0 ** -10) * terms + HALF_STEP[dtype] * want.abs()
    assert ((dx.double() - want).abs() <= bound).all()
