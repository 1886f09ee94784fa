"""An append inside a page that holds tokens on both sides (a token stored
again): where the page's scale grows, all of its other tokens keep their
values, to half a step of the new scale (and fp32's roundings of the old
value, its quotient and the new one: 4 2^-24 of 127 steps)."""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page,slot,n,dim,rot", [
    (16, 0, 1, 64, 64), (16, 3, 1, 64, 64), (16, 15, 1, 64, 0), (32, 7, 5, 48, 48), (64, 20, 30, 128, 128), (64, 33, 15, 80, 40),
    (64, 16, 16, 64, 64), (128, 1, 1, 256, 2), (128, 50, 60, 96, 96), (128, 127, 1, 64, 64)])
@pytest.mark.parametrize("gain", [30.0, 0.01])
def test_the_other_tokens_keep_their_values(page, slot, n, dim, rot, dtype, gain):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(slot)
    H = 2
    # sequence 0's second page
    pos = page + slot
    caches = [torch.randint(-127, 128, s, generator=g, dtype=torch.int8, device="cuda")
              for s in ((4, H, page, dim), (4, H, dim, page))]
    caches += [torch.rand((4, H), generator=g, device="cuda") + 0.5 for _ in range(2)]
    caches[2] /= 42
    caches[3] /= 42
    before = [x.double() for x in q4.kv_dequant(*caches)]
    held = [x.clone() for x in caches]
    k, v = (gain * torch.randn((n, H, dim), generator=g, device="cuda").to(dtype) for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    freq = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda") / max(rot, 1))) if rot else None
    q4.kv_append(k, v, *caches, i32([[3, 1]]), i32([0, n]), i32([pos + n]), inv_freq=freq)
    after = [x.double() for x in q4.kv_dequant(*caches)]
    others = [s for s in range(page) if not slot <= s < slot + n]
    for i in range(2):
        assert all(torch.equal(caches[j][p], held[j][p]) for p in (0, 2, 3) for j in range(4))
        if slot == 0:  # the page starts anew
            assert (after[i][1, :, others] == 0).all()
            continue
        step = caches[2 + i][1].double()[:, None, None]
        assert (caches[2 + i][1] > held[2 + i][1]).all() == (gain > 1)
        off = (after[i][1, :, others] - before[i][1, :, others]).abs()
        assert (off <= step * (0.5 + 127 * 4 * 2.0 ** -24)).all()
        if gain < 1:
            assert (off == 0).all()
    # values are not turned: the stored ones are v
    got = after[1][1, :, slot:slot + n].transpose(0, 1)
    assert ((got - v.double()).abs() <= caches[3][1].double()[None, :, None] * (0.5 + 127 * 4 * 2.0 ** -24)).all()
