"""Attention where a row's elements, or a tile's weights, lie far apart.

Queries with an outlier channel, whose keys are small in that channel: the
scores are ordinary, and so every other channel of the query has to keep its
bits.  A first token that takes most of the weight and has next to no value (a
"sink"): the outputs are made of the other tokens' weights, which have to keep
theirs.

The bounds come from the outputs' type and from fp32 arithmetic alone, whatever
form the kernel holds its operands in.  S: largest |score|, V: largest |value|,
A = sum_j p_j |v_j| of an output element.
  * fp32 throughout: a score is a sum of dim products, each rounded by 2^-24,
    in any order: (dim + 16) 2^-24 scale sum |q k|; the subtraction of the
    maximum and the exponential 4 2^-24 (S + 1); the weights and their sum 2 e
    of A, e the two together, and the sums over keys (keys / 64 + 96) 2^-24 A;
  * 16-bit outputs may lose, beside their own rounding, half as much as that
    rounding is at the row's largest output.
"""
import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu
from tests.serve_util import TORCH, Batch, rounded

pytestmark = pytest.mark.gpu


def cache_of(b, key, value, dim):
    """key, value: codes [kv_heads, length, dim] of sequence 0; the other
    sequences' pages hold zeros.  Scales 1 / 64."""
    H, L, S = key.shape[0], key.shape[1], b.page
    k = np.zeros((b.pages, H, S, dim), np.int8)
    v = np.zeros((b.pages, H, dim, S), np.int8)
    for j in range(-(-L // S)):
        n = min(S, L - j * S)
        k[b.table[0, j], :, :n] = key[:, j * S:j * S + n]
        v[b.table[0, j], :, :, :n] = np.swapaxes(value[:, j * S:j * S + n], 1, 2)
    s = np.full((b.pages, H), 1 / 64, np.float32)
    return [torch.from_numpy(x).cuda() for x in (k, v, s, s)]


def check(q, key, value, new, length, page, dtype, fill=()):
    """Sequence 0: q [new, heads, dim] over its `length` tokens; `fill` more of
    one token each, to choose the kernel."""
    need_gpu()
    heads, dim, H = q.shape[1], q.shape[2], key.shape[0]
    b = Batch([new, *fill], [length, *fill], page, 0)
    qt, qx = rounded(np.concatenate([q, np.zeros((len(fill), heads, dim))]), dtype)
    print(f"[attention] new={new} of {length} heads={heads}/{H} dim={dim} page={page} {dtype} fill={len(fill)}", flush=True)
    got = q4.attention(qt.cuda(), *cache_of(b, key, value, dim), *b.device(), max_new=new, max_len=length)
    got = got[:new].double().cpu().numpy()
    k, v = (np.repeat(x.astype(np.float64) / 64, heads // H, 0) for x in (key, value))
    worst = 0.0
    for i in range(new):
        n = length - new + i + 1
        for h in range(heads):
            terms = k[h, :n] * qx[i, h] * dim ** -0.5
            s = terms.sum(1)
            p = np.exp(s - s.max())
            p /= p.sum()
            out, size = p @ v[h, :n], p @ np.abs(v[h, :n])
            e = 2.0 ** -24 * ((dim + 16) * np.abs(terms).sum(1).max() + 4 * (np.abs(s).max() + 1))
            half = torch.finfo(TORCH[dtype]).eps / 2
            tol = size * (2 * e + (n / 64 + 96) * 2.0 ** -24) + half * np.abs(out)
            if dtype != "f32":
                tol = tol + half / 2 * np.abs(out).max()
            worst = max(worst, float((np.abs(got[i, h] - out) / tol).max()))
    print(f"            worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0


FILL = (1,) * 75  # makes the rows many enough for the kernel that shares keys
SHAPES = [(1, 700, 64, ()), (2, 700, 16, ()), (40, 700, 64, FILL), (40, 700, 32, FILL)]


@pytest.mark.parametrize("dtype,gain", [("f16", 1), ("f16", 20), ("f16", 200), ("bf16", 200), ("bf16", 1000),
                                        ("f32", 1), ("f32", 200), ("f32", 2000)])
@pytest.mark.parametrize("new,length,page,fill", SHAPES)
def test_queries_with_an_outlier_channel(new, length, page, fill, dtype, gain):
    dim, heads, H = 128, 4, 2
    g = np.random.default_rng(gain)
    q = g.normal(0, 1.5, (new, heads, dim))
    q[:, :, 5] *= gain
    key = np.clip(np.rint(g.normal(0, 40, (H, length, dim))), -127, 127)
    key[:, :, 5] = np.rint(key[:, :, 5] / gain)
    value = np.clip(np.rint(g.normal(0, 40, (H, length, dim))), -127, 127)
    check(q, key.astype(np.int8), value.astype(np.int8), new, length, page, dtype, fill)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
@pytest.mark.parametrize("new,length,page,fill", SHAPES + [(1, 60, 64, ()), (30, 100, 64, FILL), (1, 5000, 16, ())])
def test_a_token_that_takes_most_of_the_weight_and_has_no_value(new, length, page, fill, share, dtype):
    dim, heads, H = 64, 4, 2
    g = np.random.default_rng(int(100 * share))
    # channel 0 of the queries is 8, and only the first token has a key there
    q = g.normal(0, 1.0, (new, heads, dim))
    q[:, :, 0] = 8.0
    key = np.clip(np.rint(g.normal(0, 40, (H, length, dim))), -127, 127)
    key[:, :, 0] = 0
    key[:, 0] = 0
    # the others' weights sum to about exp(0.2) a token
    score = np.log(share / (1 - share) * length * 1.2)
    key[:, 0, 0] = min(127, np.rint(score * 64 * dim ** 0.5 / 8.0))
    if key[0, 0, 0] == 127:
        q[:, :, 0] *= score * 64 * dim ** 0.5 / 8.0 / 127
    value = np.clip(np.rint(g.normal(0, 40, (H, length, dim))), -127, 127)
    value[:, 0] = 0
    check(q, key.astype(np.int8), value.astype(np.int8), new, length, page, dtype, fill)
