"""Inputs and error bounds of the expert and head-loss tests.

Bounds, for a product z = sum_k x_k w_k with S = sum |x_k w_k|:
  * fp32 activations are held to 22 bits: 2^-22 S; values of a 16-bit type are
    held exactly; values computed on the way (the gated product, gradients
    times scales) are rounded to fp32 (2^-24) and then to 22 bits, or 11 for
    16-bit types: 2^-11 S;
  * the sums: a matrix instruction adds 16 or 32 products and its start value,
    one rounding of at most 2^-23 S each (it may truncate); K / 16 of them, a
    product and an addition of 2^-24 per group of 32, at most 17 joins of
    waves, splits or pieces and 3 last steps:
        sums(K) = (K / 16 + K / 16 + 20) 2^-23.
"""
import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {k: torch.finfo(t).eps / 2 for k, t in TORCH.items()}
KEPT = {"f32": 2.0 ** -22, "f16": 2.0 ** -11, "bf16": 2.0 ** -11}  # of values computed on the way
GIVEN = {"f32": 2.0 ** -22, "f16": 0.0, "bf16": 0.0}               # of inputs


def sums(K):
    return (K / 8 + 20) * 2.0 ** -23


def rounded(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype])
    return t, t.double().numpy()


def packed(rng, lead, rows, depth, group, spread=0.5):
    codes = rng.integers(0, 256, (*lead, rows, depth // 2)).astype(np.uint8)
    shape = (*lead, rows) if group == 0 else (*lead, -(-depth // group), rows)
    scales = (np.exp(rng.uniform(-spread, spread, shape)) / (4.6 * depth ** 0.5)).astype(np.float32)
    return codes, scales


def strided(t, kind):
    """A 2-D tensor on the GPU in one of several layouts."""
    t = t.cuda()
    if kind == "packed":
        return t.contiguous()
    if kind == "wide":  # rows of a wider array, poisoned around it
        buf = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device="cuda")
        buf[:, 8:8 + t.shape[1]] = t
        return buf[:, 8:8 + t.shape[1]]
    if kind == "odd":  # element alignment only
        buf = torch.full((t.shape[0] * (t.shape[1] + 1) + 1,), float("nan"), dtype=t.dtype, device="cuda")
        view = buf[1:].view(t.shape[0], t.shape[1] + 1)[:, :t.shape[1]]
        view.copy_(t)
        return view
    raise ValueError(kind)


def product_bound(x, ex, w, kept):
    """Error bound of x @ w.T whose rows x carry errors ex."""
    a = np.abs(w).T
    return ex @ a + (kept + sums(w.shape[1])) * (np.abs(x) @ a)


def expert_bounds(x, ids, weights, gate_up, down, dtype, sigmoid):
    """(pre, its bound, out's bound before the last rounding)."""
    T, k = ids.shape
    W = gate_up[0].shape[0] // 2
    pre, epre = np.zeros((T, k, 2 * W)), np.zeros((T, k, 2 * W))
    eout = np.zeros(x.shape)
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            row = x[t:t + 1]
            z = row @ gate_up[e].T
            ez = product_bound(row, 0 * row, gate_up[e], GIVEN[dtype])
            pre[t, j], epre[t, j] = z[0], ez[0]
            g, u, eg, eu = z[:, :W], z[:, W:], ez[:, :W], ez[:, W:]
            silu = g * sigmoid(g)
            h = silu * u
            # |silu'| <= 1.1; exponential, division and products: 16 roundings at most
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 2.0 ** -20 * np.abs(h)
            y = h @ down[e].T
            ey = product_bound(h, eh, down[e], KEPT[dtype])
            eout[t] += abs(weights[t, j]) * (ey[0] + (k + 1) * 2.0 ** -24 * np.abs(y[0]))
    return pre, epre, eout


def expert_grad_bounds(dout, ids, weights, pre, gate_up, down, dtype, sigmoid):
    """Bounds of dx (before its last rounding) and dweights."""
    T, k = ids.shape
    W = pre.shape[2] // 2
    edx, edw = np.zeros(dout.shape), np.zeros(weights.shape)
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            g, u = pre[t, j, :W], pre[t, j, W:]
            s = sigmoid(g)
            z = dout[t:t + 1] @ down[e]
            # two parts whatever the type, of a product rounded to fp32
            ez = product_bound(dout[t:t + 1], 0 * dout[t:t + 1], down[e].T, 2.0 ** -22 + 2.0 ** -24)
            h = np.abs(g * s * u)
            edw[t, j] = h @ ez[0] + (sums(W) + 2.0 ** -20) * (h @ np.abs(z[0]))
            w = abs(weights[t, j])
            fg, fu = np.abs(u * s * (1 + g * (1 - s))), np.abs(g * s)
            # 1 + g sigmoid(-g) may cancel: its rounding is relative to its terms
            loose = np.abs(u * s) * (1 + np.abs(g) * (1 - s))
            d = np.concatenate([z[0] * fg, z[0] * fu]) * w
            ed = w * np.concatenate([ez[0] * fg + 2.0 ** -20 * np.abs(z[0]) * loose,
                                     ez[0] * fu + 2.0 ** -20 * np.abs(z[0]) * fu])
            row = product_bound(d[None], ed[None], gate_up[e].T, KEPT[dtype] + 2.0 ** -24)
            edx[t] += row[0] + k * 2.0 ** -24 * (np.abs(d) @ np.abs(gate_up[e]))
    return edx, edw


def assert_within(got, want, bound, what):
    got = got.detach().cpu().double().numpy()
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all(), f"{what}: NaN in other places"
    over = np.abs(got - want)[~nan] - bound[~nan]
    worst = over.max() if over.size else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} past its bound (at {np.argmax(over)})"
