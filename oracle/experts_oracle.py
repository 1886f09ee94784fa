"""Plain fp64 forms of routing, packed experts and the packed head's cross
entropy, with their gradients (test infrastructure only), one token at a time
from their definitions.  No code is shared with the HIP path.  All arrays are
numpy, on the CPU."""
import math

import numpy as np


def matrix(codes, scales, group, high_first=False):
    """[rows, depth] that packed codes [rows, depth / 2] and scales ([groups,
    rows], or [rows] with group 0) stand for."""
    rows, depth = codes.shape[0], 2 * codes.shape[1]
    w = np.zeros((rows, depth))
    for k in range(depth):
        byte = codes[:, k // 2].astype(np.int64)
        upper = (k % 2 == 1) != high_first
        code = (byte >> 4 if upper else byte & 15) - 8
        s = scales if group == 0 else scales[k // group]
        w[:, k] = code * s.astype(np.float64)
    return w


def scores(z, kind):
    """Scores of one row of logits."""
    z = np.asarray(z, dtype=np.float64)
    if kind == "sigmoid":
        return np.array([1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in z])
    top = max(z)
    e = np.array([0.0 if v == -math.inf else math.exp(v - top) for v in z])
    return e / e.sum()


def route(z, top_k, kind="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(ids, weights) of one row; -1 and 0 where no expert is eligible."""
    z = np.asarray(z, dtype=np.float64)
    E = len(z)
    s = scores(z, kind) if np.any(z > -math.inf) else np.zeros(E)
    value = z if bias is None else s + np.asarray(bias, dtype=np.float64)
    open_ = [e for e in range(E) if z[e] > -math.inf and value[e] > -math.inf]
    if groups > 1:
        per = E // groups
        lead = {}
        for e in open_:
            lead.setdefault(e // per, []).append(value[e])
        lead = {g: sum(sorted(v, reverse=True)[:1 if bias is None else 2]) for g, v in lead.items()}
        kept = sorted(lead, key=lambda g: (-lead[g], g))[:top_groups]
        open_ = [e for e in open_ if e // per in kept]
    ids = sorted(open_, key=lambda e: (-value[e], e))[:top_k]
    if renormalize and kind == "softmax" and ids:  # the divisor falls away
        w = scores(z[ids], "softmax")
    else:
        w = s[ids]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
    missing = top_k - len(ids)
    return np.array(ids + [-1] * missing), np.concatenate([w * scale, np.zeros(missing)])


def route_grad(z, ids, g, kind="softmax", renormalize=True, scale=1.0):
    """d/dz of sum(g * weights) of one row, the choice held fixed."""
    z = np.asarray(z, dtype=np.float64)
    dz = np.zeros(len(z))
    if not np.any(z > -math.inf):
        return dz
    s = scores(z, kind)
    on = [j for j, e in enumerate(ids) if e >= 0]
    ds = np.zeros(len(z))
    total = sum(s[ids[j]] for j in on)
    mean = sum(g[j] * s[ids[j]] for j in on) / total if total else 0.0
    for j in on:
        ds[ids[j]] += scale * ((g[j] - mean) / total if renormalize else g[j]) if total else 0.0
    if kind == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - np.dot(ds, s))


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def expert_rows(x, gate_up):
    """gate and up of rows x."""
    z = x @ gate_up.T
    w = gate_up.shape[0] // 2
    return z[:, :w], z[:, w:]


def experts(x, ids, weights, gate_up, down):
    """out [T, hidden] with fp64 matrices gate_up[e], down[e]."""
    out = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            g, u = expert_rows(x[t:t + 1], gate_up[e])
            out[t] += weights[t, j] * ((g * sigmoid(g) * u) @ down[e].T)[0]
    return out


def experts_grad(dout, ids, weights, pre, gate_up, down):
    """(dx, dweights) given gate and up before the product, pre [T, k, 2 w]."""
    dx, dw = np.zeros(dout.shape), np.zeros(weights.shape)
    w = pre.shape[2] // 2
    for t in range(dout.shape[0]):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            g, u = pre[t, j, :w], pre[t, j, w:]
            s = sigmoid(g)
            dh = dout[t] @ down[e]
            dw[t, j] = np.dot(g * s * u, dh)
            dh = dh * weights[t, j]
            dx[t] += np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s]) @ gate_up[e]
    return dx, dw


def cross_entropy(x, w, targets):
    """(loss, lse) of logits x w^T."""
    z = x @ w.T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    loss = np.array([0.0 if t < 0 else math.nan if t >= w.shape[0] else lse[m] - z[m, t]
                     for m, t in enumerate(targets)])
    return loss, lse


def cross_entropy_grad(x, w, targets, g):
    z = x @ w.T
    p = np.exp(z - z.max(1)[:, None])
    p /= p.sum(1)[:, None]
    for m, t in enumerate(targets):
        if t < 0:
            p[m] = 0
        elif t < w.shape[0]:
            p[m, t] -= 1
        else:
            p[m] = math.nan
    return (p * g[:, None]) @ w
