"""Plain fp64 forms of the decode-side operators (test infrastructure only):
the cache append, attention over the cache and token log probabilities with
their gradient, one token and one head at a time, from their definitions.  No
code is shared with the HIP path.  All arrays are numpy, on the CPU.
"""
import math

import numpy as np


def spans(cu_new, lengths):
    """(first row, new tokens, position of the first) of each sequence."""
    return [(int(a), int(b) - int(a), int(n) - (int(b) - int(a)))
            for a, b, n in zip(cu_new[:-1], cu_new[1:], lengths)]


def rotate(x, pos, inv_freq, interleaved=False):
    """One head vector turned: pair i by pos * inv_freq[i]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i, f in enumerate(np.asarray(inv_freq, dtype=np.float64)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = math.cos(pos * f), math.sin(pos * f)
        y[a], y[b] = x[a] * c - x[b] * s, x[a] * s + x[b] * c
    return y


def append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, lengths,
           inv_freq=(), interleaved=False):
    """Unrounded state after an append: (k, v, k_scale, v_scale, touched).

    k and v are float64 [pages, kv_heads, page, head_dim]: the quotients that
    the codes round (a code is right if it is within half a step of them),
    codes of untouched slots as they were; touched the set of (page, slots
    now in use) pairs.  v_cache is [pages, kv_heads, head_dim, page]."""
    P, H, S, D = k_cache.shape
    kq = k_cache.astype(np.float64)
    vq = np.swapaxes(v_cache, 2, 3).astype(np.float64)
    ks, vs = k_scale.astype(np.float64), v_scale.astype(np.float64)
    touched = []
    for b, (t0, n, pos0) in enumerate(spans(cu_new, lengths)):
        i = max(0, -pos0)
        while i < n:
            pos = pos0 + i
            idx, slot = pos // S, pos % S
            m = min(S - slot, n - i)
            page = int(page_table[b][idx]) if idx < page_table.shape[1] else -1
            if 0 <= page < P:
                touched.append((page, slot + m))
                for h in range(H):
                    rows_k = np.array([rotate(k[t0 + i + e, h], pos + e, inv_freq, interleaved)
                                       for e in range(m)])
                    rows_v = v[t0 + i:t0 + i + m, h].astype(np.float64)
                    for rows, q, s in ((rows_k, kq, ks), (rows_v, vq, vs)):
                        old = 0.0 if slot == 0 else s[page, h]
                        new = max(old, np.abs(rows).max() / 127.0)
                        if new == 0.0:
                            q[page, h] = 0.0
                        else:
                            q[page, h, :slot] *= old / new
                            if slot == 0:
                                q[page, h] = 0.0
                            q[page, h, slot:slot + m] = np.clip(rows / new, -127, 127)
                        s[page, h] = new
            i += m
    return kq, vq, ks, vs, touched


def attention(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, lengths, *, scale=None,
              window=0):
    """(out, bound): the attention outputs and, per sequence and query head,
    the quantities an error bound needs: largest |score|, largest |value|,
    largest sum |k| of a key and largest |q|."""
    T, Hq, D = q.shape
    P, H, S, _ = k_cache.shape
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros((T, Hq, D))
    bound = np.zeros((T, Hq, 4))
    for b, (t0, n, pos0) in enumerate(spans(cu_new, lengths)):
        L = int(lengths[b])
        if n == 0 or L <= 0:
            continue
        ids = [int(p) for p in page_table[b][:(L + S - 1) // S]]
        for h in range(H):
            def values(cache, sc, swap):
                parts = []
                for j in range((L + S - 1) // S):
                    p = ids[j] if j < len(ids) else -1
                    if 0 <= p < P:
                        c = cache[p, h].astype(np.float64) * float(sc[p, h])
                        parts.append(c.T if swap else c)
                    else:
                        parts.append(np.full((S, D), np.nan))
                return np.concatenate(parts)[:L]
            key, val = values(k_cache, k_scale, False), values(v_cache, v_scale, True)
            for i in range(n):
                pos = pos0 + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < 0 or lo > pos:
                    continue
                kk, vv = key[lo:pos + 1], val[lo:pos + 1]
                for m in range(h * G, (h + 1) * G):
                    x = q[t0 + i, m].astype(np.float64)
                    s = kk @ x * scale
                    e = np.exp(s - s.max())
                    out[t0 + i, m] = e @ vv / e.sum()
                    bound[t0 + i, m] = (np.abs(s).max(), np.abs(vv).max(),
                                        np.abs(kk).sum(1).max(), np.abs(x).max())
    return out, bound


def logprobs(x, targets, top_k=0):
    """(logprob, entropy, lse, ids, top) of logits [M, V]."""
    x = x.astype(np.float64)
    M, V = x.shape
    lp, ent, lse = np.zeros(M), np.zeros(M), np.zeros(M)
    ids, top = np.zeros((M, top_k), np.int64), np.zeros((M, top_k))
    for m in range(M):
        row = x[m]
        best = row.max()
        if best == -np.inf:
            lse[m] = -np.inf
        else:
            lse[m] = best + math.log(np.exp(row - best).sum())
            l = (row - best) - math.log(np.exp(row - best).sum())
            ok = np.exp(l) > 0
            ent[m] = -(np.exp(l[ok]) * l[ok]).sum()
        if targets is not None:
            t = int(targets[m])
            lp[m] = 0.0 if t < 0 else (-np.inf if best == -np.inf else l[t])
        order = np.lexsort((np.arange(V), -row))[:top_k]
        ids[m] = order
        top[m] = l[order] if best > -np.inf else -np.inf
    return lp, ent, lse, ids, top


def logprobs_grad(x, targets, lse, entropy, g, h):
    """The formula, for given lse and entropy."""
    x = x.astype(np.float64)
    out = np.zeros_like(x)
    for m in range(x.shape[0]):
        if lse[m] == -np.inf:
            continue
        t = int(targets[m]) if targets is not None else -1
        gm = float(g[m]) if g is not None and t >= 0 else 0.0
        hm = float(h[m]) if h is not None else 0.0
        for v in range(x.shape[1]):
            l = x[m, v] - float(lse[m])
            p = math.exp(l)
            out[m, v] = gm * ((1.0 if v == t else 0.0) - p)
            if p > 0.0:
                out[m, v] -= hm * p * (l + float(entropy[m]))
    return out
