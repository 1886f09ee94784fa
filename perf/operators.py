"""Measured cases of the decode-side operators: appending to a paged 8-bit
key/value cache, attention over that cache, and token log probabilities with
their gradient.

``run`` computes each operator in its plain form (elementary torch operations
in fp32, angles in fp64) while ``own`` is false, and through the package's
entry points while it is true.  ``exact`` gives the same outputs in fp64 from
the operators' definitions.

The cache (one layer): pages of ``page`` tokens.
  k_cache  int8 [pages, kv_heads, page, head_dim]
  v_cache  int8 [pages, kv_heads, head_dim, page]   (tokens innermost)
  k_scale, v_scale  float32 [pages, kv_heads]: one scale per page and head;
  an element stands for code * scale.
Sequence b owns the pages page_table[b, 0], page_table[b, 1], ...; its
``lengths[b]`` tokens include the cu_new[b + 1] - cu_new[b] new ones of this
call, which are its last.  A second append of the same tokens writes the same
slots again, so every pass does the work of a step.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CODE_MAX = 127.0


def listed():
    return [
        # one decode step of 32 short and long conversations, Llama-3.2-1B head shapes: latency counts
        dict(name="append_decode_1b", op="append", dtype="f32", batch=32, new_lo=1, new_hi=1, len_lo=1, len_hi=4096,
             heads=32, kv_heads=8, head_dim=64, page=16, rot=64, interleaved=False, spread=1),
        # prompts of a prefill batch entering the cache, Llama-3.1-8B head shapes
        dict(name="append_prefill_8b", op="append", dtype="f32", batch=6, new_lo=600, new_hi=2048, len_lo=0, len_hi=0,
             heads=32, kv_heads=8, head_dim=128, page=64, rot=128, interleaved=False, spread=2),
        # chunks of any size joining far-advanced contexts: odd head counts, a partial interleaved rotation, bf16
        dict(name="append_chunks_far", op="append", dtype="bf16", batch=9, new_lo=1, new_hi=301, len_lo=1000, len_hi=1000000,
             heads=14, kv_heads=2, head_dim=80, page=32, rot=40, interleaved=True, spread=3),
        # a single conversation's decode step over a short context: the smallest call
        dict(name="attn_decode_one", op="attention", dtype="f32", batch=1, new_lo=1, new_hi=1, len_lo=257, len_hi=257,
             heads=32, kv_heads=8, head_dim=64, page=16, window=0, spread=4),
        # a serving batch of decode steps over ragged contexts
        dict(name="attn_decode_batch", op="attention", dtype="f32", batch=64, new_lo=1, new_hi=1, len_lo=500, len_hi=8000,
             heads=32, kv_heads=8, head_dim=128, page=64, window=0, spread=5),
        # two very long contexts: few rows, a long axis to split
        dict(name="attn_decode_long", op="attention", dtype="bf16", batch=2, new_lo=1, new_hi=1, len_lo=131072, len_hi=200003,
             heads=32, kv_heads=8, head_dim=128, page=64, window=0, spread=6),
        # a few drafted tokens checked at once, under a sliding window, with a padded head size
        dict(name="attn_verify_window", op="attention", dtype="f16", batch=16, new_lo=2, new_hi=6, len_lo=100, len_hi=3001,
             heads=24, kv_heads=8, head_dim=96, page=32, window=1024, spread=7),
        # chunked prefill: many rows, each over its own part of a long context
        dict(name="attn_prefill_chunk", op="attention", dtype="bf16", batch=3, new_lo=300, new_hi=2048, len_lo=2048, len_hi=8192,
             heads=32, kv_heads=8, head_dim=128, page=64, window=0, spread=8),
        # the output head's logits of a small decode batch, with the alternatives a user asks to see
        dict(name="logprobs_decode", op="logprobs", dtype="f32", rows=4, vocab=128257, top_k=20),
        # scoring a prompt: the head's logits of 512 positions
        dict(name="logprobs_score", op="logprobs", dtype="f32", rows=512, vocab=128257, top_k=5),
        # the head's gradient in a policy update: log probability and entropy terms together
        dict(name="logprobs_grad_head", op="logprobs_grad", dtype="f32", rows=512, vocab=128257),
        # a small odd vocabulary in 16 bits
        dict(name="logprobs_grad_odd", op="logprobs_grad", dtype="bf16", rows=65, vocab=32003),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "logprobs", "logprobs_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("logprobs", "logprobs_grad"):
        vocab = _log_int(rng, 1000, 160000)
        rows = _log_int(rng, 1, max(2, min(4096, 60_000_000 // vocab)))
        c = dict(op=op, dtype=dtype, rows=rows, vocab=vocab)
        if op == "logprobs":
            c["top_k"] = rng.choice([0, 1, 5, 20, 32])
        return c
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    head_dim = rng.choice([64, 80, 96, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    c = dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, spread=rng.randrange(1000))
    if op == "append":
        new = _log_int(rng, 1, 2000)
        batch = _log_int(rng, 1, max(2, min(200, 8000 // new)))
        c.update(batch=batch, new_lo=max(1, new // 3), new_hi=new, len_lo=0, len_hi=rng.choice([0, 5000, 1000000]),
                 rot=rng.choice([head_dim, head_dim, head_dim // 2]), interleaved=rng.random() < 0.3)
        return c
    kind = rng.choice(["decode", "decode", "few", "chunk"])
    if kind == "chunk":
        new, high = _log_int(rng, 16, 1500), _log_int(rng, 1500, 8000)
        batch = rng.randint(1, 2)
    else:
        new = 1 if kind == "decode" else rng.randint(2, 12)
        high = _log_int(rng, 20, 60000)
        batch = _log_int(rng, 1, max(2, min(128, 250_000 // high)))
    c.update(batch=batch, new_lo=max(1, new // 2), new_hi=new, len_lo=max(new, high // 5), len_hi=high,
             window=rng.choice([0, 0, 0, max(8, high // 3)]))
    return c


def _spans(case):
    """New tokens and lengths (new ones included) of each sequence, by the case alone."""
    rng = random.Random(case["spread"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    if case["op"] == "append":  # the lengths before the call, spread over their logarithm
        lo, hi = max(1, case["len_lo"]), case["len_hi"]
        return new, [n + (_log_int(rng, lo, hi) if hi else 0) for n in new]
    return new, [max(n, _log_int(rng, case["len_lo"], case["len_hi"])) for n in new]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    if case["op"] in ("logprobs", "logprobs_grad"):
        M, V = case["rows"], case["vocab"]
        # a trained head's logits: a broad bulk and a few likely tokens per row
        logits = randn(M, V) * 2.5
        likely = torch.randint(0, V, (M, 8), generator=g, device=dev)
        logits.scatter_add_(1, likely, 8.0 + 3.0 * randn(M, 8))
        state = dict(op=case["op"], logits=logits.to(dt), targets=likely[:, 0].contiguous(), top_k=case.get("top_k", 0))
        if case["op"] == "logprobs_grad":  # what the forward pass left and the loss's gradients
            x = state["logits"].double()
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            state.update(lse=lse.float(), entropy=(lse - (p * x).sum(1)).float(), g_logprob=randn(M), g_entropy=0.01 * randn(M))
        return state
    new, lengths = _spans(case)
    B, Hq, Hk, D, PS = case["batch"], case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    T = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    append = case["op"] == "append"
    # an append touches the pages from the first new token's on: only those are kept here, however far the context reaches
    first = [(L - n) // PS if append else 0 for n, L in zip(new, lengths)]
    last = [(L + PS - 1) // PS for L in lengths]
    pages = sum(b - a for a, b in zip(first, last))
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(last)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, first[b]:last[b]] = perm[at:at + last[b] - first[b]]
        at += last[b] - first[b]
    codes = lambda *s: (randn(*s) * 42.0).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
    k_cache, v_cache = codes(pages, Hk, PS, D), codes(pages, Hk, D, PS)
    scale = lambda: (0.7 + 0.7 * torch.rand((pages, Hk), generator=g, device=dev)) / 42.0  # noqa: E731
    state = dict(op=case["op"], k_cache=k_cache, v_cache=v_cache, k_scale=scale(), v_scale=scale(), page_table=table,
                 cu_new=torch.tensor(cu, dtype=torch.int32, device=dev), lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
                 max_new=max(new), max_len=max(lengths), q=(randn(T, Hq, D) * (1.0 if append else 1.5)).to(dt))
    if append:
        # keys and values as a fused projection leaves them: one row per token
        rows = randn(T, 2 * Hk, D).to(dt)
        state.update(k=rows[:, :Hk], v=rows[:, Hk:], interleaved=case["interleaved"],
                     inv_freq=(500000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])).float())
        # slots that hold no token yet are 0
        used = torch.zeros(pages, dtype=torch.int64, device=dev)
        for b in range(B):
            used[table[b, first[b]].long()] = (lengths[b] - new[b]) % PS
        empty = torch.arange(PS, device=dev)[None, :] >= used[:, None]
        k_cache.masked_fill_(empty[:, None, :, None], 0)
        v_cache.masked_fill_(empty[:, None, None, :], 0)
    else:
        state["window"] = case["window"]
    return state


def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


def _own(s):
    import bit_weight_only_int4_amd as q4
    op = s["op"]
    if op == "append":
        q = q4.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["cu_new"],
                         s["lengths"], q=s["q"], inv_freq=s["inv_freq"], interleaved=s["interleaved"], max_new=s["max_new"])
        k, v = q4.kv_dequant(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], dtype=torch.bfloat16)
        return dict(q=q, k=k, v=v, k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "attention":
        return q4.attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["cu_new"],
                            s["lengths"], window=s["window"], max_new=s["max_new"], max_len=s["max_len"])
    if op == "logprobs":
        r = q4.token_logprobs(s["logits"], s["targets"], top_k=s["top_k"])
        return dict(logprob=r.logprob, entropy=r.entropy, lse=r.lse, top_ids=r.top_ids, top_logprobs=r.top_logprobs)
    return q4.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"])


def _tokens(s):
    """Sequence and position of every new token."""
    cu, lengths = s["cu_new"].long(), s["lengths"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return t, b, lengths[b] - cu[b + 1] + t


def _rotate(x, pos, inv_freq, interleaved):
    """Pairs of the first 2 * len(inv_freq) elements turned by pos * inv_freq; angles in 64 bits, products in 32."""
    half = inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()[None, :]
    c, n = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    y = x.float().clone()
    if interleaved:
        a, b = y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * n, b * c + a * n
    else:
        a, b = y[..., :half].clone(), y[..., half:2 * half].clone()
        y[..., :half], y[..., half:2 * half] = a * c - b * n, b * c + a * n
    return y


def _store(x, cache, scale, page, off):
    """New rows x [T, kv_heads, head_dim] into a cache viewed as [pages, kv_heads, page, head_dim]: a page's scale
    grows to fit them and what the page held is coded anew; a page whose slot 0 is written starts from nothing."""
    P, Hk = scale.shape
    amax = torch.zeros((P, Hk), device=x.device).scatter_reduce_(0, page[:, None].expand(-1, Hk), x.abs().amax(2), "amax")
    touched = torch.zeros(P, dtype=torch.bool, device=x.device)
    touched[page] = True
    # 1 where slot 0 is written (a sum, as a page has many tokens)
    fresh = torch.zeros(P, device=x.device).index_add_(0, page, (off == 0).float()) > 0
    old = torch.where(fresh[:, None], 0.0, scale)
    grown = torch.where(touched[:, None], torch.maximum(old, amax / CODE_MAX), old)
    ratio = torch.where(grown > 0, old / grown, 0.0)
    codes = (cache.float() * ratio[:, :, None, None]).round()
    sx = grown[page][:, :, None]
    codes[page, :, off] = torch.where(sx > 0, (x / sx).round().clamp(-CODE_MAX, CODE_MAX), 0.0)
    cache.copy_(codes)
    scale.copy_(grown)


def _plain_append(s):
    t, b, pos = _tokens(s)
    PS = s["k_cache"].shape[2]
    page, off = s["page_table"][b, pos // PS].long(), pos % PS
    _store(_rotate(s["k"], pos, s["inv_freq"], s["interleaved"]), s["k_cache"], s["k_scale"], page, off)
    _store(s["v"].float(), s["v_cache"].transpose(2, 3), s["v_scale"], page, off)
    value = lambda c, sc: (c.float() * sc[:, :, None, None]).to(torch.bfloat16)  # noqa: E731
    return dict(q=_rotate(s["q"], pos, s["inv_freq"], s["interleaved"]).to(s["q"].dtype), k=value(s["k_cache"], s["k_scale"]),
                v=value(s["v_cache"], s["v_scale"]).transpose(2, 3).contiguous(), k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_attention(s):
    q, table = s["q"], s["page_table"]
    PS, (T, Hq, D) = s["k_cache"].shape[2], q.shape
    Hk, B = s["k_cache"].shape[1], table.shape[0]
    G, N, L = Hq // Hk, s["max_new"], s["max_len"]
    n_pages = (L + PS - 1) // PS
    pages = table[:, :n_pages].clamp(min=0).long()
    # keys [B, Hk, D, L'] and values [B, Hk, L', D] of every sequence, padded to the longest
    keys = (s["k_cache"][pages].float() * s["k_scale"][pages][..., None, None]).permute(0, 2, 4, 1, 3).reshape(B, Hk, D, n_pages * PS)
    values = (s["v_cache"][pages].float() * s["v_scale"][pages][..., None, None]).permute(0, 2, 1, 4, 3).reshape(B, Hk, n_pages * PS, D)
    t, b, pos = _tokens(s)
    i = t - s["cu_new"].long()[b]
    rows = torch.zeros((B, N, Hq, D), device=q.device)
    rows[b, i] = q.float()
    at = torch.full((B, N), -1, dtype=torch.long, device=q.device)
    at[b, i] = pos
    rows = rows.reshape(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * G, D)
    scores = torch.matmul(rows, keys).mul_(1.0 / math.sqrt(D)).view(B, Hk, N, G, -1)
    j = torch.arange(n_pages * PS, device=q.device)
    seen = j[None, None, :] <= at[:, :, None]
    if s["window"]:
        seen &= j[None, None, :] > at[:, :, None] - s["window"]
    scores.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top > float("-inf"), top, 0.0)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.view(B, Hk, N * G, -1), values).view(B, Hk, N, G, D)
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)[b, i].to(q.dtype)


def _plain_logprobs(s):
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    y = x - top
    e = torch.exp(y)
    total = e.sum(1)
    log_total = torch.log(total)
    logprob = y.gather(1, s["targets"][:, None])[:, 0] - log_total
    entropy = log_total - (e * y).sum(1) / total
    # a stable sort keeps equal values in the order of their index
    best, ids = torch.sort(y, dim=1, descending=True, stable=True)
    k = s["top_k"]
    return dict(logprob=logprob, entropy=entropy, lse=top[:, 0] + log_total, top_ids=ids[:, :k].contiguous(),
                top_logprobs=best[:, :k] - log_total[:, None])


def _plain_logprobs_grad(s):
    logp = s["logits"].float() - s["lse"][:, None]
    grad = -torch.exp(logp) * (s["g_logprob"][:, None] + s["g_entropy"][:, None] * (logp + s["entropy"][:, None]))
    grad.scatter_add_(1, s["targets"][:, None], s["g_logprob"][:, None])
    return grad.to(s["logits"].dtype)


PLAIN = {"append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad}


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] in ("logprobs", "logprobs_grad"):
        n = case["rows"] * case["vocab"]
        back = case["op"] == "logprobs_grad"
        return {"bytes": n * e * (2 if back else 1) + case["rows"] * (20 + 12 * case.get("top_k", 0)), "flops": 5 * n}
    new, lengths = _spans(case)
    T, Hq, Hk, D, PS = sum(new), case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        # q read and written, new keys and values read and their codes written, then every page's values given back in 16 bits
        slots = PS * sum(-(-L // PS) - (L - n) // PS for n, L in zip(new, lengths))
        return {"bytes": 2 * T * Hq * D * e + 2 * T * Hk * D * (e + 1) + 2 * slots * Hk * D * 3, "flops": 3 * T * (Hq + Hk) * D}
    w = case["window"]
    keys = sum(min(L, w + n - 1) if w else L for n, L in zip(new, lengths))
    pairs = sum(min(p + 1, w) if w else p + 1 for n, L in zip(new, lengths) for p in range(L - n, L))
    return {"bytes": 2 * keys * Hk * D + 2 * T * Hq * D * e, "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        logp = torch.log_softmax(s["logits"].double(), 1)
        lse = torch.logsumexp(s["logits"].double(), 1)
        k = s["top_k"]
        # whole numbers are compared between the two sides; here only the values
        return dict(logprob=logp[torch.arange(logp.shape[0], device=logp.device), s["targets"]], entropy=-(logp.exp() * logp).sum(1),
                    lse=lse, top_ids=None, top_logprobs=torch.topk(logp, k, 1).values)
    if case["op"] == "logprobs_grad":
        x = s["logits"].double().requires_grad_(True)
        logp = torch.log_softmax(x, 1)
        chosen = logp[torch.arange(x.shape[0], device=x.device), s["targets"]]
        entropy = -(logp.exp() * logp).sum(1)
        loss = (chosen * s["g_logprob"].double()).sum() + (entropy * s["g_entropy"].double()).sum()
        return torch.autograd.grad(loss, x)[0]
    new, lengths = _spans(case)
    PS, D = case["page"], case["head_dim"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    table = s["page_table"].cpu()
    dev = s["q"].device
    if case["op"] == "attention":
        Hk, G = case["kv_heads"], case["heads"] // case["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        for b, (n, L) in enumerate(zip(new, lengths)):
            ids = table[b, :-(-L // PS)].long().to(dev)
            rows = s["q"][cu[b]:cu[b + 1]].double()
            ahead = torch.arange(L, device=dev)[None, :] - torch.arange(L - n, L, device=dev)[:, None]
            hidden = ahead > 0
            if case["window"]:
                hidden |= ahead <= -case["window"]
            for h in range(Hk):
                key = (s["k_cache"][ids, h].double() * s["k_scale"][ids, h, None, None].double()).reshape(-1, D)[:L]
                value = (s["v_cache"][ids, h].double() * s["v_scale"][ids, h, None, None].double()).transpose(1, 2).reshape(-1, D)[:L]
                for m in range(h * G, (h + 1) * G):
                    z = (rows[:, m] @ key.t() / math.sqrt(D)).masked_fill_(hidden, float("-inf"))
                    out[cu[b]:cu[b + 1], m] = torch.softmax(z, 1) @ value
        return out
    # the append, page by page
    def turned(x, positions):
        half = s["inv_freq"].numel()
        z = torch.polar(torch.ones((), dtype=torch.float64, device=dev), positions[:, None] * s["inv_freq"].double())[:, None, :]
        x = x.double()
        lead = x[..., :2 * half]
        pairs = lead.unflatten(-1, (half, 2)) if case["interleaved"] else lead.unflatten(-1, (2, half)).transpose(-1, -2)
        w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        w = w.flatten(-2) if case["interleaved"] else w.transpose(-1, -2).flatten(-2)
        return torch.cat([w, x[..., 2 * half:]], -1)

    q = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    k, v = s["k_cache"].double(), s["v_cache"].transpose(2, 3).double()
    ks, vs = s["k_scale"].double(), s["v_scale"].double()
    for b, (n, L) in enumerate(zip(new, lengths)):
        positions = torch.arange(L - n, L, dtype=torch.float64, device=dev)
        at = slice(cu[b], cu[b + 1])
        q[at] = turned(s["q"][at], positions)
        rows = (turned(s["k"][at], positions), s["v"][at].double())
        for j in range((L - n) // PS, -(-L // PS)):
            lo, hi = max(L - n, j * PS), min(L, (j + 1) * PS)
            page = int(table[b, j])
            for x, codes, scales in ((rows[0], k, ks), (rows[1], v, vs)):
                part = x[lo - (L - n):hi - (L - n)].transpose(0, 1)
                old = scales[page] if lo % PS else torch.zeros_like(scales[page])
                grown = torch.maximum(old, part.abs().amax((1, 2)) / CODE_MAX)
                codes[page] = (codes[page] * (old / grown)[:, None, None]).round()
                codes[page, :, lo % PS:lo % PS + hi - lo] = (part / grown[:, None, None]).round().clamp(-CODE_MAX, CODE_MAX)
                scales[page] = grown
    return dict(q=q, k=k * ks[:, :, None, None], v=v * vs[:, :, None, None], k_scale=ks, v_scale=vs)
