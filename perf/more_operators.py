"""Measured cases of the operators around packed experts and the packed output
head: routing tokens to experts, the experts' gated 4-bit products, and the
head's softmax cross entropy without its logits, each with its gradient.

``run`` computes each operator in its plain form (elementary torch operations
in fp32, the values that decide a choice in fp64) while ``own`` is false, and
through the package's entry points while it is true.  ``exact`` gives the same
outputs in fp64 from the operators' definitions.

Packed weights are those of the 4-bit layer, one matrix after the other:
  gate_up  uint8 [experts, 2 * width, hidden / 2]  (gate rows first), scales
           float32 [experts, ceil(hidden / group), 2 * width]
  down     uint8 [experts, hidden, width / 2], scales [experts, ceil(width /
           group), hidden]
  head     uint8 [vocab, hidden / 2], scales [ceil(hidden / group), vocab]
with a scale per row ([experts, rows], [vocab]) where group is 0.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # a decode step's routing: softmax scores, renormalised; latency counts
        dict(name="route_decode", op="route", dtype="f32", tokens=32, experts=64, top_k=8, score="softmax", bias=False,
             groups=1, top_groups=1, renormalize=True, scale=1.0),
        # a prompt batch over many experts in groups, balanced by a bias
        dict(name="route_prompt_groups", op="route", dtype="f32", tokens=8192, experts=256, top_k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, renormalize=True, scale=2.5),
        # a training batch's routing with its gradient, in 16 bits, weights left as they are
        dict(name="route_train", op="route_train", dtype="bf16", tokens=4096, experts=60, top_k=4, score="softmax",
             bias=False, groups=1, top_groups=1, renormalize=False, scale=1.0),
        # one conversation's decode step through a layer's experts: the smallest call
        dict(name="experts_decode_one", op="experts", dtype="f32", tokens=1, hidden=2048, width=1024, experts=64, top_k=8,
             group=32),
        # a decode batch: most experts in use, a few tokens each
        dict(name="experts_decode_batch", op="experts", dtype="f32", tokens=48, hidden=2048, width=1024, experts=64,
             top_k=8, group=128),
        # a few drafted tokens over large experts of an odd width
        dict(name="experts_few_wide", op="experts", dtype="f16", tokens=7, hidden=4096, width=1416, experts=16, top_k=2,
             group=64),
        # a prompt batch in bf16, an odd number of tokens
        dict(name="experts_prompt", op="experts", dtype="bf16", tokens=4099, hidden=2048, width=1024, experts=64, top_k=8,
             group=128),
        # a prompt over few large experts in fp32 with small groups
        dict(name="experts_prompt_f32", op="experts", dtype="f32", tokens=2000, hidden=4096, width=3584, experts=8,
             top_k=2, group=32),
        # a training step over frozen experts: forward, and the gradients of the tokens and of the routing weights
        dict(name="experts_train", op="experts_train", dtype="bf16", tokens=2048, hidden=2048, width=1408, experts=32,
             top_k=4, group=128),
        # scoring a prompt without keeping its logits
        dict(name="head_loss_score", op="head", dtype="f32", rows=512, vocab=128257, hidden=2048, group=0),
        # a training batch: loss and its gradient
        dict(name="head_loss_train", op="head_train", dtype="bf16", rows=2048, vocab=128257, hidden=2048, group=0),
        # a small odd vocabulary and an odd depth, grouped scales, fp32
        dict(name="head_loss_odd", op="head_train", dtype="f32", rows=333, vocab=32003, hidden=2008, group=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_train", "experts", "experts", "experts_train", "head", "head_train"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op.startswith("route"):
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 384])
        bias = rng.random() < 0.5
        groups = rng.choice([1, 1, 4, 8]) if E % 8 == 0 and E >= 32 else 1
        top_groups = 1 if groups == 1 else rng.randint(2, groups)
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 16384), experts=E,
                    top_k=rng.randint(1, min(10, E * top_groups // groups)), score=rng.choice(["softmax", "sigmoid"]),
                    bias=bias, groups=groups, top_groups=top_groups, renormalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]))
    if op.startswith("experts"):
        E = rng.choice([4, 8, 16, 60, 64, 128])
        hidden = 8 * _log_int(rng, 32, 640)
        width = 8 * _log_int(rng, 16, max(17, min(448, 500_000_000 // (12 * hidden * E))))
        k = rng.randint(1, min(8, E))
        top = 300_000_000_000 // (6 * hidden * width * k)
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, max(2, min(8192, top))), hidden=hidden, width=width,
                    experts=E, top_k=k, group=rng.choice([0, 32, 64, 128, 128]))
    hidden = 8 * _log_int(rng, 32, 512)
    vocab = _log_int(rng, 1000, 160000)
    top = min(2048, 500_000_000_000 // (vocab * hidden), 250_000_000 // vocab)
    return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, max(2, top)), vocab=vocab, hidden=hidden,
                group=rng.choice([0, 0, 32, 128]))


def _packed(g, dev, lead, rows, depth, group, gain=1.0):
    """Random codes [*lead, rows, depth / 2] with scales that keep outputs near unit size."""
    codes = torch.randint(0, 256, (*lead, rows, depth // 2), generator=g, device=dev, dtype=torch.uint8)
    shape = (*lead, rows) if group == 0 else (*lead, -(-depth // group), rows)
    scales = (0.5 + torch.rand(shape, generator=g, device=dev)) * (gain / (4.6 * depth ** 0.5))
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    op = case["op"]
    state = dict(case)
    if op.startswith("route"):
        T, E = case["tokens"], case["experts"]
        # some experts are more popular than others
        state["logits"] = (1.5 * randn(T, E) + 0.5 * randn(E)).to(dt)
        state["balance"] = 0.1 * randn(E) if case["bias"] else None
        if op == "route_train":
            state["g_weights"] = randn(T, case["top_k"])
    elif op.startswith("experts"):
        T, H, W, E, k = case["tokens"], case["hidden"], case["width"], case["experts"], case["top_k"]
        state["gate_up"], state["gate_up_scales"] = _packed(g, dev, (E,), 2 * W, H, case["group"])
        state["down"], state["down_scales"] = _packed(g, dev, (E,), H, W, case["group"])
        state["x"] = randn(T, H).to(dt)
        # as a router leaves them
        best, ids = torch.topk(1.5 * randn(T, E) + 0.5 * randn(E), k, 1)
        state["ids"], state["weights"] = ids.to(torch.int32), torch.softmax(best, 1)
        if op == "experts_train":
            state["dout"] = randn(T, H).to(dt)
    else:
        M, V, H = case["rows"], case["vocab"], case["hidden"]
        state["qw"], state["scales"] = _packed(g, dev, (), V, H, case["group"], 2.5)
        state["x"] = randn(M, H).to(dt)
        state["targets"] = torch.randint(0, V, (M,), generator=g, device=dev)
        if op == "head_train":  # a tenth of the positions are not trained on
            state["targets"][torch.rand(M, generator=g, device=dev) < 0.1] = -1
            state["g_loss"] = torch.full((M,), 1.0 / M, device=dev)
    return state


def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


def _own(s):
    import bit_weight_only_int4_amd as q4
    op = s["op"]
    if op.startswith("route"):
        r = q4.route(s["logits"], s["top_k"], score=s["score"], bias=s["balance"], groups=s["groups"],
                     top_groups=s["top_groups"], renormalize=s["renormalize"], scale=s["scale"])
        out = dict(ids=r.ids, weights=r.weights)
        if op == "route_train":
            out["dlogits"] = q4.route_backward(s["logits"], r.ids, s["g_weights"], score=s["score"],
                                               renormalize=s["renormalize"], scale=s["scale"])
        return out
    if op == "experts":
        return q4.experts(s["x"], s["ids"], s["weights"], s["gate_up"], s["gate_up_scales"], s["down"], s["down_scales"],
                          group_size=s["group"])
    if op == "experts_train":
        out, pre = q4.experts(s["x"], s["ids"], s["weights"], s["gate_up"], s["gate_up_scales"], s["down"],
                              s["down_scales"], group_size=s["group"], keep=True)
        dx, dweights = q4.experts_backward(s["dout"], s["ids"], s["weights"], pre, s["gate_up"], s["gate_up_scales"],
                                           s["down"], s["down_scales"], group_size=s["group"])
        return dict(out=out, dx=dx, dweights=dweights)
    r = q4.head_cross_entropy(s["x"], s["qw"], s["scales"], s["targets"], group_size=s["group"], nibble_order="high_first")
    out = dict(loss=r.loss, lse=r.lse)
    if op == "head_train":
        out["dx"] = q4.head_cross_entropy_backward(s["x"], s["qw"], s["scales"], s["targets"], r.lse, s["g_loss"],
                                                   group_size=s["group"], nibble_order="high_first")
    return out


def _order(values, k):
    """Indices of the k largest of each row; a stable sort keeps equal values in the order of their index."""
    return torch.sort(values, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s):
    z = s["logits"].float()
    T, E = z.shape
    k, G = s["top_k"], s["groups"]
    scores = torch.softmax(z, 1) if s["score"] == "softmax" else torch.sigmoid(z)
    # without a bias the scores' order is the logits'; with one, the sums next to each other are told apart in 64 bits
    choice = s["logits"].double()
    if s["balance"] is not None:
        choice = (torch.softmax(choice, 1) if s["score"] == "softmax" else torch.sigmoid(choice)) + s["balance"].double()
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        value = best[..., 0] if s["balance"] is None else best[..., :2].sum(2)
        kept = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, _order(value, s["top_groups"]), True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, 1), float("-inf"))
    ids = _order(choice, k)
    weights = scores.gather(1, ids)
    if s["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return dict(ids=ids.to(torch.int32), weights=weights * s["scale"])


def _plain_route_train(s):
    out = _plain_route(s)
    z, ids, g = s["logits"].float(), out["ids"].long(), s["g_weights"] * s["scale"]
    scores = torch.softmax(z, 1) if s["score"] == "softmax" else torch.sigmoid(z)
    chosen = scores.gather(1, ids)
    if s["renormalize"]:
        total = chosen.sum(1, keepdim=True)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(z).scatter_(1, ids, g)
    if s["score"] == "softmax":
        dz = scores * (ds - (ds * scores).sum(1, keepdim=True))
    else:
        dz = ds * scores * (1 - scores)
    out["dlogits"] = dz.to(s["logits"].dtype)
    return out


def _matrix(codes, scales, group, low_first=True):
    """The fp32 matrix [rows, depth] that packed codes [rows, depth / 2] stand for."""
    low, high = codes & 15, codes >> 4
    w = torch.stack((low, high) if low_first else (high, low), -1).flatten(-2).float() - 8.0
    if group == 0:
        return w * scales[:, None]
    return w * scales.repeat_interleave(group, 0)[:w.shape[1]].t()


def _plain_experts(s, train=False):
    x, ids, weights = s["x"].float(), s["ids"].long(), s["weights"]
    W = s["width"]
    out, dx, dweights = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(weights)
    for e in torch.unique(ids).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        gate_up = _matrix(s["gate_up"][e], s["gate_up_scales"][e], s["group"])
        down = _matrix(s["down"][e], s["down_scales"][e], s["group"])
        gate, up = (x[t] @ gate_up.t()).split(W, 1)
        sig = torch.sigmoid(gate)
        h = gate * sig * up
        w = weights[t, j][:, None]
        out.index_add_(0, t, w * (h @ down.t()))
        if train:
            dh = s["dout"][t].float() @ down
            dweights[t, j] = (h * dh).sum(1)
            dh = dh * w
            dgate = dh * up * sig * (1 + gate * (1 - sig))
            dx.index_add_(0, t, torch.cat([dgate, dh * gate * sig], 1) @ gate_up)
    dt = s["x"].dtype
    return dict(out=out.to(dt), dx=dx.to(dt), dweights=dweights) if train else out.to(dt)


def _plain_head(s, train=False):
    x, targets = s["x"].float(), s["targets"]
    w = _matrix(s["qw"], s["scales"], s["group"], low_first=False)
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    chosen = z.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    out = dict(loss=torch.where(targets >= 0, lse - chosen, 0.0), lse=lse)
    if train:
        g = torch.where(targets >= 0, s["g_loss"], 0.0)[:, None]
        p = z.sub_(lse[:, None]).exp_().mul_(g)
        p.scatter_add_(1, targets.clamp(min=0)[:, None], -g)
        out["dx"] = (p @ w).to(s["x"].dtype)
    return out


PLAIN = {"route": _plain_route, "route_train": _plain_route_train, "experts": _plain_experts,
         "experts_train": lambda s: _plain_experts(s, True), "head": _plain_head, "head_train": lambda s: _plain_head(s, True)}


def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    if op.startswith("route"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        train = op == "route_train"
        return {"bytes": T * E * e * (2 if train else 1) + T * k * (12 if train else 8), "flops": (9 if train else 5) * T * E}
    if op.startswith("experts"):
        T, H, W, E, k = (case[n] for n in ("tokens", "hidden", "width", "experts", "top_k"))
        used = min(E, T * k)
        scales = 2 * W + H if case["group"] == 0 else -(-H // case["group"]) * 2 * W + -(-W // case["group"]) * H
        train = op == "experts_train"
        return {"bytes": used * (3 * H * W // 2 + 4 * scales) + T * H * e * (4 if train else 2) + T * k * (12 if train else 8),
                "flops": (12 if train else 6) * T * k * H * W}
    M, V, H = case["rows"], case["vocab"], case["hidden"]
    scales = V * (1 if case["group"] == 0 else -(-H // case["group"]))
    train = op == "head_train"
    return {"bytes": V * H // 2 + 4 * scales + M * H * e * (2 if train else 1) + M * 16, "flops": (6 if train else 2) * M * V * H}


def _exact_matrix(codes, scales, group, high_first=False):
    """The packed matrix in fp64, column by column of its bytes."""
    rows, depth = codes.shape[0], 2 * codes.shape[1]
    w = torch.empty((rows, depth), dtype=torch.float64, device=codes.device)
    first = 1 if high_first else 0
    w[:, first::2] = (codes % 16).double()
    w[:, 1 - first::2] = (codes // 16).double()
    w -= 8
    if group == 0:
        return w.mul_(scales.double()[:, None])
    at = torch.arange(depth, device=codes.device) // group
    return w.mul_(scales.double().t()[:, at])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("route"):
        z = s["logits"].double().requires_grad_(True)
        scores = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) if case["score"] == "softmax" else 1 / (1 + torch.exp(-z))
        # the choice is compared between the two sides; here only the values
        with torch.no_grad():
            value = (scores if s["balance"] is not None else z) + (0 if s["balance"] is None else s["balance"].double())
            first = lambda v, n: torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]  # noqa: E731
            if case["groups"] > 1:
                parts = torch.stack(value.chunk(case["groups"], 1), 1)
                lead = parts.topk(1 if s["balance"] is None else 2, 2).values.sum(2)
                at = torch.arange(len(parts), device=parts.device)[:, None], first(lead, case["top_groups"])
                value = torch.full_like(parts, -math.inf).index_put(at, parts[at]).flatten(1)
            ids = first(value, case["top_k"])
        w = scores.gather(1, ids)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        w = w * case["scale"]
        if op == "route":
            return dict(ids=None, weights=w.detach())
        return dict(ids=None, weights=w.detach(), dlogits=torch.autograd.grad((w * s["g_weights"].double()).sum(), z)[0])
    if op.startswith("experts"):
        train = op == "experts_train"
        x = s["x"].double().requires_grad_(train)
        w = s["weights"].double().requires_grad_(train)
        parts, rows = [], []
        for e in range(case["experts"]):
            t, j = torch.where(s["ids"] == e)
            if t.numel() == 0:
                continue
            gu = _exact_matrix(s["gate_up"][e], s["gate_up_scales"][e], case["group"])
            d = _exact_matrix(s["down"][e], s["down_scales"][e], case["group"])
            pre = x[t] @ gu.t()
            h = torch.nn.functional.silu(pre[:, :case["width"]]) * pre[:, case["width"]:]
            parts.append((h @ d.t()) * w[t, j][:, None])
            rows.append(t)
        out = torch.zeros_like(x).index_add(0, torch.cat(rows), torch.cat(parts))
        if not train:
            return out
        dx, dweights = torch.autograd.grad(out, (x, w), s["dout"].double())
        return dict(out=out.detach(), dx=dx, dweights=dweights)
    w = _exact_matrix(s["qw"], s["scales"], case["group"], True)
    z = s["x"].double() @ w.t()
    lse = torch.logsumexp(z, 1)
    used = s["targets"] >= 0
    at = torch.where(used, s["targets"], 0)
    loss = torch.where(used, lse - z[torch.arange(len(at), device=at.device), at], 0.0)
    out = dict(loss=loss, lse=lse)
    if op == "head_train":
        p = torch.softmax(z, 1)
        p[torch.arange(len(at), device=at.device), at] -= 1
        out["dx"] = (p * (s["g_loss"].double() * used)[:, None]) @ w
    return out
