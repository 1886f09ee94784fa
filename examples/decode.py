"""A decoder with 4-bit weights and an 8-bit cache, run with this package's
operators: prompts of different lengths enter together, tokens are decoded
greedily, a text is scored, and the score's gradient reaches the output head's
input.

    python examples/decode.py                # Llama-3.2-1B layer shapes, 4 layers
    python examples/decode.py --layers 16 --steps 64

Weights are random (seeded); there is no tokenizer.  Per layer: a root-mean-
square norm, the fused q/k/v projection (q4 linear), ``kv_append`` (keys and
values into the paged cache, queries and keys turned on the way, the queries in
place in the projection's rows), ``attention``, the output projection, and a
gated feed-forward part; then the output head and ``token_logprobs``.
"""
import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_weight_only_int4_amd as q4  # noqa: E402


@dataclass(frozen=True)
class Shape:
    hidden: int = 2048
    layers: int = 4
    heads: int = 32
    kv_heads: int = 8
    head_dim: int = 64
    ffn: int = 8192
    vocab: int = 128257
    group: int = 32
    page: int = 64
    rope_base: float = 500000.0


class Linear:
    """Random 4-bit weights [N, K] with grouped (or per-channel) scales."""

    def __init__(self, N, K, group, gen, device):
        self.K, self.group = K, group
        self.qw = torch.randint(0, 256, (N, (K + 1) // 2), generator=gen, dtype=torch.uint8).to(device)
        shape = (N,) if group == 0 else (-(-K // group), N)
        # codes have a standard deviation of about 4.6: outputs of unit scale
        self.scales = ((0.5 + torch.rand(shape, generator=gen)) / (4.6 * K ** 0.5)).to(device)

    def __call__(self, x):
        return q4.linear(x, self.qw, self.scales, K=self.K, group_size=self.group)

    def backward(self, dout):
        return q4.linear_backward(dout, self.qw, self.scales, K=self.K, group_size=self.group)


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)


class Decoder:
    def __init__(self, shape: Shape, pages: int, batch: int, max_pages: int, seed: int = 0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        s = self.shape = shape
        make = lambda n, k: Linear(n, k, s.group, gen, device)  # noqa: E731
        self.embed = torch.randn((s.vocab, s.hidden), generator=gen).to(device)
        self.layers = [dict(qkv=make((s.heads + 2 * s.kv_heads) * s.head_dim, s.hidden),
                            out=make(s.hidden, s.heads * s.head_dim), up=make(2 * s.ffn, s.hidden),
                            down=make(s.hidden, s.ffn),
                            cache=q4.new_cache(pages, s.kv_heads, s.head_dim, s.page, device))
                       for _ in range(s.layers)]
        self.head = Linear(s.vocab, s.hidden, 0, gen, device)
        self.inv_freq = (s.rope_base ** (-torch.arange(0, s.head_dim, 2, dtype=torch.float64) / s.head_dim)
                         ).float().to(device)
        # the pages of a batch's sequences, given out in order as they grow
        self.free = list(range(pages))[::-1]
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32)
        self.lengths = [0] * batch

    def step(self, tokens, new, trace=None):
        """new[b] next tokens of every sequence, packed: the hidden state of each."""
        s = self.shape
        for b, n in enumerate(new):
            have, self.lengths[b] = -(-self.lengths[b] // s.page), self.lengths[b] + n
            for j in range(have, -(-self.lengths[b] // s.page)):
                self.table[b, j] = self.free.pop()
        dev = tokens.device
        table = self.table.to(dev)
        cu = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device=dev)
        lengths = torch.tensor(self.lengths, dtype=torch.int32, device=dev)
        bounds = dict(max_new=max(new), max_len=max(self.lengths))
        x = self.embed[tokens]
        for i, layer in enumerate(self.layers):
            rows = layer["qkv"](norm(x)).view(len(tokens), s.heads + 2 * s.kv_heads, s.head_dim)
            q, k, v = rows.split([s.heads, s.kv_heads, s.kv_heads], 1)
            if trace is not None:
                trace.append(dict(layer=i, q_in=q.clone(), k=k.clone(), v=v.clone(), table=table, cu=cu, lengths=lengths,
                                  before=[c.clone() for c in layer["cache"]]))
            q4.kv_append(k, v, *layer["cache"], table, cu, lengths, q=q, q_out=q, inv_freq=self.inv_freq,
                         max_new=bounds["max_new"])
            o = q4.attention(q, *layer["cache"], table, cu, lengths, **bounds)
            if trace is not None:
                trace[-1].update(q=q.clone(), out=o, after=[c.clone() for c in layer["cache"]])
            x = x + layer["out"](o.view(len(tokens), -1))
            gate, up = layer["up"](norm(x)).chunk(2, 1)
            x = x + layer["down"](torch.nn.functional.silu(gate) * up)
        return norm(x)

    def logits(self, hidden):
        return self.head(hidden.contiguous())


def last_of(new, device):
    """The row of each sequence's last token."""
    return torch.tensor(new, device=device).cumsum(0) - 1


def generate(model, prompts, steps, top_k=3):
    """Greedy continuations [batch, steps] of packed prompts, their log
    probabilities, and the first choices' alternatives."""
    new = [len(p) for p in prompts]
    hidden = model.step(torch.cat(prompts), new)[last_of(new, prompts[0].device)]
    ids, logprobs, first = [], [], None
    for _ in range(steps):
        r = q4.token_logprobs(model.logits(hidden), top_k=top_k)
        first = first if first is not None else r
        ids.append(r.top_ids[:, 0])
        logprobs.append(r.top_logprobs[:, 0])
        hidden = model.step(ids[-1], [1] * len(prompts))
    return torch.stack(ids, 1), torch.stack(logprobs, 1), first


def score(model, hidden, targets, entropy_weight=0.01):
    """Log probability and entropy of each target after its hidden state, and
    the gradient of mean(logprob + entropy_weight * entropy) with respect to
    the hidden states."""
    logits = model.logits(hidden)
    r = q4.token_logprobs(logits, targets)
    g = torch.full_like(r.logprob, 1.0 / len(targets))
    dlogits = q4.token_logprobs_backward(logits, targets, r.lse, r.entropy, g, entropy_weight * g, dlogits=logits)
    return r, model.head.backward(dlogits)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompts", type=int, nargs="+", default=[17, 300, 64, 129])
    a = ap.parse_args()
    shape = Shape(layers=a.layers)
    per = -(-(max(a.prompts) + a.steps + 1) // shape.page)
    model = Decoder(shape, pages=per * len(a.prompts), batch=len(a.prompts), max_pages=per)
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, shape.vocab, (n,), generator=gen).cuda() for n in a.prompts]
    start = time.perf_counter()
    ids, logprobs, first = generate(model, prompts, a.steps)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    print(f"{len(prompts)} prompts of {a.prompts} tokens, {a.steps} decoded each, {took * 1e3:.1f} ms")
    for b in range(len(prompts)):
        alternatives = ", ".join(f"{i} ({p:.2f})" for i, p in zip(first.top_ids[b].tolist(), first.top_logprobs[b].tolist()))
        print(f"  {b}: {ids[b, :8].tolist()} ... sum of log probabilities {logprobs[b].sum():.2f}; first from {alternatives}")
    model2 = Decoder(shape, pages=per, batch=1, max_pages=per)
    hidden = model2.step(prompts[1][:-1], [len(prompts[1]) - 1])
    r, dx = score(model2, hidden, prompts[1][1:])
    print(f"prompt 1 scored: mean log probability {r.logprob.mean():.3f}, mean entropy {r.entropy.mean():.3f}, "
          f"gradient norm {dx.norm():.3e}")


if __name__ == "__main__":
    main()
