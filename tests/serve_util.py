"""Inputs of the cache and attention tests: ragged sequences on shuffled
pages, everything around them poisoned (page numbers past the sequences out of
range, unused slots with codes, unused pages with NaN scales)."""
import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """new[b] new tokens, the last of lengths[b], over pages of `page` tokens."""

    def __init__(self, new, lengths, page, seed, spare_pages=3, extra_cols=2):
        self.new, self.lengths, self.page = list(new), list(lengths), page
        g = np.random.default_rng(seed)
        need = [max(0, -(-n // page)) for n in lengths]
        self.pages = sum(need) + spare_pages
        ids = g.permutation(self.pages)
        cols = max(need + [1]) + extra_cols
        # entries that no token uses name no page
        self.table = g.choice([-1, -(1 << 31), self.pages, (1 << 31) - 1],
                              size=(len(need), cols)).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.used = ids[:at]
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.len = np.array(self.lengths, dtype=np.int32)
        self.T = int(self.cu[-1])

    def device(self):
        return [torch.from_numpy(x).cuda() for x in (self.table, self.cu, self.len)]


def random_cache(batch, kv_heads, dim, seed, scale_spread=1.0):
    """Codes over the whole range -127 .. 127 in every slot, scales of used
    pages random, of the others NaN."""
    g = np.random.default_rng(seed)
    P, S = batch.pages, batch.page
    k = np.clip(np.rint(g.normal(0, 42, (P, kv_heads, S, dim))), -127, 127).astype(np.int8)
    v = np.clip(np.rint(g.normal(0, 42, (P, kv_heads, dim, S))), -127, 127).astype(np.int8)
    ks = np.full((P, kv_heads), np.nan, np.float32)
    vs = np.full((P, kv_heads), np.nan, np.float32)
    u = batch.used
    ks[u] = np.exp(g.uniform(-scale_spread, scale_spread, (len(u), kv_heads))) / 42
    vs[u] = np.exp(g.uniform(-scale_spread, scale_spread, (len(u), kv_heads))) / 42
    return k, v, ks, vs


def rounded(x, dtype):
    """numpy fp64 -> (torch CPU tensor of dtype, the fp64 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype])
    return t, t.double().numpy()


def strided(t, kind):
    """The tensor [T, heads, dim] on the GPU in one of several layouts."""
    t = t.cuda()
    T, H, D = t.shape
    if kind == "packed":
        return t.contiguous()
    if kind == "fused":  # a slice of a wider row, poisoned around it
        buf = torch.full((T, H + 3, D + 16), float("nan"), dtype=t.dtype, device="cuda")
        buf[:, 1:H + 1, :D] = t
        return buf[:, 1:H + 1, :D]
    if kind == "heads_first":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if kind == "odd":  # element alignment only
        buf = torch.full((T * H * (D + 1) + 1,), float("nan"), dtype=t.dtype, device="cuda")
        view = buf[1:].view(T, H, D + 1)[:, :, :D]
        view.copy_(t)
        return view
    raise ValueError(kind)
