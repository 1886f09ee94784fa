"""Python binding of ``include/q4serve.h``: the paged 8-bit key/value cache,
attention over it, and token log probabilities of the output head's logits.

As in ``q4linear`` this is argument marshalling only: tensors are checked
against the sizes the kernels will use (the C ABI sees pointers and strides,
not extents), outputs and workspaces are allocated with torch, and the work
runs in the HIP library on torch's current stream.  There is no CPU fallback.

The cache of one layer (``new_cache`` makes an empty one):
  k_cache  int8 [pages, kv_heads, page, head_dim]
  v_cache  int8 [pages, kv_heads, head_dim, page]  (tokens innermost)
  k_scale, v_scale  float32 [pages, kv_heads]
Sequence b's new tokens of a call are rows ``cu_new[b] : cu_new[b + 1]`` of the
packed inputs; ``lengths[b]`` counts all of its tokens, the new ones last;
position p lies in slot ``p % page`` of page ``page_table[b, p // page]``.
"""
import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from .q4linear import Q4_OK, Q4Error, _need, lib

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
PAGES = (16, 32, 64, 128)
MAX_TOP = 32

# exported symbols of include/q4serve.h
SYMBOLS = ("q4_kv_append", "q4_kv_dequant", "q4_attention", "q4_attention_workspace_bytes",
           "q4_token_logprobs", "q4_token_logprobs_workspace_bytes",
           "q4_token_logprobs_backward")

_bound = None


def _lib() -> ctypes.CDLL:
    """The HIP library with these entry points' argument types declared."""
    global _bound
    if _bound is None:
        L = lib()
        P, I, I32, SZ, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                            ctypes.c_float)
        L.q4_kv_append.argtypes = ([P, I, I] * 4 + [I32] + [I] * 5 + [P] * 4 + [I, I, P, I, I, P, P, I]
                                   + [P, I, I32, P])
        L.q4_kv_dequant.argtypes = [P] * 4 + [I] * 4 + [I32, P, P, P]
        L.q4_attention.argtypes = ([P, I, I] * 2 + [I32] + [I] * 5 + [P] * 4
                                   + [I, I, P, I, I, P, P, I, I, F, I, P, SZ, P])
        L.q4_attention_workspace_bytes.argtypes = [I32] + [I] * 9
        L.q4_token_logprobs.argtypes = [P, I, I32, I, I, P, I, P, P, P, P, P, P, SZ, P]
        L.q4_token_logprobs_workspace_bytes.argtypes = [I, I, I, I32]
        L.q4_token_logprobs_backward.argtypes = [P, I, I32, I, I, P, P, P, P, P, P, I, P]
        for name in SYMBOLS:
            getattr(L, name).restype = SZ if name.endswith("_bytes") else I32
        _bound = L
    return _bound


def _stream(t: torch.Tensor) -> int:
    """The current stream of the tensor's device."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _check(status: int, what: str) -> None:
    if status != Q4_OK:
        raise Q4Error(status, what)


def _dtype(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _rows3(t: torch.Tensor, name: str, dtype, device) -> Tuple[int, int]:
    """Token and head strides of a [T, heads, head_dim] tensor."""
    if t.dim() != 3 or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a 3-D {dtype} tensor on {device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    st = t.stride()
    if st[2] != 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return st[0], st[1]


def _vector(t: torch.Tensor, name: str, n: int, dtype, device) -> int:
    if t.dtype != dtype or t.device != device or t.dim() != 1 or t.numel() != n \
            or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on {device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _cache_sizes(k_cache, v_cache, k_scale, v_scale, device) -> Tuple[int, int, int, int]:
    """(pages, kv_heads, page, head_dim) of a cache whose four tensors fit together."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be int8 [pages, kv_heads, page, head_dim]")
    P, H, S, D = k_cache.shape
    if not (k_cache.dtype == v_cache.dtype == torch.int8 and v_cache.shape == (P, H, D, S)
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_cache.device == device and v_cache.device == device):
        raise ValueError("k_cache [pages, kv_heads, page, head_dim] and v_cache [pages, kv_heads, "
                         f"head_dim, page] must be contiguous int8 on {device}, got "
                         f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    if not (k_scale.dtype == v_scale.dtype == torch.float32 and k_scale.shape == (P, H)
            and v_scale.shape == (P, H) and k_scale.is_contiguous() and v_scale.is_contiguous()
            and k_scale.device == device and v_scale.device == device):
        raise ValueError(f"k_scale and v_scale must be contiguous float32 [{P}, {H}] on {device}")
    if S not in PAGES or D % 16 or not 16 <= D <= 256:
        raise ValueError(f"a page has 16, 32, 64 or 128 tokens and head_dim is a multiple of 16 up "
                         f"to 256, got {S} and {D}")
    return P, H, S, D


def _tables(page_table, cu_new, lengths, device) -> Tuple[int, int, int, int, int, int]:
    """(batch, page_table, its row pitch, its columns, cu_new, lengths), pointers where tensors."""
    if page_table.dtype != torch.int32 or page_table.device != device or page_table.dim() != 2 \
            or (page_table.size(1) > 1 and page_table.stride(1) != 1):
        raise ValueError(f"page_table must be int32 [batch, max_pages] on {device} with unit stride "
                         "along its rows")
    B, n = page_table.shape
    ld = page_table.stride(0) if B > 1 else n
    return (B, page_table.data_ptr(), ld, n, _vector(cu_new, "cu_new", B + 1, torch.int32, device),
            _vector(lengths, "lengths", B, torch.int32, device))


def new_cache(pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda"):
    """An empty cache: (k_cache, v_cache, k_scale, v_scale)."""
    _need(page in PAGES and head_dim % 16 == 0 and 16 <= head_dim <= 256,
          f"a page has 16, 32, 64 or 128 tokens and head_dim is a multiple of 16 up to 256, got "
          f"{page} and {head_dim}")
    return (torch.zeros((pages, kv_heads, page, head_dim), dtype=torch.int8, device=device),
            torch.zeros((pages, kv_heads, head_dim, page), dtype=torch.int8, device=device),
            torch.zeros((pages, kv_heads), dtype=torch.float32, device=device),
            torch.zeros((pages, kv_heads), dtype=torch.float32, device=device))


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              k_scale: torch.Tensor, v_scale: torch.Tensor, page_table: torch.Tensor,
              cu_new: torch.Tensor, lengths: torch.Tensor, *, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
              interleaved: bool = False, max_new: Optional[int] = None) -> Optional[torch.Tensor]:
    """Stores new keys and values [T, kv_heads, head_dim] in the cache, keys
    turned by pos * inv_freq (float32 [rot / 2]; None: not turned); queries q
    [T, heads, head_dim] are turned likewise into q_out (default: a new
    tensor, returned; q itself turns them in place).  ``lengths`` already
    counts the new tokens.  ``max_new`` bounds the new tokens of one sequence
    (default T)."""
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("k must be a device tensor")
    code = _dtype(k, "k")
    k_ts, k_hs = _rows3(k, "k", k.dtype, dev)
    v_ts, v_hs = _rows3(v, "v", k.dtype, dev)
    P, H, S, D = _cache_sizes(k_cache, v_cache, k_scale, v_scale, dev)
    T = k.shape[0]
    if k.shape != (T, H, D) or v.shape != (T, H, D):
        raise ValueError(f"k and v must be [T, {H}, {D}], got {tuple(k.shape)} and {tuple(v.shape)}")
    B, table, ld, n, cu, ln = _tables(page_table, cu_new, lengths, dev)
    heads, qp, q_ts, q_hs, op, o_ts, o_hs = H, None, 0, 0, None, 0, 0
    if q is not None:
        q_ts, q_hs = _rows3(q, "q", k.dtype, dev)
        heads = q.shape[1]
        if q.shape[0] != T or q.shape[2] != D or heads % H:
            raise ValueError(f"q must be [{T}, a multiple of {H}, {D}], got {tuple(q.shape)}")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        o_ts, o_hs = _rows3(q_out, "q_out", k.dtype, dev)
        if q_out.shape != q.shape:
            raise ValueError(f"q_out must be {tuple(q.shape)}, got {tuple(q_out.shape)}")
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot, fp = 0, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        fp = _vector(inv_freq, "inv_freq", rot // 2, torch.float32, dev)
        if rot > D:
            raise ValueError(f"inv_freq has {rot // 2} entries, more than head_dim / 2 = {D // 2}")
    _check(_lib().q4_kv_append(
        k.data_ptr(), k_ts, k_hs, v.data_ptr(), v_ts, v_hs, qp, q_ts, q_hs, op, o_ts, o_hs, code,
        T, B, heads, H, D, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), P, S, table, ld, n, cu, ln, T if max_new is None else max_new, fp, rot,
        1 if interleaved else 0, _stream(k)), "q4_kv_append")
    return q_out


def kv_dequant(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, *, dtype=torch.float32) -> Tuple[torch.Tensor, torch.Tensor]:
    """The values a cache stands for, code * scale: k and v, both [pages,
    kv_heads, page, head_dim]."""
    dev = k_cache.device
    if dev.type != "cuda":
        raise ValueError("k_cache must be a device tensor")
    P, H, S, D = _cache_sizes(k_cache, v_cache, k_scale, v_scale, dev)
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    k = torch.empty((P, H, S, D), dtype=dtype, device=dev)
    v = torch.empty((P, H, S, D), dtype=dtype, device=dev)
    _check(_lib().q4_kv_dequant(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), P, H, S, D, DTYPES[dtype], k.data_ptr(),
                                v.data_ptr(), _stream(k)), "q4_kv_dequant")
    return k, v


def attention_workspace_bytes(T: int, batch: int, heads: int, kv_heads: int, head_dim: int, *,
                              page: int, max_new: int, max_len: int, window: int = 0,
                              dtype=torch.float32) -> int:
    return int(_lib().q4_attention_workspace_bytes(DTYPES[dtype], T, batch, heads, kv_heads,
                                                   head_dim, page, max_new, max_len, window))


def attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
              v_scale: torch.Tensor, page_table: torch.Tensor, cu_new: torch.Tensor,
              lengths: torch.Tensor, *, softmax_scale: Optional[float] = None, window: int = 0,
              max_new: Optional[int] = None, max_len: Optional[int] = None,
              out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the new tokens' queries q [T, heads, head_dim] over their
    sequences' cached tokens up to their own position (and, with window > 0,
    the last ``window`` of those).  ``softmax_scale`` defaults to head_dim **
    -0.5; ``max_new`` and ``max_len`` bound the new tokens and the length of a
    sequence (default: T and the page table's reach) and size the launch."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be a device tensor")
    code = _dtype(q, "q")
    q_ts, q_hs = _rows3(q, "q", q.dtype, dev)
    P, H, S, D = _cache_sizes(k_cache, v_cache, k_scale, v_scale, dev)
    T, heads = q.shape[0], q.shape[1]
    if q.shape[2] != D or heads % H or heads == 0:
        raise ValueError(f"q must be [T, a multiple of {H}, {D}], got {tuple(q.shape)}")
    B, table, ld, n, cu, ln = _tables(page_table, cu_new, lengths, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    o_ts, o_hs = _rows3(out, "out", q.dtype, dev)
    if out.shape != q.shape:
        raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
    if max_new is None:
        max_new = T
    if max_len is None:
        max_len = n * S
    L = _lib()
    if workspace is None:
        need = L.q4_attention_workspace_bytes(code, T, B, heads, H, D, S, max_new, max_len, window)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wp, wn = None, 0
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {dev}")
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(L.q4_attention(
        q.data_ptr(), q_ts, q_hs, out.data_ptr(), o_ts, o_hs, code, T, B, heads, H, D,
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), P, S, table,
        ld, n, cu, ln, max_new, max_len, D ** -0.5 if softmax_scale is None else softmax_scale,
        window, wp, wn, _stream(q)), "q4_attention")
    return out


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]       # float32 [M]; None without targets
    entropy: torch.Tensor                 # float32 [M]
    lse: torch.Tensor                     # float32 [M]
    top_ids: torch.Tensor                 # int64 [M, top_k]
    top_logprobs: torch.Tensor            # float32 [M, top_k]


def _logit_rows(t: torch.Tensor, name: str) -> int:
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2 or t.size(1) < 1 or (t.size(1) > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D [M, vocab] with unit stride along its rows, got "
                         f"{tuple(t.shape)}")
    return t.stride(0) if t.size(0) > 1 else t.size(1)


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, top_k: int = 0,
                   workspace: Optional[torch.Tensor] = None) -> TokenLogprobs:
    """Log probability of each row's target (int64 [M]; negative: none, 0),
    the distribution's entropy, log sum exp, and the top_k (<= 32) most likely
    tokens with their log probabilities, of logits [M, vocab]."""
    ld = _logit_rows(logits, "logits")
    code = _dtype(logits, "logits")
    dev = logits.device
    M, V = logits.shape
    if not 0 <= top_k <= min(MAX_TOP, V):
        raise ValueError(f"top_k must be 0 .. {min(MAX_TOP, V)}, got {top_k}")
    tp = None if targets is None else _vector(targets, "targets", M, torch.int64, dev)
    stats = torch.empty((3, M), dtype=torch.float32, device=dev)
    logprob, entropy, lse = stats.unbind(0)
    ids = torch.empty((M, top_k), dtype=torch.int64, device=dev)
    top = torch.empty((M, top_k), dtype=torch.float32, device=dev)
    L = _lib()
    if workspace is None:
        need = L.q4_token_logprobs_workspace_bytes(M, V, top_k, code)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wp, wn = None, 0
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {dev}")
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    at = stats.data_ptr()
    _check(L.q4_token_logprobs(logits.data_ptr(), ld, code, M, V, tp, top_k,
                               None if tp is None else at, at + 4 * M, at + 8 * M, ids.data_ptr(),
                               top.data_ptr(), wp, wn, _stream(logits)), "q4_token_logprobs")
    return TokenLogprobs(None if tp is None else logprob, entropy, lse, ids, top)


def token_logprobs_backward(logits: torch.Tensor, targets: Optional[torch.Tensor],
                            lse: torch.Tensor, entropy: torch.Tensor,
                            g_logprob: Optional[torch.Tensor],
                            g_entropy: Optional[torch.Tensor] = None, *,
                            dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to the logits of sum(g_logprob * logprob) +
    sum(g_entropy * entropy), given what ``token_logprobs`` returned; of the
    logits' type.  ``dlogits`` may be the logits themselves."""
    ld = _logit_rows(logits, "logits")
    code = _dtype(logits, "logits")
    dev = logits.device
    M, V = logits.shape
    f32 = torch.float32
    tp = None if targets is None else _vector(targets, "targets", M, torch.int64, dev)
    gl = None if g_logprob is None else _vector(g_logprob, "g_logprob", M, f32, dev)
    ge = None if g_entropy is None else _vector(g_entropy, "g_entropy", M, f32, dev)
    if dlogits is None:
        dlogits = torch.empty((M, V), dtype=logits.dtype, device=dev)
    ldd = _logit_rows(dlogits, "dlogits")
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype or dlogits.device != dev:
        raise ValueError(f"dlogits must be {logits.dtype} {tuple(logits.shape)} on {dev}")
    _check(_lib().q4_token_logprobs_backward(
        logits.data_ptr(), ld, code, M, V, tp, _vector(lse, "lse", M, f32, dev),
        _vector(entropy, "entropy", M, f32, dev), gl, ge, dlogits.data_ptr(), ldd,
        _stream(logits)), "q4_token_logprobs_backward")
    return dlogits
