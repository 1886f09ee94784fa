"""Python binding of ``include/q4serve.h``: the paged 8-bit key/value cache,
attention over it, and token log probabilities of the output head's logits.

As in ``q4linear`` this is argument marshalling only: tensors are checked
against the sizes the kernels will use (the C ABI sees pointers and strides,
not extents), outputs and workspaces are allocated with torch, and the work
runs in the HIP library on torch's current stream.  There is no CPU fallback.
The checks are in C++ (``csrc/q4_serve_py.cpp``), since a decode step's calls
take no longer on the GPU than they took in Python.  A wrong tensor raises
``ValueError``, a status of the library ``Q4Error``.

The cache of one layer (``new_cache`` makes an empty one):
  k_cache  int8 [pages, kv_heads, page, head_dim]
  v_cache  int8 [pages, kv_heads, head_dim, page]  (tokens innermost)
  k_scale, v_scale  float32 [pages, kv_heads]
Sequence b's new tokens of a call are rows ``cu_new[b] : cu_new[b + 1]`` of the
packed inputs; ``lengths[b]`` counts all of its tokens, the new ones last;
position p lies in slot ``p % page`` of page ``page_table[b, p // page]``.
"""
import ctypes
import os
from typing import NamedTuple, Optional, Tuple

import torch

from . import build as _build
from .q4linear import Q4Error, _need, lib

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
PAGES = (16, 32, 64, 128)

# exported symbols of include/q4serve.h
SYMBOLS = ("q4_kv_append", "q4_kv_dequant", "q4_attention", "q4_attention_workspace_bytes",
           "q4_token_logprobs", "q4_token_logprobs_workspace_bytes",
           "q4_token_logprobs_backward")

_bound = None
_module = None
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


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


def _native():
    """The C++ half of this binding."""
    global _module
    if _module is None:
        lib()  # reports a library that is missing or does not match the sources
        if not os.path.exists(_build.NATIVE):
            raise RuntimeError(
                f"{_build.NATIVE} is not built; run "
                "`python -c 'import __graft_entry__ as g; g.build()'` first")
        why = _build.stale_reason(_build.NATIVE)
        if why:
            raise RuntimeError(f"{_build.NATIVE} does not match the sources: {why}; rebuild it "
                               "(`python -c 'import __graft_entry__ as g; g.build()'`)")
        from . import _serve_native
        _serve_native.set_error(Q4Error)
        _module = _serve_native
    return _module


def _stream(t: torch.Tensor) -> int:
    """The current stream of the tensor's device (0 for a host tensor and for
    what is no tensor, which are refused later)."""
    d = t.get_device() if isinstance(t, torch.Tensor) else -1
    return _raw_stream(d) if d >= 0 else 0


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
    return (_module or _native()).kv_append(
        k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, lengths, q, q_out, inv_freq,
        interleaved, max_new, _stream(k))


def kv_dequant(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, *, dtype=torch.float32) -> Tuple[torch.Tensor, torch.Tensor]:
    """The values a cache stands for, code * scale: k and v, both [pages,
    kv_heads, page, head_dim]."""
    code = DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    return (_module or _native()).kv_dequant(k_cache, v_cache, k_scale, v_scale, code, _stream(k_cache))


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
    sequence (default: T and the page table's reach) and size the launch: rows
    past max_new and rows of no sequence are left as they are in ``out`` and
    undefined in a new tensor."""
    return (_module or _native()).attention(
        q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, lengths, softmax_scale, window,
        max_new, max_len, out, workspace, _stream(q))


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]       # float32 [M]; None without targets
    entropy: torch.Tensor                 # float32 [M]
    lse: torch.Tensor                     # float32 [M]
    top_ids: torch.Tensor                 # int64 [M, top_k]
    top_logprobs: torch.Tensor            # float32 [M, top_k]


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, top_k: int = 0,
                   workspace: Optional[torch.Tensor] = None) -> TokenLogprobs:
    """Log probability of each row's target (int64 [M]; negative: none, 0),
    the distribution's entropy, log sum exp, and the top_k (<= 32) most likely
    tokens with their log probabilities, of logits [M, vocab]."""
    return TokenLogprobs._make((_module or _native()).token_logprobs(
        logits, targets, top_k, workspace, _stream(logits)))


def token_logprobs_backward(logits: torch.Tensor, targets: Optional[torch.Tensor],
                            lse: torch.Tensor, entropy: torch.Tensor,
                            g_logprob: Optional[torch.Tensor],
                            g_entropy: Optional[torch.Tensor] = None, *,
                            dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient with respect to the logits of sum(g_logprob * logprob) +
    sum(g_entropy * entropy), given what ``token_logprobs`` returned; of the
    logits' type.  ``dlogits`` may be the logits themselves."""
    return (_module or _native()).token_logprobs_backward(
        logits, targets, lse, entropy, g_logprob, g_entropy, dlogits, _stream(logits))
