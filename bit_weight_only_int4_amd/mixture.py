"""Python binding of ``include/q4experts.h``: routing tokens to experts, the
experts' gated feed-forward over packed 4-bit weights, and the packed output
head's softmax cross entropy without its logits, each with its gradient.

As in ``serve`` this is argument marshalling only, checked in C++
(``csrc/q4_experts_py.h``); outputs and workspaces are allocated with torch and
the work runs in the HIP library on torch's current stream.  There is no CPU
fallback.  A wrong tensor raises ``ValueError``, a status of the library
``Q4Error``.

Packed weights are those of ``linear``, contiguous, one matrix after the other
for experts:
  codes   uint8 [experts, rows, depth / 2]
  scales  float32 [experts, ceil(depth / group_size), rows], or [experts, rows]
          with group_size 0
with depths that are multiples of 8 and a group_size of 0, 32 or a multiple of
64.  They are constants: gradients are those of the activations, which are
float32, float16 or bfloat16.
"""
import ctypes
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import serve as _serve
from .q4linear import ORDERS, lib
from .serve import DTYPES, _stream

SCORES = {"softmax": 0, "sigmoid": 1}

# exported symbols of include/q4experts.h
SYMBOLS = ("q4_route", "q4_route_backward", "q4_experts", "q4_experts_workspace_bytes",
           "q4_experts_backward", "q4_experts_backward_workspace_bytes", "q4_head_cross_entropy",
           "q4_head_cross_entropy_workspace_bytes", "q4_head_cross_entropy_backward",
           "q4_head_cross_entropy_backward_workspace_bytes")

_bound = None


def _lib() -> ctypes.CDLL:
    """The HIP library with these entry points' argument types declared."""
    global _bound
    if _bound is None:
        L = lib()
        P, I, I32, SZ, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                            ctypes.c_float)
        L.q4_route.argtypes = [P, I, I32, I, I, I, I32, P, I, I, I32, F, P, P, P]
        L.q4_route_backward.argtypes = [P, I, I32, I, I, I, P, I32, I32, F, P, P, I, P]
        L.q4_experts.argtypes = ([P, I, I32] + [I] * 5 + [P] * 6 + [I, I32, P, I, P, P, SZ, P])
        L.q4_experts_backward.argtypes = ([P, I, I32] + [I] * 5 + [P] * 7
                                          + [I, I32, P, I, P, P, SZ, P])
        L.q4_head_cross_entropy.argtypes = [P, I, I32, I, I, I, P, P, I, I32, P, P, P, P, SZ, P]
        L.q4_head_cross_entropy_backward.argtypes = [P, I, I32, I, I, I, P, P, I, I32, P, P, P, P, I,
                                                     P, SZ, P]
        L.q4_experts_workspace_bytes.argtypes = [I32] + [I] * 6
        L.q4_experts_backward_workspace_bytes.argtypes = [I32] + [I] * 6
        L.q4_head_cross_entropy_workspace_bytes.argtypes = [I32] + [I] * 4
        L.q4_head_cross_entropy_backward_workspace_bytes.argtypes = [I32] + [I] * 4
        for name in SYMBOLS:
            getattr(L, name).restype = SZ if name.endswith("_bytes") else I32
        _bound = L
    return _bound


def _native():
    return _serve._module or _serve._native()


def _choice(table, value, name):
    code = table.get(value) if isinstance(value, str) else None
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {value!r}")
    return code


class Route(NamedTuple):
    ids: torch.Tensor      # int32 [T, top_k]; -1 where fewer experts are eligible
    weights: torch.Tensor  # float32 [T, top_k]


def route(logits: torch.Tensor, top_k: int, *, score: str = "softmax",
          bias: Optional[torch.Tensor] = None, groups: int = 1, top_groups: int = 1,
          renormalize: bool = True, scale: float = 1.0) -> Route:
    """The top_k experts of each row of logits [T, experts], in descending
    order (ties to the lowest index), and their weights: scale * score, the
    scores divided by the sum of the chosen if ``renormalize``.  ``bias``
    (float32 [experts]) is added to the scores for the choice alone.  With
    ``groups`` > 1 only the ``top_groups`` groups of consecutive experts with
    the largest best expert (with a bias: sum of the two best) take part.  An
    expert whose logit is -inf takes no part."""
    return Route._make(_native().route(logits, top_k, _choice(SCORES, score, "score"), bias, groups,
                                       top_groups, renormalize, scale, _stream(logits)))


def route_backward(logits: torch.Tensor, ids: torch.Tensor, g_weights: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of sum(g_weights * weights) with respect to the logits, of
    their type, for the choice ``ids`` that ``route`` made.  ``dlogits`` may be
    the logits themselves."""
    return _native().route_backward(logits, ids, g_weights, _choice(SCORES, score, "score"),
                                    renormalize, scale, dlogits, _stream(logits))


def experts_workspace_bytes(T: int, hidden: int, width: int, experts: int, top_k: int, *,
                            group_size: int, dtype=torch.float32) -> int:
    return int(_lib().q4_experts_workspace_bytes(DTYPES[dtype], T, hidden, width, experts, top_k,
                                                 group_size))


def experts_backward_workspace_bytes(T: int, hidden: int, width: int, experts: int, top_k: int, *,
                                     group_size: int, dtype=torch.float32) -> int:
    return int(_lib().q4_experts_backward_workspace_bytes(DTYPES[dtype], T, hidden, width, experts,
                                                          top_k, group_size))


def experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up: torch.Tensor,
            gate_up_scales: torch.Tensor, down: torch.Tensor, down_scales: torch.Tensor, *,
            group_size: int, nibble_order: str = "low_first", keep: bool = False,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
            ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """out[t] = sum_j weights[t, j] * down_e (silu(gate_e x[t]) * (up_e x[t]))
    with e = ids[t, j], of x's type [T, hidden].  ids int32 and weights float32
    are [T, top_k], as ``route`` gives them: a negative id is an empty slot, one
    past the experts makes its token NaN.  gate_up holds [experts, 2 * width,
    hidden / 2], the gate's rows first, down [experts, hidden, width / 2].  With
    ``keep`` also returns what ``experts_backward`` needs: gate and up before
    the product, float32 [T, top_k, 2 * width] (undefined in empty slots)."""
    return _native().experts(x, ids, weights, gate_up, gate_up_scales, down, down_scales, group_size,
                             _choice(ORDERS, nibble_order, "nibble_order"), keep, out, workspace,
                             _stream(x))


def experts_backward(dout: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, pre: torch.Tensor,
                     gate_up: torch.Tensor, gate_up_scales: torch.Tensor, down: torch.Tensor,
                     down_scales: torch.Tensor, *, group_size: int, nibble_order: str = "low_first",
                     dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradients of sum(dout * out): (dx of dout's type [T, hidden], dweights
    float32 [T, top_k]).  ``pre`` is what ``experts`` kept."""
    return _native().experts_backward(dout, ids, weights, pre, gate_up, gate_up_scales, down,
                                      down_scales, group_size,
                                      _choice(ORDERS, nibble_order, "nibble_order"), dx, workspace,
                                      _stream(dout))


class HeadLoss(NamedTuple):
    loss: torch.Tensor  # float32 [M]
    lse: torch.Tensor   # float32 [M]


def head_cross_entropy_workspace_bytes(M: int, vocab: int, K: int, *, group_size: int,
                                       dtype=torch.float32) -> int:
    return int(_lib().q4_head_cross_entropy_workspace_bytes(DTYPES[dtype], M, vocab, K, group_size))


def head_cross_entropy_backward_workspace_bytes(M: int, vocab: int, K: int, *, group_size: int,
                                                dtype=torch.float32) -> int:
    return int(_lib().q4_head_cross_entropy_backward_workspace_bytes(DTYPES[dtype], M, vocab, K,
                                                                     group_size))


def head_cross_entropy(x: torch.Tensor, qw: torch.Tensor, scales: torch.Tensor,
                       targets: torch.Tensor, *, group_size: int, nibble_order: str = "low_first",
                       workspace: Optional[torch.Tensor] = None) -> HeadLoss:
    """Softmax cross entropy of the packed head's logits of x [M, K] against
    targets (int64 [M]; negative: none, loss 0), and log sum exp of the logits,
    which are never stored."""
    return HeadLoss._make(_native().head_cross_entropy(
        x, qw, scales, targets, group_size, _choice(ORDERS, nibble_order, "nibble_order"), workspace,
        _stream(x)))


def head_cross_entropy_backward(x: torch.Tensor, qw: torch.Tensor, scales: torch.Tensor,
                                targets: torch.Tensor, lse: torch.Tensor, g_loss: torch.Tensor, *,
                                group_size: int, nibble_order: str = "low_first",
                                dx: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of sum(g_loss * loss) with respect to x, of x's type, given
    the lse that ``head_cross_entropy`` returned."""
    return _native().head_cross_entropy_backward(
        x, qw, scales, targets, group_size, _choice(ORDERS, nibble_order, "nibble_order"), lse, g_loss,
        dx, workspace, _stream(x))
