"""What stands around the products of routed experts, for torch tensors: the router's
choice, rows laid out by expert, their weighted sum, and the gradients.

    ids, weights = route_topk(logits, k)
    r = dispatch_rows(x, ids, experts, quantize=True)
    out = gemm_fp8_grouped(r.rows, r.scales, B, SB, r.offsets)     # or gemm_w4_grouped
    y = combine_rows(out, r.row_of, weights)

Marshalling only (the native binding, as for the 8-bit operators): no call waits for the
device or is recorded by autograd.  The gradients are calls of their own, for an
autograd.Function of the caller's: y's through combine_rows_backward (to the rows and
the weights), the rows' through combine_rows without weights (to x), the weights'
through route_topk_backward (to the logits).
"""
from __future__ import annotations

from typing import NamedTuple, Optional

from .fp8 import _on_stream, _ops


class RouteOut(NamedTuple):
    """Results of route_topk."""
    ids: object                 # (T, k) int32, best first; -1 where no expert was left
    weights: object             # (T, k) float32


class DispatchOut(NamedTuple):
    """Results of dispatch_rows."""
    rows: object                # (T k, C): x by expert, or its codes with quantize=True
    scales: Optional[object]    # row scales of the codes
    offsets: object             # (experts + 1,) int32: the grouped products' m_offsets
    row_of: object              # (T, k) int32: the row of each choice, -1 without one


class CombineGrads(NamedTuple):
    """Results of combine_rows_backward."""
    drows: object
    dweights: object


def _sigmoid(score: str) -> bool:
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return score == "sigmoid"


def route_topk(logits, k: int, score: str = "softmax", bias=None, groups: int = 1,
               top_groups: int = 1, group_sum: int = 1, renormalize: bool = True,
               scale: float = 1.0, stream=None) -> RouteOut:
    """k experts and their weights for each row of CUDA logits (T, E), float32, float16
    or bfloat16.

    Experts are chosen by p + bias with p = softmax(logits) or sigmoid(logits), best
    first, ties to the lowest index; ``bias`` is float32 (E,).  With ``groups`` the E
    experts are that many runs of equal length, of which the ``top_groups`` whose
    ``group_sum`` (1 or 2) best values have the largest sum are chosen from.  The weights
    are scale * p, without the bias, divided by their sum over the chosen with
    ``renormalize``.  A logit of -inf closes an expert; choices that none is left for get
    id -1 and weight 0.  A bias of +inf puts its expert first, -inf last.

    E is at most 512 and k 32; the grouped products that follow take 384 experts.
    """
    args = (logits, k, _sigmoid(score), bias, groups, top_groups, group_sum, renormalize, scale)
    if stream is None:
        return RouteOut(*_ops().route_topk(*args))
    return RouteOut(*_on_stream(stream, _ops().route_topk, *args))


def route_topk_backward(logits, ids, dweights, score: str = "softmax", renormalize: bool = True,
                        scale: float = 1.0, stream=None):
    """The gradient of the logits (T, E), in their type, from that of route_topk's weights
    (T, k) float32, with the choice ``ids`` held fixed.  A token's ids are different experts,
    as route_topk makes them; those outside 0 .. E - 1 have no gradient."""
    args = (logits, ids, dweights, _sigmoid(score), renormalize, scale)
    if stream is None:
        return _ops().route_topk_backward(*args)
    return _on_stream(stream, _ops().route_topk_backward, *args)


def dispatch_rows(x, ids, experts: int, quantize: bool = False, stream=None) -> DispatchOut:
    """Rows of CUDA x (T, C), fp16 or bf16, laid out by expert: a row for each choice in
    ``ids`` (T, k) int32, in the order of the experts and, for one expert, of the choices.
    Choices outside 0 .. experts - 1 get no row, and rows past the last are undefined.

    ``quantize`` makes the rows float8_e4m3fn codes with row scales, the operands of
    gemm_fp8_grouped.  The gradient of x is combine_rows(drows, row_of).
    """
    if stream is None:
        return DispatchOut(*_ops().dispatch_rows(x, ids, experts, quantize))
    return DispatchOut(*_on_stream(stream, _ops().dispatch_rows, x, ids, experts, quantize))


def combine_rows(rows, row_of, weights=None, stream=None):
    """y[t] = sum_j weights[t, j] * rows[row_of[t, j]] for CUDA rows (R, C), fp16 or bf16:
    (T, C) in their type.  ``weights`` is (T, k) float32, or None for ones; choices whose
    row_of is -1 add nothing."""
    if stream is None:
        return _ops().combine_rows(rows, row_of, weights)
    return _on_stream(stream, _ops().combine_rows, rows, row_of, weights)


def combine_rows_backward(dy, rows, row_of, weights, stream=None) -> CombineGrads:
    """Gradients of combine_rows from dy (T, C): of the rows, in their type (rows that no
    choice has are undefined), and of the weights, float32.  No row may have two
    choices."""
    if stream is None:
        return CombineGrads(*_ops().combine_rows_backward(dy, rows, row_of, weights))
    return CombineGrads(*_on_stream(stream, _ops().combine_rows_backward, dy, rows, row_of,
                                    weights))
