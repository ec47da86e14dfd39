"""Linear layers with 4-bit weights and group scales, for torch tensors.

Marshalling only (the native binding, as for the 8-bit operators).  A weight is
(q - z) * s: codes q of 0 .. 15, two to a byte with the even column in the low half,
scales s in the activations' type and zero points z (bytes of 0 .. 15; 8 where none are
given), one of each per row and ``group`` columns.

No call is recorded by autograd.
"""
from __future__ import annotations

from .fp8 import _on_stream, _ops


def gemm_w4(A, B, SB, ZB=None, group: int = 128, out=None, stream=None):
    """D (M, N) = A @ W.T for CUDA A (M, K), fp16 or bf16, and 4-bit weights: codes B
    (N, K / 2) uint8, scales SB (N, ceil(K / group)) in A's type and zero points ZB of the
    same shape, uint8, or None.  Summed in FP32, rounded once to A's type.

    ``group`` is 32, 64 or 128; K % 32 == 0.  Meant for the few tokens of decoding.
    """
    args = (A, B, SB, ZB, None, group, out)
    if stream is None:
        return _ops().product_w4(*args)
    return _on_stream(stream, _ops().product_w4, *args)


def gemm_w4_grouped(A, B, SB, m_offsets, ZB=None, group: int = 128, out=None, stream=None):
    """The same by expert: rows m_offsets[g] .. m_offsets[g + 1] - 1 of A with B[g], SB[g]
    and ZB[g].

    B (G, N, K / 2), SB and ZB (G, N, ceil(K / group)); m_offsets is a CUDA int32 tensor
    (G + 1,), read by the kernel (dispatch_rows makes it).  Rows outside every group are
    left as they are in ``out`` (undefined in a new result).
    """
    if m_offsets is None:
        raise TypeError("m_offsets must be a CUDA tensor")
    args = (A, B, SB, ZB, m_offsets, group, out)
    if stream is None:
        return _ops().product_w4(*args)
    return _on_stream(stream, _ops().product_w4, *args)
