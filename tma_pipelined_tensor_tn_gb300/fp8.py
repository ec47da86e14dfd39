"""Block-scaled 8-bit linear layers and the norms between them, for torch tensors.

Marshalling only, like the rest of the binding, but native
(``csrc/torch_ops.cpp``): the operands are checked, results and workspaces
allocated, and the C ABI called.  8-bit matrices are ``torch.float8_e4m3fn``
with float32 scales, one per 128 values along K: per row for activations, per
128 x 128 values for weights.

No call is recorded by autograd: what it makes never requires gradients, whatever the
inputs do.  The norms' gradients come from norm_residual_backward, for an
autograd.Function of the caller's own; the products and the quantiser have none.

Results are allocated on the stream the call runs on.  With an explicit
``stream`` that is not the current one, the inputs are recorded on it, so that
the caching allocator does not hand their memory out again too early; ordering
it after the work that makes them is the caller's.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional

from ._binding import TmaGemmError, lib

FP8_BLOCK = 128
_FUNCTIONS = ("quantize_fp8", "gemm_fp8", "gemm_fp8_grouped", "norm_residual",
              "norm_residual_backward", "norm_residual_backward_workspace_size")
_lock = threading.Lock()
_native = None


def _ops():
    """The native binding, with the library's functions bound (raises if either
    has not been built)."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (its libraries are what the module links to)
        with _lock:
            path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_torch_ops.so")
            if not os.path.exists(path):
                raise RuntimeError(f"{path} not found: build it first (python -c "
                                   "'import __graft_entry__ as g; g.build()')")
            from . import _torch_ops
            library = lib()
            _torch_ops.bind({name: ctypes.cast(getattr(library, name), ctypes.c_void_p).value
                             for name in _FUNCTIONS}, TmaGemmError)
            _native = _torch_ops
    return _native


def _on_stream(stream, function, *args):
    """function(*args) with `stream` current and the tensors recorded on it."""
    import torch
    tensors = [t for t in args if isinstance(t, torch.Tensor)]
    for t in tensors:
        if t.is_cuda and t.device != stream.device:
            raise ValueError(f"the stream is on {stream.device}, a tensor on {t.device}")
    if stream != torch.cuda.current_stream(stream.device):
        for t in tensors:
            if t.is_cuda:
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        return function(*args)


def _type_flag(dtype, out) -> int:
    """1 for bf16, 0 for fp16, -1 for the type of `out`."""
    import torch
    if dtype is None:
        return 1 if out is None else -1
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"the type must be torch.float16 or torch.bfloat16, got {dtype}")
    return int(dtype == torch.bfloat16)


def quantize_fp8(X, block_rows: int = 1, stream=None):
    """Block quantisation of a CUDA fp16 or bf16 matrix X (M, K) -> (Q, S).

    Q is float8_e4m3fn (M, K); S is float32 (ceil(M / block_rows),
    ceil(K / 128)) with ``block_rows`` 1 (activations) or 128 (weights).  Row
    scales are laid out with consecutive rows next to each other, the layout
    the products read fastest; weight scales are row-major.
    """
    if stream is None:
        return _ops().quantize_fp8(X, block_rows)
    return _on_stream(stream, _ops().quantize_fp8, X, block_rows)


def gemm_fp8(A, SA, B, SB, dtype=None, out=None, stream=None):
    """D (M, N) = (A * SA) @ (B * SB).T with block scales, in ``dtype`` (bf16 by
    default, or fp16).

    A (M, K) and B (N, K) are float8_e4m3fn; SA (M, ceil(K / 128)) float32 with
    any strides, SB (ceil(N / 128), ceil(K / 128)) float32, row-major.
    K % 16 == 0 and N % 8 == 0.
    """
    flag = _type_flag(dtype, out)
    if stream is None:
        return _ops().product(A, SA, B, SB, None, flag, out)
    return _on_stream(stream, _ops().product, A, SA, B, SB, None, flag, out)


def gemm_fp8_grouped(A, SA, B, SB, m_offsets, dtype=None, out=None, stream=None):
    """Grouped D[rows of g] = (A * SA)[rows of g] @ (B[g] * SB[g]).T, where the
    rows of group g are m_offsets[g] .. m_offsets[g + 1] - 1.

    m_offsets is a CUDA int32 tensor (G + 1,), read by the kernel (no copy to
    the host); rows outside every group are left as they are in ``out``
    (undefined in a new result).  A (M, K), B (G, N, K), SB (G, ceil(N / 128),
    ceil(K / 128)); the rest as for gemm_fp8.
    """
    flag = _type_flag(dtype, out)
    if m_offsets is None:
        raise TypeError("m_offsets must be a CUDA tensor")
    if stream is None:
        return _ops().product(A, SA, B, SB, m_offsets, flag, out)
    return _on_stream(stream, _ops().product, A, SA, B, SB, m_offsets, flag, out)


class NormOut(NamedTuple):
    """Results of norm_residual; None where a part was not asked for."""
    h: object                       # the residual stream after the block
    x: Optional[object]             # the next block's input (codes with quantize=True)
    scales: Optional[object]        # row scales of the codes
    rstd_post: Optional[object]     # the rsqrt factors, for the backward
    rstd_pre: Optional[object]


class NormGrads(NamedTuple):
    """Results of norm_residual_backward; None where the operand was not given."""
    dh: object
    dy: Optional[object]
    dgate: Optional[object]
    dw_post: Optional[object]
    dw_pre: Optional[object]


def norm_residual(h, y=None, gate=None, w_post=None, w_pre=None, alpha: float = 1.0,
                  eps: float = 1e-6, quantize: bool = False, save_rstd: bool = False,
                  stream=None) -> NormOut:
    """The norms around a block, its gate and its residual, in one pass:

        u  = y * rsqrt(mean(y^2) + eps) * w_post    (u = y without w_post)
        h' = h + alpha * gate * u                   (h' = h without y)
        x  = h' * rsqrt(mean(h'^2) + eps) * w_pre   (no x without w_pre)

    h and y are (T, C) fp16 or bf16; gate is (C,), (T, 1), (T, C) or None.  (A gate
    per channel has one dimension: (1, C) is a gate per element of one token.)
    ``quantize`` makes x float8_e4m3fn codes with row scales, the operands of
    gemm_fp8; ``save_rstd`` keeps the two rsqrt factors for the backward.
    """
    if stream is None:
        r = _ops().norm_residual(h, y, gate, w_post, w_pre, alpha, eps, quantize, save_rstd)
    else:
        r = _on_stream(stream, _ops().norm_residual, h, y, gate, w_post, w_pre, alpha, eps,
                       quantize, save_rstd)
    return NormOut(h, *r[1:]) if y is None else NormOut(*r)


def norm_residual_backward(h, y=None, dh=None, dx=None, gate=None, w_post=None, w_pre=None,
                           alpha: float = 1.0, rstd_post=None, rstd_pre=None,
                           stream=None) -> NormGrads:
    """Gradients of norm_residual from its inputs, its rsqrt factors
    (``save_rstd=True``) and the gradients of its results: dh of h' (None:
    zero) and dx of x (given if and only if w_pre is).

    dh, dy and a (T, C) gate's gradient have the type of h; the weights' and the
    other gates' gradients are float32 sums.
    """
    args = (h, y, dh, dx, gate, w_post, w_pre, alpha, rstd_post, rstd_pre)
    if stream is None:
        return NormGrads(*_ops().norm_residual_backward(*args))
    return NormGrads(*_on_stream(stream, _ops().norm_residual_backward, *args))
