"""Block-scaled 8-bit linear layers and the norms between them, for torch tensors.

Marshalling only, like the rest of the binding: arguments are checked, results
and workspaces allocated, and the C ABI called.  8-bit matrices are
``torch.float8_e4m3fn`` with float32 scales, one per 128 values along K: per
row for activations, per 128 x 128 values for weights.

Results are allocated on the stream the call runs on.  With an explicit
``stream`` that is not the current one, the inputs are recorded on it, so that
the caching allocator does not hand their memory out again too early; ordering
it after the work that makes them is the caller's.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import NamedTuple, Optional

from ._binding import TMAGEMM_OK, TmaGemmError, TmagemmNorm, lib

FP8_BLOCK = 128
_GATE_NONE, _GATE_CHANNEL, _GATE_TOKEN, _GATE_ELEMENT = range(4)


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _on_stream(device, stream, inputs):
    """A context in which `device` is current and, with an explicit stream, that
    stream is (so that results are allocated on it), and the stream's handle."""
    import torch
    if stream is None:
        ctx = (nullcontext() if device.index == torch.cuda.current_device()
               else torch.cuda.device(device))
        return ctx, torch.cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    if stream != torch.cuda.current_stream(device):
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
    return torch.cuda.stream(stream), stream.cuda_stream


def _check(name, t, dtype, shape, device=None, contiguous=True):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _bf16(dtype) -> int:
    import torch
    if dtype == torch.bfloat16:
        return 1
    if dtype == torch.float16:
        return 0
    raise TypeError(f"the type must be torch.float16 or torch.bfloat16, got {dtype}")


def _strides2(t):
    """(row, column) strides of a scale matrix; a stride that is never stepped
    (a dimension of one) counts as 1.  Broadcast (zero) strides are refused by
    the library."""
    r, c = t.stride()
    return (r if t.shape[0] > 1 else 1), (c if t.shape[1] > 1 else 1)


def _raise(status, what):
    if status != TMAGEMM_OK:
        raise TmaGemmError(status, what)


def quantize_fp8(X, block_rows: int = 1, stream=None):
    """Block quantisation of a CUDA fp16 or bf16 matrix X (M, K) -> (Q, S).

    Q is float8_e4m3fn (M, K); S is float32 (ceil(M / block_rows),
    ceil(K / 128)) with ``block_rows`` 1 (activations) or 128 (weights).  Row
    scales are laid out with consecutive rows next to each other, the layout
    the products read fastest; weight scales are row-major.
    """
    import torch
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise TypeError("X must be a CUDA matrix")
    bf16 = _bf16(X.dtype)
    _check("X", X, X.dtype, None)
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    M, K = X.shape
    rows, blocks = -(-M // block_rows), _blocks(K)
    ctx, handle = _on_stream(X.device, stream, (X,))
    with ctx:
        Q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=X.device)
        if block_rows == 1:
            S = torch.empty((blocks, rows), dtype=torch.float32, device=X.device)
            s_row, s_blk = 1, max(rows, 1)
        else:
            S = torch.empty((rows, blocks), dtype=torch.float32, device=X.device)
            s_row, s_blk = max(blocks, 1), 1
        _raise(lib().quantize_fp8(M, K, X.data_ptr(), bf16, block_rows, Q.data_ptr(),
                                  S.data_ptr(), s_row, s_blk, handle), "quantize_fp8")
    return Q, (S.t() if block_rows == 1 else S)


def gemm_fp8(A, SA, B, SB, dtype=None, out=None, stream=None):
    """D (M, N) = (A * SA) @ (B * SB).T with block scales, in ``dtype`` (bf16 by
    default, or fp16).

    A (M, K) and B (N, K) are float8_e4m3fn; SA (M, ceil(K / 128)) float32 with
    any strides, SB (ceil(N / 128), ceil(K / 128)) float32, row-major.
    K % 16 == 0 and N % 8 == 0.
    """
    import torch
    if out is not None:
        dtype = out.dtype if dtype is None else dtype
    bf16 = _bf16(dtype if dtype is not None else torch.bfloat16)
    dtype = torch.bfloat16 if bf16 else torch.float16
    f8, f32 = torch.float8_e4m3fn, torch.float32
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be matrices")
    M, K = A.shape
    N = B.shape[0]
    dev = A.device
    _check("A", A, f8, None)
    _check("B", B, f8, (N, K), dev)
    _check("SA", SA, f32, (M, _blocks(K)), dev, contiguous=False)
    _check("SB", SB, f32, (_blocks(N), _blocks(K)), dev)
    sa_row, sa_blk = _strides2(SA)
    ctx, handle = _on_stream(dev, stream, (A, SA, B, SB, out))
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=dtype, device=dev)
        else:
            _check("out", out, dtype, (M, N), dev)
        _raise(lib().gemm_fp8(M, N, K, A.data_ptr(), SA.data_ptr(), sa_row, sa_blk, B.data_ptr(),
                              SB.data_ptr(), out.data_ptr(), bf16, handle), "gemm_fp8")
    return out


def gemm_fp8_grouped(A, SA, B, SB, m_offsets, dtype=None, out=None, stream=None):
    """Grouped D[rows of g] = (A * SA)[rows of g] @ (B[g] * SB[g]).T, where the
    rows of group g are m_offsets[g] .. m_offsets[g + 1] - 1.

    m_offsets is a CUDA int32 tensor (G + 1,), read by the kernel (no copy to
    the host); rows outside every group are left as they are in ``out``
    (undefined in a new result).  A (M, K), B (G, N, K), SB (G, ceil(N / 128),
    ceil(K / 128)); the rest as for gemm_fp8.
    """
    import torch
    if out is not None:
        dtype = out.dtype if dtype is None else dtype
    bf16 = _bf16(dtype if dtype is not None else torch.bfloat16)
    dtype = torch.bfloat16 if bf16 else torch.float16
    f8, f32 = torch.float8_e4m3fn, torch.float32
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be a matrix and B a stack of matrices")
    M, K = A.shape
    G, N = B.shape[:2]
    dev = A.device
    _check("A", A, f8, None)
    _check("B", B, f8, (G, N, K), dev)
    _check("SA", SA, f32, (M, _blocks(K)), dev, contiguous=False)
    _check("SB", SB, f32, (G, _blocks(N), _blocks(K)), dev)
    _check("m_offsets", m_offsets, torch.int32, (G + 1,), dev)
    sa_row, sa_blk = _strides2(SA)
    ctx, handle = _on_stream(dev, stream, (A, SA, B, SB, m_offsets, out))
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=dtype, device=dev)
        else:
            _check("out", out, dtype, (M, N), dev)
        _raise(lib().gemm_fp8_grouped(G, m_offsets.data_ptr(), M, N, K, A.data_ptr(),
                                      SA.data_ptr(), sa_row, sa_blk, B.data_ptr(), SB.data_ptr(),
                                      out.data_ptr(), bf16, handle), "gemm_fp8_grouped")
    return out


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


def _norm_struct(h, y, gate, w_post, w_pre, alpha, eps):
    """The checked operands as a TmagemmNorm."""
    import torch
    if not isinstance(h, torch.Tensor) or h.dim() != 2:
        raise TypeError("h must be a CUDA matrix (tokens, channels)")
    T, C = h.shape
    dt, dev = h.dtype, h.device
    p = TmagemmNorm()
    p.bf16 = _bf16(dt)
    _check("h", h, dt, None)
    if y is None and (w_pre is None or w_post is not None or gate is not None):
        raise ValueError("without y there is neither w_post nor gate, and w_pre is needed")
    for name, t, shape in (("y", y, (T, C)), ("w_post", w_post, (C,)), ("w_pre", w_pre, (C,))):
        if t is not None:
            _check(name, t, dt, shape, dev)
            setattr(p, name, t.data_ptr())
    p.T, p.C, p.alpha, p.eps, p.h = T, C, alpha, eps, h.data_ptr()
    if gate is not None:
        shape = tuple(gate.shape)
        if shape == (C,) or shape == (1, C):
            # With one token, (1, C) is also that token's elements; the
            # gradient is then the same but for its type.
            p.gate_mode = _GATE_CHANNEL if shape == (C,) or T != 1 else _GATE_ELEMENT
        elif shape == (T, C):
            p.gate_mode = _GATE_ELEMENT
        elif shape == (T, 1):
            p.gate_mode = _GATE_TOKEN
        else:
            raise ValueError(f"gate must be (C,), (1, C), (T, 1) or (T, C), got {shape}")
        _check("gate", gate, dt, None, dev)
        p.gate = gate.data_ptr()
    return p


def norm_residual(h, y=None, gate=None, w_post=None, w_pre=None, alpha: float = 1.0,
                  eps: float = 1e-6, quantize: bool = False, save_rstd: bool = False,
                  stream=None) -> NormOut:
    """The norms around a block, its gate and its residual, in one pass:

        u  = y * rsqrt(mean(y^2) + eps) * w_post    (u = y without w_post)
        h' = h + alpha * gate * u                   (h' = h without y)
        x  = h' * rsqrt(mean(h'^2) + eps) * w_pre   (no x without w_pre)

    h and y are (T, C) fp16 or bf16; gate is (C,), (T, 1), (T, C) or None.
    ``quantize`` makes x float8_e4m3fn codes with row scales, the operands of
    gemm_fp8; ``save_rstd`` keeps the two rsqrt factors for the backward.
    """
    import torch
    p = _norm_struct(h, y, gate, w_post, w_pre, alpha, eps)
    if quantize and w_pre is None:
        raise ValueError("quantize needs w_pre")
    T, C = h.shape
    dev = h.device
    ctx, handle = _on_stream(dev, stream, (h, y, gate, w_post, w_pre))
    h_out, x, scales, r_post, r_pre = h, None, None, None, None
    with ctx:
        if y is not None:
            h_out = torch.empty_like(h)
            p.h_out = h_out.data_ptr()
        if w_pre is not None and quantize:
            x = torch.empty((T, C), dtype=torch.float8_e4m3fn, device=dev)
            scales = torch.empty((_blocks(C), T), dtype=torch.float32, device=dev)
            p.q, p.scales, p.s_row_stride, p.s_block_stride = (
                x.data_ptr(), scales.data_ptr(), 1, max(T, 1))
            scales = scales.t()
        elif w_pre is not None:
            x = torch.empty_like(h)
            p.x = x.data_ptr()
        if save_rstd and w_post is not None:
            r_post = torch.empty((T,), dtype=torch.float32, device=dev)
            p.rstd_post = r_post.data_ptr()
        if save_rstd and w_pre is not None:
            r_pre = torch.empty((T,), dtype=torch.float32, device=dev)
            p.rstd_pre = r_pre.data_ptr()
        _raise(lib().norm_residual(ctypes.byref(p), handle), "norm_residual")
    return NormOut(h_out, x, scales, r_post, r_pre)


def norm_residual_backward(h, y=None, dh=None, dx=None, gate=None, w_post=None, w_pre=None,
                           alpha: float = 1.0, rstd_post=None, rstd_pre=None,
                           stream=None) -> NormGrads:
    """Gradients of norm_residual from its inputs, its rsqrt factors
    (``save_rstd=True``) and the gradients of its results: dh of h' (None:
    zero) and dx of x (given if and only if w_pre is).

    dh, dy and a (T, C) gate's gradient have the type of h; the weights' and the
    other gates' gradients are float32 sums.
    """
    import torch
    p = _norm_struct(h, y, gate, w_post, w_pre, alpha, 0.0)
    T, C = h.shape
    dt, dev = h.dtype, h.device
    f32 = torch.float32
    if (dx is None) != (w_pre is None):
        raise ValueError("dx is given if and only if w_pre is")
    for name, field, t in (("dh", "dh_out", dh), ("dx", "dx", dx)):
        if t is not None:
            _check(name, t, dt, (T, C), dev)
            setattr(p, field, t.data_ptr())
    for name, t, w in (("rstd_post", rstd_post, w_post), ("rstd_pre", rstd_pre, w_pre)):
        if w is not None:
            _check(name, t, f32, (T,), dev)
            setattr(p, name, t.data_ptr())
    ctx, handle = _on_stream(dev, stream, (h, y, dh, dx, gate, w_post, w_pre, rstd_post, rstd_pre))
    dy = dgate = dw_post = dw_pre = None
    with ctx:
        need = lib().norm_residual_backward_workspace_size(T, C)
        if need < 0:
            raise TmaGemmError(int(need), "norm_residual_backward_workspace_size")
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
        dh_in = torch.empty_like(h)
        p.dh = dh_in.data_ptr()
        if y is not None:
            dy = torch.empty_like(h)
            p.dy = dy.data_ptr()
        if gate is not None:
            dgate = torch.empty(gate.shape, device=dev,
                                dtype=dt if p.gate_mode == _GATE_ELEMENT else f32)
            p.dgate = dgate.data_ptr()
        if w_post is not None:
            dw_post = torch.empty((C,), dtype=f32, device=dev)
            p.dw_post = dw_post.data_ptr()
        if w_pre is not None:
            dw_pre = torch.empty((C,), dtype=f32, device=dev)
            p.dw_pre = dw_pre.data_ptr()
        _raise(lib().norm_residual_backward(ctypes.byref(p), workspace.data_ptr(), need, handle),
               "norm_residual_backward")
    return NormGrads(dh_in, dy, dgate, dw_post, dw_pre)
