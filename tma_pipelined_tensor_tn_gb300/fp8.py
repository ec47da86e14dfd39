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
from typing import NamedTuple, Optional

import torch

from ._binding import TMAGEMM_OK, TmaGemmError, TmagemmNorm, lib

FP8_BLOCK = 128
_GATE_NONE, _GATE_CHANNEL, _GATE_TOKEN, _GATE_ELEMENT = range(4)
_F8, _F32 = torch.float8_e4m3fn, torch.float32
_IS_BF16 = {torch.bfloat16: 1, torch.float16: 0}
# These calls are as short as their launches: names are bound once, and the
# current device and stream are asked for as numbers (a Stream object alone
# costs as much as a launch).
_Tensor, _empty, _empty_like, _empty_strided = (torch.Tensor, torch.empty, torch.empty_like,
                                                torch.empty_strided)
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _launch(device, stream, inputs, body):
    """body(handle) with `device` current and, for an explicit stream, that
    stream current too, so that the results body() allocates belong to it."""
    if stream is None:
        index = device.index
        if index == _current_device():
            return body(_current_stream(index))
        with torch.cuda.device(device):
            return body(_current_stream(index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    if stream != torch.cuda.current_stream(device):
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _check(name, t, dtype, shape, device, contiguous=True):
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.device == device
            and (shape is None or t.shape == shape) and (not contiguous or t.is_contiguous())):
        return
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous (row-major)")


def _first(name, t, dims):
    """The device of a call's first operand: a CUDA tensor of `dims` dimensions."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.device


def _bf16(dtype) -> int:
    flag = _IS_BF16.get(dtype)
    if flag is None:
        raise TypeError(f"the type must be torch.float16 or torch.bfloat16, got {dtype}")
    return flag


def _raise(status, what):
    if status != TMAGEMM_OK:
        raise TmaGemmError(status, what)


class _Functions:
    """The library's functions, each looked up once (loading the library at the
    first use)."""

    def __getattr__(self, name):
        fn = getattr(lib(), name)
        setattr(self, name, fn)
        return fn


_fn = _Functions()


def quantize_fp8(X, block_rows: int = 1, stream=None):
    """Block quantisation of a CUDA fp16 or bf16 matrix X (M, K) -> (Q, S).

    Q is float8_e4m3fn (M, K); S is float32 (ceil(M / block_rows),
    ceil(K / 128)) with ``block_rows`` 1 (activations) or 128 (weights).  Row
    scales are laid out with consecutive rows next to each other, the layout
    the products read fastest; weight scales are row-major.
    """
    dev = _first("X", X, 2)
    bf16 = _bf16(X.dtype)
    if not X.is_contiguous():
        raise ValueError("X must be contiguous (row-major)")
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    M, K = X.shape
    blocks = _blocks(K)

    def body(handle):
        Q = _empty_like(X, dtype=_F8)
        if block_rows == 1:
            S = _empty_strided((M, blocks), (1, max(M, 1)), dtype=_F32, device=dev)
            strides = 1, max(M, 1)
        else:
            S = _empty((_blocks(M), blocks), dtype=_F32, device=dev)
            strides = max(blocks, 1), 1
        _raise(_fn.quantize_fp8(M, K, X.data_ptr(), bf16, block_rows, Q.data_ptr(),
                                  S.data_ptr(), *strides, handle), "quantize_fp8")
        return Q, S

    return _launch(dev, stream, (X,), body)


def _product(what, A, SA, B, SB, offsets, dtype, out, stream):
    """The checks, result and call that gemm_fp8 and gemm_fp8_grouped share;
    `offsets` None: dense."""
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    bf16 = _bf16(dtype)
    dev = _first("A", A, 2)
    M, K = A.shape
    *lead, N, _ = B.shape
    blocks = _blocks(K)
    _check("A", A, _F8, None, dev)
    _check("B", B, _F8, (*lead, N, K), dev)
    _check("SA", SA, _F32, (M, blocks), dev, contiguous=False)
    _check("SB", SB, _F32, (*lead, _blocks(N), blocks), dev)
    if out is not None:
        _check("out", out, dtype, (M, N), dev)
    # A stride that is never stepped (a dimension of one) counts as 1.
    # Broadcast (zero) strides are refused by the library.
    sa_row, sa_blk = SA.stride()
    if M <= 1:
        sa_row = 1
    if K <= FP8_BLOCK:
        sa_blk = 1

    def body(handle):
        D = _empty((M, N), dtype=dtype, device=dev) if out is None else out
        if offsets is None:
            status = _fn.gemm_fp8(M, N, K, A.data_ptr(), SA.data_ptr(), sa_row, sa_blk,
                                  B.data_ptr(), SB.data_ptr(), D.data_ptr(), bf16, handle)
        else:
            status = _fn.gemm_fp8_grouped(lead[0], offsets.data_ptr(), M, N, K, A.data_ptr(),
                                          SA.data_ptr(), sa_row, sa_blk, B.data_ptr(),
                                          SB.data_ptr(), D.data_ptr(), bf16, handle)
        if status:
            _raise(status, what)
        return D

    return _launch(dev, stream, (A, SA, B, SB, offsets, out), body)


def gemm_fp8(A, SA, B, SB, dtype=None, out=None, stream=None):
    """D (M, N) = (A * SA) @ (B * SB).T with block scales, in ``dtype`` (bf16 by
    default, or fp16).

    A (M, K) and B (N, K) are float8_e4m3fn; SA (M, ceil(K / 128)) float32 with
    any strides, SB (ceil(N / 128), ceil(K / 128)) float32, row-major.
    K % 16 == 0 and N % 8 == 0.
    """
    _first("B", B, 2)
    return _product("gemm_fp8", A, SA, B, SB, None, dtype, out, stream)


def gemm_fp8_grouped(A, SA, B, SB, m_offsets, dtype=None, out=None, stream=None):
    """Grouped D[rows of g] = (A * SA)[rows of g] @ (B[g] * SB[g]).T, where the
    rows of group g are m_offsets[g] .. m_offsets[g + 1] - 1.

    m_offsets is a CUDA int32 tensor (G + 1,), read by the kernel (no copy to
    the host); rows outside every group are left as they are in ``out``
    (undefined in a new result).  A (M, K), B (G, N, K), SB (G, ceil(N / 128),
    ceil(K / 128)); the rest as for gemm_fp8.
    """
    _first("B", B, 3)
    _check("m_offsets", m_offsets, torch.int32, (B.shape[0] + 1,), B.device)
    return _product("gemm_fp8_grouped", A, SA, B, SB, m_offsets, dtype, out, stream)


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
    dev = _first("h", h, 2)
    shape = T, C = h.shape
    dt = h.dtype
    bf16 = _bf16(dt)
    _check("h", h, dt, None, dev)
    if y is None and (w_pre is None or w_post is not None or gate is not None):
        raise ValueError("without y there is neither w_post nor gate, and w_pre is needed")
    mode = _GATE_NONE
    ptr = dict.fromkeys(("y", "w_post", "w_pre", "gate"))
    if y is not None:
        _check("y", y, dt, shape, dev)
        ptr["y"] = y.data_ptr()
    if w_post is not None:
        _check("w_post", w_post, dt, (C,), dev)
        ptr["w_post"] = w_post.data_ptr()
    if w_pre is not None:
        _check("w_pre", w_pre, dt, (C,), dev)
        ptr["w_pre"] = w_pre.data_ptr()
    if gate is not None:
        _check("gate", gate, dt, None, dev)
        if gate.shape == shape:
            mode = _GATE_ELEMENT
        elif gate.shape == (C,) or gate.shape == (1, C):
            mode = _GATE_CHANNEL
        elif gate.shape == (T, 1):
            mode = _GATE_TOKEN
        else:
            raise ValueError(f"gate must be (C,), (1, C), (T, 1) or (T, C), got "
                             f"{tuple(gate.shape)}")
        ptr["gate"] = gate.data_ptr()
    return TmagemmNorm(T, C, bf16, mode, alpha, eps, h.data_ptr(), ptr["y"], ptr["gate"],
                       ptr["w_post"], ptr["w_pre"])


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
    p = _norm_struct(h, y, gate, w_post, w_pre, alpha, eps)
    if quantize and w_pre is None:
        raise ValueError("quantize needs w_pre")
    T, C = h.shape
    dev = h.device

    def body(handle):
        h_out, x, scales, r_post, r_pre = h, None, None, None, None
        if y is not None:
            h_out = _empty_like(h)
            p.h_out = h_out.data_ptr()
        if w_pre is not None and quantize:
            x = _empty_like(h, dtype=_F8)
            scales = _empty_strided((T, _blocks(C)), (1, max(T, 1)), dtype=_F32, device=dev)
            p.q, p.scales, p.s_row_stride, p.s_block_stride = (
                x.data_ptr(), scales.data_ptr(), 1, max(T, 1))
        elif w_pre is not None:
            x = _empty_like(h)
            p.x = x.data_ptr()
        if save_rstd and w_post is not None:
            r_post = _empty((T,), dtype=_F32, device=dev)
            p.rstd_post = r_post.data_ptr()
        if save_rstd and w_pre is not None:
            r_pre = _empty((T,), dtype=_F32, device=dev)
            p.rstd_pre = r_pre.data_ptr()
        _raise(_fn.norm_residual(ctypes.byref(p), handle), "norm_residual")
        return NormOut(h_out, x, scales, r_post, r_pre)

    return _launch(dev, stream, (h, y, gate, w_post, w_pre), body)


def norm_residual_backward(h, y=None, dh=None, dx=None, gate=None, w_post=None, w_pre=None,
                           alpha: float = 1.0, rstd_post=None, rstd_pre=None,
                           stream=None) -> NormGrads:
    """Gradients of norm_residual from its inputs, its rsqrt factors
    (``save_rstd=True``) and the gradients of its results: dh of h' (None:
    zero) and dx of x (given if and only if w_pre is).

    dh, dy and a (T, C) gate's gradient have the type of h; the weights' and the
    other gates' gradients are float32 sums.
    """
    p = _norm_struct(h, y, gate, w_post, w_pre, alpha, 0.0)
    T, C = h.shape
    dt, dev = h.dtype, h.device
    if (dx is None) != (w_pre is None):
        raise ValueError("dx is given if and only if w_pre is")
    for name, field, t in (("dh", "dh_out", dh), ("dx", "dx", dx)):
        if t is not None:
            _check(name, t, dt, (T, C), dev)
            setattr(p, field, t.data_ptr())
    for name, t, w in (("rstd_post", rstd_post, w_post), ("rstd_pre", rstd_pre, w_pre)):
        if w is not None:
            _check(name, t, _F32, (T,), dev)
            setattr(p, name, t.data_ptr())

    def body(handle):
        dy = dgate = dw_post = dw_pre = None
        need = _fn.norm_residual_backward_workspace_size(T, C)
        if need < 0:
            raise TmaGemmError(int(need), "norm_residual_backward_workspace_size")
        workspace = _empty((need,), dtype=torch.uint8, device=dev)
        dh_in = _empty_like(h)
        p.dh = dh_in.data_ptr()
        if y is not None:
            dy = _empty_like(h)
            p.dy = dy.data_ptr()
        if gate is not None:
            dgate = _empty(gate.shape, device=dev,
                                dtype=dt if p.gate_mode == _GATE_ELEMENT else _F32)
            p.dgate = dgate.data_ptr()
        if w_post is not None:
            dw_post = _empty((C,), dtype=_F32, device=dev)
            p.dw_post = dw_post.data_ptr()
        if w_pre is not None:
            dw_pre = _empty((C,), dtype=_F32, device=dev)
            p.dw_pre = dw_pre.data_ptr()
        _raise(_fn.norm_residual_backward(ctypes.byref(p), workspace.data_ptr(), need, handle),
               "norm_residual_backward")
        return NormGrads(dh_in, dy, dgate, dw_post, dw_pre)

    return _launch(dev, stream, (h, y, dh, dx, gate, w_post, w_pre, rstd_post, rstd_pre), body)
