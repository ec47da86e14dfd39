"""Host-side tests of the 8-bit operators and the norms: refusals before any
CUDA call, the binding's argument checks, the argument struct's layout."""
import ctypes
import os
import shutil
import subprocess

import pytest

import tma_pipelined_tensor_tn_gb300 as tg
from tma_pipelined_tensor_tn_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an aligned address that no refused call may touch
OK, INVALID, ALIGN, UNSUPPORTED = (tg.TMAGEMM_OK, tg.TMAGEMM_ERR_INVALID, tg.TMAGEMM_ERR_ALIGN,
                                   tg.TMAGEMM_ERR_UNSUPPORTED)


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    return tg.lib()


@pytest.mark.parametrize("change,expect", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID),
    (dict(S=None), INVALID), (dict(block_rows=64), INVALID), (dict(s_row=0), INVALID),
    (dict(s_blk=-1), INVALID), (dict(K=260), ALIGN), (dict(X=P + 2), ALIGN), (dict(Q=P + 8), ALIGN),
    (dict(S=P + 2), ALIGN), (dict(M=1 << 31), UNSUPPORTED), (dict(M=0, X=None, Q=None, S=None), OK),
])
def test_quantize_refusals(change, expect):
    a = dict(M=4, K=256, X=P, bf16=1, block_rows=1, Q=P, S=P, s_row=1, s_blk=4)
    a.update(change)
    assert tg.lib().quantize_fp8(*a.values(), None) == expect


GEMM = dict(M=4, N=128, K=256, A=P, SA=P, sa_row=1, sa_blk=4, B=P, SB=P, D=P, bf16=1)
GEMM_REFUSALS = [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID), (dict(A=None), INVALID),
    (dict(SA=None), INVALID), (dict(B=None), INVALID), (dict(SB=None), INVALID),
    (dict(D=None), INVALID), (dict(sa_row=0), INVALID), (dict(sa_blk=0), INVALID),
    (dict(K=264), ALIGN), (dict(N=100), ALIGN), (dict(A=P + 8), ALIGN), (dict(B=P + 4), ALIGN),
    (dict(D=P + 2), ALIGN), (dict(SA=P + 1), ALIGN), (dict(SB=P + 2), ALIGN),
    (dict(M=1 << 31), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED),
    (dict(M=0, A=None, SA=None, D=None), OK),
]


@pytest.mark.parametrize("change,expect", GEMM_REFUSALS)
def test_gemm_refusals(change, expect):
    assert tg.lib().gemm_fp8(*{**GEMM, **change}.values(), None) == expect


@pytest.mark.parametrize("change,expect", GEMM_REFUSALS + [
    (dict(G=0), INVALID), (dict(offsets=None), INVALID), (dict(G=385), UNSUPPORTED),
    (dict(offsets=P + 2), ALIGN), (dict(G=300, N=1 << 23), UNSUPPORTED)])
def test_grouped_refusals(change, expect):
    a = {**dict(G=3, offsets=P), **GEMM, **change}
    assert tg.lib().gemm_fp8_grouped(*a.values(), None) == expect


def test_grouped_rows_whose_tiles_pass_32_bits_are_refused():
    """A group of more than 2^31 - 256 rows has a last tile that ends past 2^31."""
    a = {**dict(G=3, offsets=P), **GEMM, "N": 8, "K": 16}
    for M in ((1 << 31) - 255, (1 << 31) - 1):
        assert tg.lib().gemm_fp8_grouped(*{**a, "M": M}.values(), None) == UNSUPPORTED


def norm_struct(**fields):
    p = tg.TmagemmNorm()
    for k, v in {**dict(T=4, C=256, alpha=1.0, eps=1e-6, h=P), **fields}.items():
        setattr(p, k, v)
    return p


FORWARD = dict(y=P, w_post=P, w_pre=P, h_out=P, x=P)


@pytest.mark.parametrize("fields,expect", [
    (dict(T=-1), INVALID), (dict(C=0), INVALID), (dict(h=None), INVALID), (dict(gate_mode=4), INVALID),
    (dict(gate_mode=1), INVALID), (dict(gate_mode=-1), INVALID),
    (dict(y=None, w_post=None, w_pre=None), INVALID), (dict(y=None), INVALID),
    (dict(y=None, w_post=None, gate_mode=1, gate=P), INVALID), (dict(h_out=None), INVALID),
    (dict(x=None), INVALID), (dict(x=None, q=P, scales=P), INVALID),
    (dict(x=None, q=P, scales=P, s_row_stride=1), INVALID),
    (dict(C=260), ALIGN), (dict(h=P + 2), ALIGN), (dict(y=P + 8), ALIGN), (dict(w_pre=P + 2), ALIGN),
    (dict(gate_mode=1, gate=P + 2), ALIGN), (dict(gate_mode=2, gate=P + 1), ALIGN),
    (dict(x=P + 8), ALIGN), (dict(rstd_pre=P + 2), ALIGN), (dict(C=16392), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=0, h=None, h_out=None, x=None), OK),
])
def test_norm_forward_refusals(fields, expect):
    p = norm_struct(**{**FORWARD, **fields})
    assert tg.lib().norm_residual(ctypes.byref(p), None) == expect
    assert tg.lib().norm_residual(None, None) == INVALID


BACKWARD = dict(y=P, w_post=P, w_pre=P, rstd_post=P, rstd_pre=P, dh_out=P, dx=P, dh=P, dy=P,
                dw_post=P, dw_pre=P)


@pytest.mark.parametrize("fields,expect", [
    (dict(dx=None), INVALID), (dict(w_pre=None), INVALID), (dict(dw_post=None), INVALID),
    (dict(dw_pre=None), INVALID), (dict(dh=None), INVALID), (dict(dy=None), INVALID),
    (dict(rstd_post=None), INVALID), (dict(rstd_pre=None), INVALID),
    (dict(gate_mode=2, gate=P), INVALID), (dict(dh=P + 2), ALIGN), (dict(dw_pre=P + 2), ALIGN),
    (dict(gate_mode=3, gate=P, dgate=P + 8), ALIGN), (dict(gate_mode=1, gate=P, dgate=P + 2), ALIGN),
])
def test_norm_backward_refusals(fields, expect):
    p = norm_struct(**{**BACKWARD, **fields})
    assert tg.lib().norm_residual_backward(ctypes.byref(p), P, 1 << 30, None) == expect


def test_norm_of_no_rows_needs_its_channel_gate():
    """A per-channel gate has no rows, so it is needed with T = 0 too: the column sums
    would read it."""
    p = norm_struct(**{**BACKWARD, "T": 0}, gate_mode=1, dgate=P)
    assert tg.lib().norm_residual_backward(ctypes.byref(p), None, 0, None) == INVALID
    assert tg.lib().norm_residual(ctypes.byref(p), None) == INVALID
    p.gate = P
    assert tg.lib().norm_residual_backward(ctypes.byref(p), None, 0, None) != INVALID
    p.dgate = None
    assert tg.lib().norm_residual_backward(ctypes.byref(p), None, 0, None) == INVALID


@pytest.mark.parametrize("gate_mode", [2, 3])
def test_norm_backward_of_no_rows_needs_no_gate_gradient_per_row(gate_mode):
    """With T = 0 a per-token or per-element gate and its gradient are empty (NULL):
    the call is valid (and fails here only for want of a device)."""
    p = norm_struct(T=0, h=None, y=None, gate_mode=gate_mode)
    assert tg.lib().norm_residual_backward(ctypes.byref(p), None, 0, None) != INVALID


def test_norm_workspace_refusals():
    f = tg.lib().norm_residual_backward_workspace_size
    assert f(-1, 256) == INVALID and f(4, 0) == INVALID and f(4, 16392) == UNSUPPORTED
    assert f(0, 256) == 0


def test_norm_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("gcc not available")
    names = [n for n, _ in tg.TmagemmNorm._fields_]
    body = "".join(f'printf("%zu\\n", offsetof(tmagemm_norm, {n}));' for n in names)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "tmagemm.h"\n'
                   f'int main(void) {{ {body} printf("%zu\\n", sizeof(tmagemm_norm)); return 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [getattr(tg.TmagemmNorm, n).offset for n in names] + [ctypes.sizeof(tg.TmagemmNorm)]
    assert got == want


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q = torch.zeros((4, 256), dtype=torch.float8_e4m3fn)
    s = torch.zeros((4, 2))
    with pytest.raises(TypeError):
        tg.quantize_fp8(x)
    with pytest.raises(TypeError):
        tg.gemm_fp8(q, s, q, s)
    with pytest.raises(TypeError):
        tg.gemm_fp8_grouped(q, s, q[None], s[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        tg.norm_residual(x, x)


# Clusters of 2, 3, .. 8 CTAs that a GB300 with 152 SMs was seen to hold: of the
# kernels for up to 64 tokens, two CTAs an SM, and of the one for 128.
HELD = (152, 97, 74, 58, 46, 38, 36)
HELD_128 = (76, 46, 36, 28, 23, 15, 15)


@pytest.mark.parametrize("M,N,K,tokens,tiles,slices", [
    (3, 2360, 432, 16, 19, 1), (33, 14336, 1040, 64, 112, 2), (12, 9664, 1584, 16, 76, 3),
    (60, 8200, 2064, 64, 65, 4), (5, 5088, 2656, 16, 40, 5), (17, 5632, 3088, 32, 44, 6),
    (9, 4864, 4112, 16, 38, 7), (2, 520, 4304, 16, 5, 8),                 # the largest that fit
    (1, 4864, 14336, 16, 38, 7), (1, 4992, 14336, 16, 39, 6), (12, 9728, 5632, 16, 76, 3),
    (1, 4096, 14336, 16, 32, 8), (9, 520, 3600, 16, 5, 7),                # 29 k-blocks
    (100, 14336, 272, 128, 112, 1), (128, 9000, 1040, 128, 71, 2), (65, 3400, 2064, 128, 27, 4),
    (128, 2568, 3344, 128, 21, 6), (300, 640, 4112, 128, 15, 8), (129, 8192, 1024, 0, 0, 0)])
def test_slices_of_few_rows(M, N, K, tokens, tiles, slices):
    held = HELD_128 if M > 64 else HELD
    assert tg.tmagemm_gemm_fp8_few_rows_plan(M, N, K, 152, held) == {
        "tokens": tokens, "tiles": tiles, "slices": slices}


def test_slices_of_few_rows_follow_the_device():
    plan = tg.tmagemm_gemm_fp8_few_rows_plan
    assert plan(1, 4864, 14336, 152, [0] * 7)["slices"] == 1
    assert plan(1, 4864, 14336, 152, [100, 38, 37, 0, 0, 0, 0])["slices"] == 3
    with pytest.raises(tg.TmaGemmError):
        plan(0, 128, 128, 152, HELD)


@pytest.mark.parametrize("source", ["few_rows_fp8.cu", "gemm_fp8.cu"])
def test_aligned_barriers_follow_a_reconvergence(source):
    """barrier.cluster.*.aligned and bar.red need the lanes of a warp together: right
    before each, whatever per-lane branches came earlier, the warp is brought together."""
    with open(os.path.join(_build.CSRC, source), encoding="utf-8") as f:
        code = [line.split("//")[0].strip() for line in f]
    code = [line for line in code if line]
    at = [i for i, line in enumerate(code) if "cluster_sync" in line or "named_bar_and(" in line]
    assert at
    for i in at:
        before = code[i - 3:i]
        assert any("__syncwarp()" in b or "__syncthreads()" in b for b in before), code[i - 3:i + 1]
