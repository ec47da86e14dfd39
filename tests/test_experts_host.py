"""Host-side tests of the router, the rows of experts and the 4-bit products: refusals
before any CUDA call, the binding's argument checks, the argument struct's layout."""
import ctypes
import os
import shutil
import subprocess

import pytest

import tma_pipelined_tensor_tn_gb300 as tg
from tma_pipelined_tensor_tn_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an aligned address that no refused call may touch
OK, INVALID, ALIGN, UNSUPPORTED, WORKSPACE = (
    tg.TMAGEMM_OK, tg.TMAGEMM_ERR_INVALID, tg.TMAGEMM_ERR_ALIGN, tg.TMAGEMM_ERR_UNSUPPORTED,
    tg.TMAGEMM_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    return tg.lib()


def route_struct(**fields):
    p = tg.TmagemmRoute()
    for k, v in {**dict(T=4, E=64, k=6, type=2, groups=1, top_groups=1, scale=1.0, logits=P, ids=P,
                        weights=P, dweights=P, dlogits=P), **fields}.items():
        setattr(p, k, v)
    return p


COMMON = [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(type=3), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(E=513), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(logits=P + 2), ALIGN),
    (dict(type=1, logits=P + 1), ALIGN), (dict(ids=P + 2), ALIGN),
    (dict(T=0, logits=None, ids=None, weights=None, dweights=None, dlogits=None), OK),
]


@pytest.mark.parametrize("fields,expect", COMMON + [
    (dict(weights=None), INVALID), (dict(weights=P + 1), ALIGN), (dict(bias=P + 2), ALIGN),
    (dict(groups=0), INVALID), (dict(groups=5), INVALID), (dict(groups=8, top_groups=0), INVALID),
    (dict(groups=8, top_groups=9, group_sum=1), INVALID),
    (dict(groups=8, top_groups=2, group_sum=0), INVALID),
    (dict(groups=8, top_groups=2, group_sum=3), INVALID), (dict(top_groups=2), INVALID),
    (dict(groups=32, top_groups=2, group_sum=1), INVALID),     # 4 experts for a choice of 6
    (dict(groups=64, top_groups=8, group_sum=1), UNSUPPORTED)])
def test_route_refusals(fields, expect):
    assert tg.lib().route_topk(ctypes.byref(route_struct(**fields)), None) == expect
    assert tg.lib().route_topk(None, None) == INVALID


@pytest.mark.parametrize("fields,expect", COMMON + [
    (dict(dweights=None), INVALID), (dict(dlogits=None), INVALID), (dict(dweights=P + 2), ALIGN),
    (dict(dlogits=P + 2), ALIGN)])
def test_route_backward_refusals(fields, expect):
    p = route_struct(**fields)
    p.groups = p.top_groups = 0         # not read
    assert tg.lib().route_topk_backward(ctypes.byref(p), None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(C=0), INVALID),
    (dict(ids=None), INVALID), (dict(x=None), INVALID), (dict(rows=None), INVALID),
    (dict(offsets=None), INVALID), (dict(row_of=None), INVALID),
    (dict(scales=P, s_row=0), INVALID), (dict(scales=P, s_blk=-1), INVALID),
    (dict(k=33), UNSUPPORTED), (dict(E=513), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(C=(1 << 20) + 8), UNSUPPORTED), (dict(C=260), ALIGN), (dict(x=P + 8), ALIGN),
    (dict(rows=P + 2), ALIGN), (dict(ids=P + 2), ALIGN), (dict(scales=P + 1), ALIGN),
    (dict(offsets=P + 2), ALIGN), (dict(row_of=P + 1), ALIGN)])
def test_dispatch_refusals(change, expect):
    a = dict(T=4, k=2, E=8, C=256, ids=P, x=P, bf16=1, rows=P, scales=None, s_row=1, s_blk=8,
             offsets=P, row_of=P, workspace=P, bytes=1 << 30)
    a.update(change)
    assert tg.lib().dispatch_rows(*a.values(), None) == expect


def test_dispatch_workspace():
    size = tg.lib().dispatch_rows_workspace_size
    assert size(0, 4, 8) == 0
    assert size(-1, 4, 8) == INVALID and size(1, 0, 8) == INVALID and size(1, 4, 0) == INVALID
    assert size(1, 4, 513) == UNSUPPORTED and size(1 << 30, 2, 8) == UNSUPPORTED
    need = size(1 << 17, 8, 512)
    assert need > 0
    args = [1 << 17, 8, 512, 256, P, P, 1, P, None, 1, 1, P, P]
    for workspace, given in ((None, need), (P + 8, need), (P, need - 1)):
        assert tg.lib().dispatch_rows(*args, workspace, given, None) == WORKSPACE


COMBINE = [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(C=-8), INVALID), (dict(R=-1), INVALID),
    (dict(rows=None), INVALID), (dict(row_of=None), INVALID), (dict(k=33), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED), (dict(R=1 << 31), UNSUPPORTED),
    (dict(C=(1 << 20) + 8), UNSUPPORTED), (dict(C=12), ALIGN), (dict(rows=P + 8), ALIGN),
    (dict(row_of=P + 2), ALIGN), (dict(weights=P + 2), ALIGN)]


@pytest.mark.parametrize("change,expect", COMBINE + [
    (dict(y=None), INVALID), (dict(y=P + 2), ALIGN),
    (dict(T=0, rows=None, row_of=None, weights=None, y=None), OK)])
def test_combine_refusals(change, expect):
    a = {**dict(T=4, k=2, C=256, R=8, rows=P, row_of=P, weights=P, y=P, bf16=0), **change}
    assert tg.lib().combine_rows(*a.values(), None) == expect


@pytest.mark.parametrize("change,expect", COMBINE + [
    (dict(dy=None), INVALID), (dict(weights=None), INVALID), (dict(drows=None), INVALID),
    (dict(dweights=None), INVALID), (dict(dy=P + 8), ALIGN), (dict(drows=P + 4), ALIGN),
    (dict(dweights=P + 2), ALIGN),
    (dict(T=0, rows=None, row_of=None, weights=None, dy=None, drows=None, dweights=None), OK)])
def test_combine_backward_refusals(change, expect):
    a = {**dict(T=4, k=2, C=256, R=8, dy=P, rows=P, row_of=P, weights=P, drows=P, dweights=P,
                bf16=0), **change}
    assert tg.lib().combine_rows_backward(*a.values(), None) == expect


W4 = dict(M=4, N=100, K=256, group=64, A=P, B=P, SB=P, ZB=None, D=P, bf16=1)
W4_REFUSALS = [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(group=0), INVALID),
    (dict(group=256), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(SB=None), INVALID), (dict(D=None), INVALID), (dict(M=1 << 31), UNSUPPORTED),
    (dict(N=1 << 31), UNSUPPORTED), (dict(K=272), ALIGN), (dict(A=P + 8), ALIGN),
    (dict(B=P + 8), ALIGN), (dict(SB=P + 1), ALIGN), (dict(D=P + 1), ALIGN),
    (dict(M=(1 << 31) - 255), UNSUPPORTED), (dict(K=(1 << 26) + 32), UNSUPPORTED),
    (dict(M=1 << 22, N=1 << 20), UNSUPPORTED), (dict(M=0, A=None, D=None), OK)]


@pytest.mark.parametrize("change,expect", W4_REFUSALS)
def test_w4_refusals(change, expect):
    assert tg.lib().gemm_w4(*{**W4, **change}.values(), None) == expect


@pytest.mark.parametrize("change,expect", W4_REFUSALS + [
    (dict(G=0), INVALID), (dict(offsets=None), INVALID), (dict(G=385), UNSUPPORTED),
    (dict(offsets=P + 2), ALIGN), (dict(G=300, N=1 << 23), UNSUPPORTED)])
def test_w4_grouped_refusals(change, expect):
    a = {**dict(G=3, offsets=P), **W4, **change}
    assert tg.lib().gemm_w4_grouped(*a.values(), None) == expect


def test_route_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("gcc not available")
    names = [n for n, _ in tg.TmagemmRoute._fields_]
    body = "".join(f'printf("%zu\\n", offsetof(tmagemm_route, {n}));' for n in names)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "tmagemm.h"\n'
                   f'int main(void) {{ {body} printf("%zu\\n", sizeof(tmagemm_route)); return 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [getattr(tg.TmagemmRoute, n).offset for n in names] + [ctypes.sizeof(tg.TmagemmRoute)]
    assert got == want


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    logits, ids = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    x, w = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((4, 2))
    q, s = torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.bfloat16)
    for call in (lambda: tg.route_topk(logits, 2), lambda: tg.route_topk_backward(logits, ids, w),
                 lambda: tg.dispatch_rows(x, ids, 8), lambda: tg.combine_rows(x, ids, w),
                 lambda: tg.combine_rows_backward(x, x, ids, w), lambda: tg.gemm_w4(x, q, s),
                 lambda: tg.gemm_w4_grouped(x, q[None], s[None],
                                            torch.zeros(2, dtype=torch.int32)),
                 lambda: tg.gemm_w4_grouped(x, q[None], s[None], None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        tg.route_topk(logits, 2, score="relu")


@pytest.mark.parametrize("source", ["gemm_w4.cu", "gemm_w4_many.cu"])
def test_aligned_barriers_follow_a_reconvergence(source):
    """bar.sync, bar.red and barrier.cluster.*.aligned need the lanes of a warp together:
    right before each the warp is brought together."""
    with open(os.path.join(_build.CSRC, source), encoding="utf-8") as f:
        code = [line.split("//")[0].strip() for line in f]
    code = [line for line in code if line]
    at = [i for i, line in enumerate(code) if "cluster_sync" in line or "named_bar_" in line]
    assert at
    for i in at:
        before = code[i - 3:i]
        assert any("__syncwarp()" in b or "__syncthreads()" in b for b in before), code[i - 3:i + 1]
