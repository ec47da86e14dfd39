"""The router's operators together, as a layer of experts uses them: forward and backward
as an autograd.Function of the caller's would, and with 4-bit weights as in decoding."""
import numpy as np
import pytest

from tests import experts_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.mark.parametrize("T,E,k,C,score,renormalize", [
    (3, 8, 2, 264, "softmax", True), (200, 12, 4, 136, "sigmoid", True),
    (900, 64, 6, 128, "softmax", False)])
def test_layer_and_its_gradients(tg, T, E, k, C, score, renormalize):
    """logits -> weights, x -> rows -> rows * a[expert] -> y: the gradients of x and the
    logits that the calls chain to, against 64-bit autograd of the plain layer.  Rounding:
    each of rows * a, y, drows, dx is rounded to fp16 (2^-11 of itself) and the others are
    FP32; a sum of k terms of size s is off by (k + 4) 2^-11 s at most."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, C), generator=g).half().cuda()
    logits = torch.randn((T, E), generator=g).cuda()
    a = (1 + torch.rand((E, 1), generator=g)).half().cuda()
    dy = torch.randn((T, C), generator=g).half().cuda()

    ids, w = tg.route_topk(logits, k, score=score, renormalize=renormalize)
    r = tg.dispatch_rows(x, ids, E)
    expert = torch.empty(T * k, dtype=torch.long, device="cuda")
    expert[r.row_of.flatten().long()] = ids.flatten().long()
    out = (r.rows.float() * a[expert].float()).half()
    y = tg.combine_rows(out, r.row_of, w)
    d = tg.combine_rows_backward(dy, out, r.row_of, w)
    dx = tg.combine_rows((d.drows.float() * a[expert].float()).half(), r.row_of)
    dl = tg.route_topk_backward(logits, ids, d.dweights, score=score, renormalize=renormalize)
    tg.check()

    x64, l64 = x.double().requires_grad_(), logits.double().requires_grad_()
    p = torch.softmax(l64, 1) if score == "softmax" else torch.sigmoid(l64)
    c = p.gather(1, ids.long())
    w64 = c / c.sum(1, keepdim=True) if renormalize else c
    f = w64 * a.double()[ids.long(), 0]
    y64 = f.sum(1, keepdim=True) * x64
    (y64 * dy.double()).sum().backward()
    step = (k + 4) * 2.0 ** -11
    size = f.detach().abs().sum(1, keepdim=True)
    tiny = 2.0 ** -20
    assert torch.all((y.double() - y64).abs() <= step * size * x.double().abs() + tiny)
    assert torch.all((dx.double() - x64.grad).abs() <= step * size * dy.double().abs() + tiny)
    # d loss / d w is a sum over columns of dy out: its error, through the (at most unit)
    # derivatives of the weights, twice (the chosen score's own and the normalisation's)
    dw = (dy.double().abs() * x.double().abs()).sum(1, keepdim=True) * 2.0 * 2.0 ** -11
    assert torch.all((dl.double() - l64.grad).abs() <= 2 * 2 * dw + tiny)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_decoding_with_4_bit_experts(tg, T):
    """route, dispatch, a 4-bit product by expert, combine; padded tokens have no choice."""
    E, k, C, N, group = 16, 3, 544, 264, 64
    rng = np.random.default_rng(T)
    codes = rng.integers(0, 256, (E, N, C // 2)).astype(np.uint8)
    kg = -(-C // group)
    s = torch.from_numpy(rng.normal(size=(E, N, kg)) * 0.05).bfloat16()
    z = rng.integers(0, 16, (E, N, kg)).astype(np.uint8)
    x = torch.from_numpy(rng.normal(size=(T, C))).bfloat16()
    logits = torch.from_numpy(rng.normal(size=(T, E))).float()
    logits[T // 2 + 1:] = -float("inf")                 # padding
    ids, w = tg.route_topk(logits.cuda(), k)
    r = tg.dispatch_rows(x.cuda(), ids, E)
    out = tg.gemm_w4_grouped(r.rows, torch.from_numpy(codes).cuda(), s.cuda(), r.offsets,
                             torch.from_numpy(z).cuda(), group=group)
    y = tg.combine_rows(out, r.row_of, w).double().cpu().numpy()
    tg.check()
    want_ids, want_w = ref.route(logits.double().numpy(), k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    for t in range(T):
        total, bound = np.zeros(N), np.zeros(N)
        for j in range(k):
            e = want_ids[t, j]
            if e < 0:
                continue
            m = ref.weights_w4(codes[e], s[e].double().numpy(), z[e], group)
            d = m @ x[t].double().numpy()
            size = np.abs(m) @ np.abs(x[t].double().numpy())
            total += want_w[t, j] * d
            # the product's own bound, and the weight's and the sum's FP32 roundings
            bound += want_w[t, j] * (ref.w4_bound(d, size, C, group, True) + 2.0 ** -18 * np.abs(d))
        assert np.all(np.abs(y[t] - total) <= bound + 2.0 ** -8 * (np.abs(total) + bound))


def test_calls_on_two_streams_at_once(tg):
    """Calls that overlap on the GPU, of the same and of other operators, as one by one."""
    g = torch.Generator(device="cuda").manual_seed(2)
    T, E, k, C, N = 3000, 16, 4, 512, 1000
    x = torch.randn((2, T, C), device="cuda", generator=g).half()
    logits = torch.randn((2, T, E), device="cuda", generator=g)
    B = torch.randint(0, 256, (E, N, C // 2), device="cuda", generator=g).to(torch.uint8)
    S = torch.rand((E, N, C // 64), device="cuda", generator=g).half()

    def layer(i, few):
        n = 40 if few else T
        ids, w = tg.route_topk(logits[i, :n], k)
        r = tg.dispatch_rows(x[i, :n], ids, E)
        out = tg.gemm_w4_grouped(r.rows, B, S, r.offsets, group=64)
        return tg.combine_rows(out, r.row_of, w), tg.gemm_w4(x[i, :9 if few else 3], B[i], S[i],
                                                             group=64)

    want = [[layer(i, few) for few in (False, True)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append([layer(i, few) for few in (False, True)])
    torch.cuda.synchronize()
    tg.check()
    for i in range(2):
        for once in got[i]:
            for (y, d), (y0, d0) in zip(once, want[i]):
                assert torch.equal(y, y0) and torch.equal(d, d0)


def test_first_calls_inside_a_capture(tg, tmp_path):
    """What the kernels ask of the device once is asked while a graph is captured."""
    import subprocess
    import sys
    code = """
import torch, tma_pipelined_tensor_tn_gb300 as tg
x = torch.randn((20, 512), device="cuda").half()
B = torch.randint(0, 256, (300, 256), dtype=torch.uint8, device="cuda")
S = torch.rand((300, 4), device="cuda").half()
l = torch.randn((20, 8), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    r = tg.route_topk(l, 2)
    d = tg.dispatch_rows(x, r.ids, 8)
    y = tg.combine_rows(d.rows, d.row_of, r.weights)
    D = [tg.gemm_w4(x[:m], B, S) for m in (1, 12, 20)]
g.replay()
torch.cuda.synchronize()
r2 = tg.route_topk(l, 2)
assert torch.equal(r.ids, r2.ids) and torch.equal(r.weights, r2.weights)
for m, got in zip((1, 12, 20), D):
    assert torch.equal(got, tg.gemm_w4(x[:m], B, S))
tg.check()
print("fine")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
