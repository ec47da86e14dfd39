"""GPU tests of the rules that split the work: products of few rows in one to eight
slices of K (whose partial sums meet in a cluster), and the norms' column sums for
narrow and wide rows, few and many.  References and bounds are those of
test_gpu_fp8.py and test_gpu_norm.py."""
import numpy as np
import pytest

from tests import fp8_reference as ref
from tests import test_gpu_fp8 as products
from tests import test_gpu_norm as norms

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.fixture(autouse=True)
def no_device_error(tg):
    yield
    tg.check()


# Tiles of 128 outputs, k-blocks -> slices, on 152 SMs.
SLICED = [(3, 2360, 432),      # 19, 4 -> 1
          (33, 14336, 1040),   # 112, 9 -> 2
          (12, 9664, 1584),    # 76, 13 -> 3
          (60, 8200, 2064),    # 65, 17 -> 4
          (5, 5088, 2656),     # 40, 21 -> 5
          (17, 5632, 3088),    # 44, 25 -> 6
          (9, 4864, 4112),     # 38, 33 -> 7
          (2, 520, 4304),      # 5, 34 -> 8
          (100, 14336, 272),   # 112 tiles of 128 tokens, 3 -> 1
          (128, 9000, 1040),   # 71, 9 -> 2
          (65, 3400, 2064),    # 27, 17 -> 4
          (128, 2568, 3344),   # 21, 27 -> 6
          (300, 640, 4112)]    # 15 of 384 rows, 33 -> 8


@pytest.mark.parametrize("M,N,K", SLICED)
def test_sliced_integers_are_exact(tg, M, N, K):
    rng = np.random.default_rng(M + N + K)
    a, sa = products.integer_operand(rng, M, K, True)
    b, sb = products.integer_operand(rng, N, K, False)
    want, _ = ref.gemm(a, sa, b, sb)
    cuda = lambda s: torch.from_numpy(s).cuda()  # noqa: E731
    got = tg.gemm_fp8(products.f8(a), cuda(sa), products.f8(b), cuda(sb), dtype=torch.float16)
    assert np.array_equal(got.double().cpu().numpy(), products.rounded(want, torch.float16))


@pytest.mark.parametrize("M,N,K", SLICED)
def test_sliced_parity_and_bits(tg, M, N, K):
    rng = np.random.default_rng(M * N + K)
    a, sa = products.random_operand(rng, M, K, True)
    b, sb = products.random_operand(rng, N, K, False)
    cuda = lambda s: torch.from_numpy(s).cuda()  # noqa: E731
    args = (products.f8(a), cuda(sa), products.f8(b), cuda(sb))
    got = tg.gemm_fp8(*args)
    products.check_product(got, a, sa, b, sb, True)
    for _ in range(3):
        assert torch.equal(tg.gemm_fp8(*args).view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("T,C", [(2500, 264), (1293, 880), (520, 2440), (330, 5008), (900, 8192)])
@pytest.mark.parametrize("gate,post,pre", [("token", True, True), ("channel", True, True),
                                           (None, False, True)])
def test_norm_column_sums(tg, T, C, gate, post, pre):
    norms.test_forward_and_gradients(tg, T, C, "bf16", gate, post, pre)


# One to eight slices whatever the device holds of the larger clusters: few tiles, and
# four to 32 k-blocks and some more.
@pytest.mark.parametrize("M", [9, 40, 100])
@pytest.mark.parametrize("K,slices", [(880, 1), (912, 2), (1104, 2), (1552, 3), (2320, 4), (2800, 5),
                                      (3216, 6), (3600, 7), (4240, 8)])
def test_every_slice_count(tg, M, K, slices):
    N = 520
    plan = tg.tmagemm_gemm_fp8_few_rows_plan(M, N, K, 152, [5] * 7)
    assert (plan["tiles"], plan["slices"]) == (5, slices)
    rng = np.random.default_rng(M + K)
    a, sa = products.integer_operand(rng, M, K, True)
    b, sb = products.integer_operand(rng, N, K, False)
    want, _ = ref.gemm(a, sa, b, sb)
    cuda = lambda s: torch.from_numpy(s).cuda()  # noqa: E731
    got = tg.gemm_fp8(products.f8(a), cuda(sa), products.f8(b), cuda(sb), dtype=torch.float16)
    assert np.array_equal(got.double().cpu().numpy(), products.rounded(want, torch.float16))


def test_first_call_inside_a_capture(tg):
    """What is asked of the device once (how many clusters it holds) may be asked while
    a graph is captured, in a process that has not called the product before."""
    import os
    import subprocess
    import sys
    code = """
import torch
import tma_pipelined_tensor_tn_gb300 as tg
A = torch.full((9, 528), 0x38, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
B = torch.full((264, 528), 0x38, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
SA, SB = torch.ones((9, 5), device="cuda"), torch.ones((3, 5), device="cuda")
out = torch.zeros((9, 264), device="cuda", dtype=torch.float16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    tg.gemm_fp8(A, SA, B, SB, out=out)
graph.replay()
tg.check()
assert torch.all(out == 528)     # 0x38 is 1
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
