"""GPU tests of the router's operators and the 4-bit products just past the sizes from which
other kernels, or other ways through them, are chosen: sizes that prompts and training have.
They are derived from the SM count, as the choices are.  Bounds as in test_gpu_route.py,
test_gpu_dispatch.py and test_gpu_w4.py."""
import numpy as np
import pytest

from tests import experts_reference as ref
from tests import test_gpu_dispatch as rows_tests
from tests import test_gpu_route as route_tests
from tests import test_gpu_w4 as w4_tests

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.fixture(scope="module")
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# -------------------------------------------------------------------- rows ----

@pytest.mark.parametrize("columns,pieces", [(1032, 2), (1160, 2), (2056, 3), (1016, 1)])
@pytest.mark.parametrize("name,quantize", [("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("kind", ["some", "padded"])
def test_wide_pieces_of_rows(tg, sms, columns, pieces, name, quantize, kind):
    """1024 columns to a warp, from 16 pieces an SM on: the last piece whole, or a part."""
    T = -(-16 * sms // pieces) + 5
    rows_tests.test_rows_by_expert(tg, T, 3, 37, columns, kind, name, quantize)


@pytest.mark.parametrize("T,k,columns", [(256, 1, 4104), (128, 2, 8192), (32, 8, 65536 + 8)])
@pytest.mark.parametrize("name,quantize", [("f16", False), ("bf16", True)])
def test_few_slots_of_many_columns(tg, T, k, columns, name, quantize):
    """The kernel that places and copies in one, with more pieces than warps."""
    rows_tests.test_rows_by_expert(tg, T, k, 19, columns, "padded", name, quantize)


@pytest.mark.parametrize("columns,pieces", [(264, 1), (512, 1), (776, 2)])
@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
def test_sums_of_one_or_two_rows(tg, sms, columns, pieces, k, name, weighted):
    """512 columns to a warp, from 32 pieces an SM on."""
    for kind in ("some", "padded"):
        rows_tests.test_combine_and_gradients(tg, 32 * sms // pieces + 9, k, 11, columns, kind, name,
                                              weighted)


@pytest.mark.parametrize("k,columns", [(2, 264), (3, 776)])
def test_sums_with_several_pieces_a_warp(tg, sms, k, columns):
    rows_tests.test_combine_and_gradients(tg, 150 * sms, k, 11, columns, "padded", "bf16", True)


# ------------------------------------------------------------------ router ----

@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("score,kw", [
    ("softmax", {}), ("sigmoid", dict(renormalize=False)),
    ("sigmoid", dict(groups=4, top_groups=2, group_sum=2)),
    ("softmax", dict(renormalize=False, groups=4, top_groups=3, group_sum=2))])
def test_warps_with_several_tokens(tg, sms, name, score, kw):
    """More tokens than the forward's warps; biases that leave few and many candidates, and
    doubts that are settled in 64 bits, one token after the other in the same memory."""
    T, E, k = 100 * sms, 40, 5
    logits = route_tests.make(T, E, name)
    logits[::3] = torch.round(logits[::3])              # ties
    logits[1::5, 4:] = -float("inf")                    # fewer than k experts
    bias = torch.round(torch.linspace(-1, 1, E) * 4).cuda() / 8 if "groups" in kw else None
    route_tests.check(tg, logits, k, score=score, bias=bias, gradient=False, **kw)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("sigmoid", True)])
def test_gradients_of_warps_with_several_tokens(tg, sms, name, score, renormalize):
    logits = route_tests.make(150 * sms, 23, name)
    logits[::7, 2:] = -float("inf")
    route_tests.check(tg, logits, 4, score=score, renormalize=renormalize)


# ---------------------------------------------------------- 4-bit products ----

@pytest.mark.parametrize("group,zeros,name", [(128, True, "bf16"), (32, False, "f16")])
def test_several_units_of_a_cluster(tg, group, zeros, name):
    """160 units of a long K: more than the clusters that the device holds, each of which
    adds up the sums of one unit after the other."""
    M, N, K = 500, 1280, 8224
    rng = np.random.default_rng(M)
    codes, s, z = w4_tests.weights(rng, N, K, group, zeros, name)
    a = torch.from_numpy(rng.normal(size=(M, K))).to(w4_tests.TYPES[name]).cuda()
    d = tg.gemm_w4(a, *w4_tests.gpu(codes, s, z), group=group)
    w4_tests.check(d, a, codes, s, z, group, name)
    tg.check()


@pytest.mark.parametrize("M", [1, 4, 8])
@pytest.mark.parametrize("blocks,K", [(0.5, 800), (0.5, 768), (0.55, 768), (0.55, 800), (2, 544),
                                      (2.01, 544), (2.01, 96)])
def test_few_tokens_where_the_kernels_change_over(tg, sms, M, blocks, K):
    """Blocks of 128 rows around half an SM and two an SM, K around 768."""
    N = 128 * int(blocks * sms + 0.99) - 3
    rng = np.random.default_rng(M)
    codes, s, z = w4_tests.weights(rng, N, K, 128, True, "bf16")
    a = torch.from_numpy(rng.normal(size=(M, K))).bfloat16().cuda()
    d = tg.gemm_w4(a, *w4_tests.gpu(codes, s, z))
    w4_tests.check(d, a, codes, s, z, 128, "bf16")
    tg.check()


@pytest.mark.parametrize("group", [64, 128])
def test_weights_past_32_bit_offsets_in_both_kernels(tg, group):
    """Codes of more than 2^32 bytes: the last rows against a product of those rows alone."""
    N, K = 300000, 32768
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    B = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    SB = torch.rand((N, K // group), device="cuda").half()
    a = torch.randn((2, K), device="cuda").half()
    d = tg.gemm_w4(a, B, SB, group=group)
    for lo in (0, 262143, N - 70):
        codes, s = B[lo:lo + 70].cpu().numpy(), SB[lo:lo + 70].cpu()
        w4_tests.check(d[:, lo:lo + 70], a, codes, s, None, group, "f16")
