"""GPU tests of the products with 4-bit weights against 64-bit references."""
import numpy as np
import pytest

from tests import experts_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def weights(rng, N, K, group, zeros, name, whole=False):
    """Packed codes, scales and zero points on the host (scales rounded to the type);
    `whole`: scales that are powers of two, so that small sums are exact."""
    kg = -(-K // group)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = 2.0 ** rng.integers(-2, 3, (N, kg)) if whole else rng.normal(size=(N, kg)) * 0.05
    s = torch.from_numpy(s).to(TYPES[name])
    z = rng.integers(0, 16, (N, kg)).astype(np.uint8) if zeros else None
    return codes, s, z


def gpu(codes, s, z):
    return (torch.from_numpy(codes).cuda(), s.cuda(),
            None if z is None else torch.from_numpy(z).cuda())


def check(got, a, codes, s, z, group, name):
    w = ref.weights_w4(codes, s.double().numpy(), z, group)
    x = a.double().cpu().numpy()
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    bound = ref.w4_bound(want, size, x.shape[1], group, name == "bf16")
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err - bound).max())


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 7, 64), (1, 4096, 14336), (2, 33, 96), (3, 1000, 160), (8, 130, 2048),
    (9, 257, 2080), (16, 500, 4128), (17, 64, 1056), (27, 1433, 4096), (32, 5003, 544),
    (33, 40, 288), (64, 300, 2048), (100, 77, 1024), (1, 20000, 256), (5, 16, 16384),
    (31, 129, 8224)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name,zeros", [("f16", True), ("bf16", False), ("bf16", True),
                                        ("f16", False)])
def test_product(tg, M, N, K, group, name, zeros):
    rng = np.random.default_rng(M + N + K + group)
    codes, s, z = weights(rng, N, K, group, zeros, name)
    a = torch.from_numpy(rng.normal(size=(M, K))).to(TYPES[name]).cuda()
    B, SB, ZB = gpu(codes, s, z)
    d = tg.gemm_w4(a, B, SB, ZB, group=group)
    assert d.dtype == TYPES[name] and d.shape == (M, N)
    check(d, a, codes, s, z, group, name)
    tg.check()


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 5, 12, 30])
def test_whole_numbers_are_exact(tg, name, M):
    """Sums of whole numbers below 2^8 times powers of two: equal, each k in its place."""
    N, K, group = 150, 416, 32
    rng = np.random.default_rng(M)
    codes, s, z = weights(rng, N, K, group, True, name, whole=True)
    for k in range(0, K, 5):
        a = torch.zeros((M, K))
        a[:, k] = torch.arange(1, M + 1) % 8 + 1
        B, SB, ZB = gpu(codes, s, z)
        d = tg.gemm_w4(a.to(TYPES[name]).cuda(), B, SB, ZB, group=group)
        want = a.double().numpy() @ ref.weights_w4(codes, s.double().numpy(), z, group).T
        assert np.array_equal(d.double().cpu().numpy(), want)


def grouped(tg, rng, counts, N, K, group, zeros, name, pad=(0, 0)):
    G, M = len(counts), sum(counts) + sum(pad)
    off = pad[0] + np.concatenate([[0], np.cumsum(counts)])
    parts = [weights(rng, N, K, group, zeros, name) for _ in range(G)]
    a = torch.from_numpy(rng.normal(size=(M, K))).to(TYPES[name]).cuda()
    B = torch.from_numpy(np.stack([p[0] for p in parts])).cuda()
    SB = torch.stack([p[1] for p in parts]).cuda()
    ZB = torch.from_numpy(np.stack([p[2] for p in parts])).cuda() if zeros else None
    out = torch.full((M, N), 5.0, device="cuda", dtype=TYPES[name])
    tg.gemm_w4_grouped(a, B, SB, torch.tensor(off, dtype=torch.int32, device="cuda"), ZB,
                       group=group, out=out)
    assert torch.all(out[:off[0]] == 5.0) and torch.all(out[off[-1]:] == 5.0)
    for g in range(G):
        rows = slice(off[g], off[g + 1])
        check(out[rows], a[rows], *parts[g], group, name)
    tg.check()


@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 32), ([0, 3, 0, 1, 0], 136, 160), ([1] * 40, 100, 288), ([2, 0, 9, 31, 33], 391, 416),
    ([40, 0, 1, 70, 25, 17], 300, 544), ([0, 0, 0, 130], 4099, 96), ([5, 9, 0, 3], 520, 2080),
    ([200], 64, 2048), ([0, 0], 64, 64), ([8] * 16, 1030, 1056)])
@pytest.mark.parametrize("group,zeros,name", [(32, True, "f16"), (128, False, "bf16"),
                                              (64, True, "bf16")])
def test_grouped(tg, counts, N, K, group, zeros, name):
    grouped(tg, np.random.default_rng(sum(counts) + N), counts, N, K, group, zeros, name, (0, 0))


def test_grouped_rows_outside_every_group_are_left(tg):
    grouped(tg, np.random.default_rng(1), [3, 0, 40, 9], 264, 288, 64, True, "f16", (7, 20))


def test_grouped_most_groups(tg):
    rng = np.random.default_rng(2)
    grouped(tg, rng, list(rng.integers(0, 4, 384)), 40, 64, 32, True, "bf16")


@pytest.mark.parametrize("off", [[-7, 20, 1 << 30, -(1 << 31), 5], [0, 50, 20, 60],
                                 [40, 10, -3, 7, 55, 12, 90]])
def test_grouped_offsets_out_of_order_count_as_the_largest_so_far(tg, off):
    rng = np.random.default_rng(3)
    M, N, K, G = 60, 136, 160, len(off) - 1
    parts = [weights(rng, N, K, 32, False, "f16") for _ in range(G)]
    a = torch.from_numpy(rng.normal(size=(M, K))).half().cuda()
    out = torch.full((M, N), 5.0, device="cuda", dtype=torch.float16)
    tg.gemm_w4_grouped(a, torch.from_numpy(np.stack([p[0] for p in parts])).cuda(),
                       torch.stack([p[1] for p in parts]).cuda(),
                       torch.tensor(off, dtype=torch.int32, device="cuda"), group=32, out=out)
    eff = np.clip(np.maximum.accumulate(off), 0, M)
    for g in range(G):
        rows = slice(eff[g], eff[g + 1])
        if eff[g + 1] > eff[g]:
            check(out[rows], a[rows], *parts[g], 32, "f16")
    assert torch.all(out[:eff[0]] == 5.0) and torch.all(out[eff[-1]:] == 5.0)


def test_nan_stays_in_its_row(tg):
    rng = np.random.default_rng(4)
    codes, s, z = weights(rng, 70, 288, 32, True, "bf16")
    for M in (2, 11, 30):
        a = torch.from_numpy(rng.normal(size=(M, 288))).bfloat16().cuda()
        a[1, 200] = float("nan")
        s2 = s.clone()
        s2[69, 2] = float("nan")
        d = tg.gemm_w4(a, *gpu(codes, s2, z), group=32)
        assert torch.isnan(d[1]).all() and torch.isnan(d[:, 69]).all()
        keep = torch.ones(M, dtype=torch.bool)
        keep[1] = False
        assert not torch.isnan(d[keep.cuda()][:, :69]).any()


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("M", [3, 12])
def test_infinite_scales_where_k_ends_inside_a_block(tg, name, M):
    """An infinite scale makes its row infinite (or NaN where the group's sum is zero), also
    when the row's last scales are fewer than the k of a step."""
    N, K, group = 40, 2208, 32
    rng = np.random.default_rng(M)
    codes, s, z = weights(rng, N, K, group, True, name)
    a = torch.from_numpy(rng.integers(1, 5, (M, K))).to(TYPES[name]).cuda()
    for g in range(K // group):
        s[g % N, g] = float("inf")
    d = tg.gemm_w4(a, *gpu(codes, s, z), group=group).double().cpu().numpy()
    w = ref.weights_w4(codes, np.ones(s.shape), z, group)
    x = a.double().cpu().numpy()
    for n in range(N):
        mine = [g for g in range(K // group) if g % N == n]
        sums = [x[:, g * group:(g + 1) * group] @ w[n, g * group:(g + 1) * group] for g in mine]
        want = np.sum([np.where(v == 0, np.nan, np.copysign(np.inf, v)) for v in sums], axis=0) \
            if mine else None
        assert want is None or np.array_equal(d[:, n], want, equal_nan=True), n


@pytest.mark.parametrize("M,N,K", [
    (9, 128, 32), (33, 129, 96), (16, 127, 8224), (17, 300, 16384), (12, 4100, 1056),
    (65, 20000, 160), (24, 1, 12320), (300, 257, 544), (10, 390, 2944)])
@pytest.mark.parametrize("group,zeros,name", [(32, True, "bf16"), (64, True, "f16"),
                                              (128, False, "f16"), (128, True, "bf16")])
def test_more_than_eight_tokens(tg, M, N, K, group, zeros, name):
    """Short and long K (split over CTAs, or no block of it for some warps), one to many
    blocks of rows and of tokens, twice with one result."""
    rng = np.random.default_rng(M * N + K)
    codes, s, z = weights(rng, N, K, group, zeros, name)
    a = torch.from_numpy(rng.normal(size=(M, K))).to(TYPES[name]).cuda()
    b = gpu(codes, s, z)
    d = tg.gemm_w4(a, *b, group=group)
    check(d, a, codes, s, z, group, name)
    assert torch.equal(d, tg.gemm_w4(a, *b, group=group))
    tg.check()


def test_unaligned_scales_and_results(tg):
    """Scales and results need the alignment of their elements only."""
    rng = np.random.default_rng(5)
    M, N, K = 3, 37, 160
    codes, s, z = weights(rng, N, K, 32, True, "f16")
    a = torch.from_numpy(rng.normal(size=(M, K))).half().cuda()
    B, SB, ZB = gpu(codes, s, z)
    S1 = torch.empty(SB.numel() + 1, device="cuda", dtype=SB.dtype)[1:].view_as(SB).copy_(SB)
    Z1 = torch.empty(ZB.numel() + 3, device="cuda", dtype=ZB.dtype)[3:].view_as(ZB).copy_(ZB)
    out = torch.empty(M * N + 1, device="cuda", dtype=torch.float16)[1:].view(M, N)
    tg.gemm_w4(a, B, S1, Z1, group=32, out=out)
    check(out, a, codes, s, z, 32, "f16")


def test_no_rows(tg):
    rng = np.random.default_rng(6)
    B, SB, _ = gpu(*weights(rng, 40, 64, 32, False, "f16"))
    assert tg.gemm_w4(torch.empty((0, 64), device="cuda").half(), B, SB, group=32).shape == (0, 40)


def test_weights_past_32_bit_offsets(tg):
    """Codes of more than 2^32 bytes: the last rows against a product of those rows alone."""
    N, K = 300000, 32768
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    B = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    SB = torch.rand((N, K // 128), device="cuda").half()
    a = torch.randn((2, K), device="cuda").half()
    d = tg.gemm_w4(a, B, SB)
    for lo in (0, 262143, N - 70):
        codes, s = B[lo:lo + 70].cpu().numpy(), SB[lo:lo + 70].cpu()
        check(d[:, lo:lo + 70], a, codes, s, None, 128, "f16")


def test_refusals(tg):
    rng = np.random.default_rng(7)
    B, SB, ZB = gpu(*weights(rng, 40, 128, 32, True, "f16"))
    a = torch.zeros((2, 128), device="cuda").half()
    for error, args, kw in ((TypeError, (a.float(), B, SB), {}), (TypeError, (a.bfloat16(), B, SB), {}),
                            (ValueError, (a, B, SB), dict(group=64)),
                            (ValueError, (a, B, SB), dict(group=48)),
                            (ValueError, (a[:, :120].contiguous(), B, SB), {}),
                            (TypeError, (a, B, SB, ZB.short()), {}),
                            (ValueError, (a, B, SB, ZB[:, :3]), {}),
                            (ValueError, (a, B[:, :32], SB), {}),
                            (TypeError, (a, B, SB), dict(out=torch.zeros((2, 40), device="cuda")))):
        with pytest.raises(error):
            tg.gemm_w4(*args, **{"group": 32, **kw})
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        tg.gemm_w4_grouped(a, B[None], SB[None], off, group=32)
    with pytest.raises(TypeError):
        tg.gemm_w4_grouped(a, B[None], SB[None], off[:2].long(), group=32)


def test_streams_and_graphs(tg):
    """On another stream, and captured and replayed with other rows, offsets and weights."""
    rng = np.random.default_rng(8)
    G, M, N, K = 4, 40, 264, 544
    parts = [weights(rng, N, K, 64, True, "bf16") for _ in range(G)]
    B = torch.from_numpy(np.stack([p[0] for p in parts])).cuda()
    SB = torch.stack([p[1] for p in parts]).cuda()
    ZB = torch.from_numpy(np.stack([p[2] for p in parts])).cuda()
    a = torch.randn((M, K), device="cuda").bfloat16()
    off = torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32, device="cuda")

    def step(stream=None):
        return [tg.gemm_w4_grouped(a, B, SB, off, ZB, group=64, stream=stream),
                tg.gemm_w4(a[:9], B[1], SB[1], ZB[1], group=64, stream=stream),
                tg.gemm_w4(a, B[2], SB[2], ZB[2], group=64, stream=stream)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for counts in ([10, 10, 10, 10], [0, 39, 0, 1], [40, 0, 0, 0]):
        off.copy_(torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32))
        a.copy_(torch.randn((M, K), device="cuda").bfloat16())
        B.copy_(torch.randint(0, 256, B.shape, dtype=torch.uint8, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, step()))
    tg.check()
