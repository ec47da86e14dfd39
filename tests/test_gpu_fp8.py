"""GPU tests of quantize_fp8, gemm_fp8 and gemm_fp8_grouped against 64-bit
references (tests/fp8_reference.py, which also derives the bound of a product)."""
import numpy as np
import pytest

from tests import fp8_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


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


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def f8(c, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(c)).to(device).view(torch.float8_e4m3fn)


def random_operand(rng, rows, K, per_row):
    """Codes over the whole finite range and scales of mixed sizes."""
    c = rng.integers(0, 255, (rows, K)).astype(np.uint8)
    c[(c & 127) == 127] = 0
    s = np.exp(rng.normal(size=(rows if per_row else -(-rows // 128), -(-K // 128)))) * 2e-3
    return c, s.astype(np.float32)


def integer_operand(rng, rows, K, per_row):
    """Small integers and power-of-two scales: every sum is exact in FP32."""
    c = ref.encode_e4m3(rng.integers(-4, 5, (rows, K)))
    s = 2.0 ** rng.integers(-1, 2, (rows if per_row else -(-rows // 128), -(-K // 128)))
    return c, s.astype(np.float32)


def rounded(d, dtype):
    return torch.from_numpy(d).to(dtype).double().numpy()


def check_product(got, a, sa, b, sb, bf16):
    want, size = ref.gemm(a, sa, b, sb)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = ref.gemm_bound(want, size, a.shape[1], bf16)
    assert np.all(err <= bound), (err - bound).max()


# ---------------------------------------------------------------- quantise ----

@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (3, 136), (33, 1032), (129, 264), (257, 2056),
                                 (5000, 8200)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_quantize_bits(tg, M, K, block_rows, name):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn((M, K), generator=g) * torch.exp(2 * torch.randn((1, K), generator=g)))
    x = x.clamp(-6e4, 6e4).to(TYPES[name])
    Q, S = tg.quantize_fp8(x.cuda(), block_rows=block_rows)
    assert Q.dtype == torch.float8_e4m3fn and Q.shape == (M, K)
    assert S.shape == (-(-M // block_rows), -(-K // 128))
    rows = slice(None) if M < 1000 else slice(M - 300, M)      # the last rows of the large one
    first = 0 if M < 1000 else M - 300
    if block_rows == 128 and M >= 1000:
        first = (M - 300) // 128 * 128
        rows = slice(first, M)
    want_q, want_s = ref.quantize(x[rows].double().numpy(), block_rows)
    assert np.array_equal(codes(Q)[rows], want_q)
    assert np.array_equal(S.cpu().numpy()[first // block_rows:], want_s)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_zeros_infinities_and_nan(tg, name, block_rows):
    x = torch.zeros((256, 256), dtype=TYPES[name])
    x[0:128, 128:] = 1.0
    x[130, 3] = float("inf")
    x[131, 140] = float("nan")
    Q, S = (t.cpu() for t in tg.quantize_fp8(x.cuda(), block_rows=block_rows))
    q = Q.float()
    assert torch.all(q[:128, :128] == 0) and torch.isfinite(S[0]).all() and (S[0] > 0).all()
    assert torch.all(q[:128, 128:] == 448)
    at = (lambda r: r) if block_rows == 1 else (lambda r: r // 128)
    assert S[at(130), 0] == float("inf") and torch.isnan(q[130, 3])
    assert torch.all(q[130, :3] == 0)
    assert torch.isnan(S[at(131), 1]) and torch.isnan(q[131, 140])
    if block_rows == 1:
        assert torch.isfinite(S[129]).all()      # other rows are not touched


def test_quantize_smallest_values(tg):
    """Magnitudes below the scales' floor keep finite scales and quantise to 0
    or to their value times the floor's reciprocal scale."""
    x = torch.full((2, 128), 2.0 ** -130, dtype=torch.bfloat16)
    x[1] = 2.0 ** -99
    Q, S = tg.quantize_fp8(x.cuda())
    want_q, want_s = ref.quantize(x.double().numpy(), 1)
    assert np.array_equal(codes(Q), want_q) and np.array_equal(S.cpu().numpy(), want_s)


def test_quantize_no_rows(tg):
    Q, S = tg.quantize_fp8(torch.empty((0, 256), device="cuda", dtype=torch.bfloat16))
    assert Q.shape == (0, 256) and S.shape == (0, 2)


# ----------------------------------------------------------------- product ----

SHAPES = [(1, 8, 16), (1, 4096, 1040), (2, 136, 144), (7, 1000, 400), (15, 264, 4112),
          (16, 640, 128), (17, 72, 2064), (32, 520, 1024), (33, 1160, 272), (64, 256, 8192),
          (65, 392, 528), (100, 5000, 256), (128, 128, 128), (129, 136, 144), (200, 1544, 1040),
          (300, 264, 2064), (777, 2056, 528), (1000, 5000, 272), (2100, 4104, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_gemm_parity(tg, M, N, K, name):
    rng = np.random.default_rng(M * 7 + N)
    a, sa = random_operand(rng, M, K, True)
    b, sb = random_operand(rng, N, K, False)
    d = tg.gemm_fp8(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                    dtype=TYPES[name])
    assert d.shape == (M, N) and d.dtype == TYPES[name]
    check_product(d, a, sa, b, sb, name == "bf16")


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_integers_are_exact(tg, M, N, K):
    rng = np.random.default_rng(M + N + K)
    a, sa = integer_operand(rng, M, K, True)
    b, sb = integer_operand(rng, N, K, False)
    want, _ = ref.gemm(a, sa, b, sb)
    for name, dtype in TYPES.items():
        d = tg.gemm_fp8(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                        dtype=dtype)
        assert np.array_equal(d.double().cpu().numpy(), rounded(want, dtype)), name


@pytest.mark.parametrize("M,N,K", [(1, 264, 400), (40, 264, 400), (300, 264, 400)])
def test_gemm_scale_layouts(tg, M, N, K):
    """Row-major scales, columns next to each other and a strided window give
    the same bits."""
    rng = np.random.default_rng(3)
    a, sa = random_operand(rng, M, K, True)
    b, sb = random_operand(rng, N, K, False)
    A, B, SB = f8(a), f8(b), torch.from_numpy(sb).cuda()
    rows = torch.from_numpy(sa).cuda()
    wide = torch.zeros((3 * M, 2 * sa.shape[1]), device="cuda")
    window = wide[::3, ::2]
    window.copy_(rows)
    want = tg.gemm_fp8(A, rows, B, SB)
    for s in (rows.t().contiguous().t(), window):
        assert torch.equal(tg.gemm_fp8(A, s, B, SB), want)


def test_gemm_refuses_broadcast_scales(tg):
    A = f8(np.zeros((4, 256), np.uint8))
    B = f8(np.zeros((8, 256), np.uint8))
    SB = torch.ones((1, 2), device="cuda")
    with pytest.raises(tg.TmaGemmError) as e:
        tg.gemm_fp8(A, torch.ones((1, 1), device="cuda").expand(4, 2), B, SB)
    assert e.value.status == tg.TMAGEMM_ERR_INVALID


@pytest.mark.parametrize("M", [1, 20, 100, 300, 1300])
def test_gemm_nan_and_infinity_stay_in_their_rows(tg, M):
    N, K = 264, 400
    rng = np.random.default_rng(4)
    a, sa = random_operand(rng, M, K, True)
    b, sb = random_operand(rng, N, K, False)
    bad = M // 2
    a[bad, 5] = 0x7f                                   # a NaN code
    if M > 1:
        sa[0, 1] = np.inf
    b[9, 7] = 0xff
    d = tg.gemm_fp8(f8(a), torch.from_numpy(sa).cuda(), f8(b),
                    torch.from_numpy(sb).cuda()).double().cpu().numpy()
    want, _ = ref.gemm(a, sa, b, sb)
    assert np.all(np.isnan(d[bad])) and np.all(np.isnan(d[:, 9]))
    assert np.array_equal(np.isfinite(d), np.isfinite(want))
    assert np.array_equal(np.isnan(d), np.isnan(want))


def test_gemm_no_rows_and_given_result(tg):
    B, SB = f8(np.zeros((8, 128), np.uint8)), torch.ones((1, 1), device="cuda")
    A = torch.empty((0, 128), device="cuda", dtype=torch.float8_e4m3fn)
    assert tg.gemm_fp8(A, torch.empty((0, 1), device="cuda"), B, SB).shape == (0, 8)
    out = torch.full((2, 8), 7.0, device="cuda", dtype=torch.float16)
    A = f8(np.zeros((2, 128), np.uint8))
    assert tg.gemm_fp8(A, torch.ones((2, 1), device="cuda"), B, SB, out=out) is out
    assert torch.all(out == 0)
    with pytest.raises(ValueError):
        tg.gemm_fp8(A, torch.ones((2, 1), device="cuda"), B, SB, out=out[:, :4])
    with pytest.raises(TypeError):
        tg.gemm_fp8(A, torch.ones((2, 1), device="cuda"), B, SB, dtype=torch.float32)


@pytest.mark.parametrize("M,N,K", [(3, 1032, 2064), (100, 1032, 2064), (1000, 1032, 2064)])
def test_gemm_repeats_its_bits(tg, M, N, K):
    rng = np.random.default_rng(5)
    a, sa = random_operand(rng, M, K, True)
    b, sb = random_operand(rng, N, K, False)
    args = (f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda())
    want = tg.gemm_fp8(*args)
    try:
        for pdl in (1, 0):
            assert tg.tmagemm_set_pdl(pdl) == tg.TMAGEMM_OK
            for _ in range(3):
                assert torch.equal(tg.gemm_fp8(*args), want)
    finally:
        tg.tmagemm_set_pdl(1)


def test_gemm_writes_nothing_past_its_result(tg):
    """Rows before and after a window of a larger buffer keep their values."""
    rng = np.random.default_rng(6)
    for M, N in ((1, 136), (70, 136), (131, 392), (260, 1000)):
        a, sa = random_operand(rng, M, 144, True)
        b, sb = random_operand(rng, N, 144, False)
        big = torch.full((M + 64, N), 3.0, device="cuda", dtype=torch.bfloat16)
        tg.gemm_fp8(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                    out=big[32:32 + M])
        assert torch.all(big[:32] == 3.0) and torch.all(big[32 + M:] == 3.0)
        check_product(big[32:32 + M], a, sa, b, sb, True)


def test_gemm_result_past_32_bit_offsets(tg):
    M, N, K = 66000, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    A = torch.randint(-4, 5, (M, K), device="cuda", generator=g).float().to(torch.float8_e4m3fn)
    B = torch.randint(-4, 5, (N, K), device="cuda", generator=g).float().to(torch.float8_e4m3fn)
    d = tg.gemm_fp8(A, torch.ones((M, 1), device="cuda"), B, torch.ones((N // 128, 1), device="cuda"))
    assert d.numel() > 1 << 31
    rows = torch.tensor([0, 1, M // 2, M - 300, M - 1], device="cuda")
    assert torch.equal(d[rows].float(), (A[rows].float() @ B.float().t()).bfloat16().float())


@pytest.mark.parametrize("grouped", [False, True])
def test_product_of_the_most_rows(tg, grouped):
    """The last row whose index fits 32 bits (dense), and as many rows as groups may
    have, in a last group that starts inside a tile: about 77 GB."""
    M, N, K = (1 << 31) - (256 if grouped else 1), 8, 16
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    rng = np.random.default_rng(15)
    b, _ = integer_operand(rng, N, K, False)
    B, SB = f8(b), torch.ones((1, 1), device="cuda")
    A = f8(ref.encode_e4m3(np.arange(16) % 5 - 2)).view(torch.uint8).expand(M, K).contiguous()
    marks = torch.tensor([0, 1, 4, 5, 6, 300, M // 2, M - 257, M - 129, M - 2, M - 1])
    A[marks.cuda()] = f8(ref.encode_e4m3(rng.integers(-4, 5, (len(marks), K)))).view(torch.uint8)
    A = A.view(torch.float8_e4m3fn)
    SA = torch.ones((M, 1), device="cuda")
    out = torch.full((M, N), float("nan"), device="cuda", dtype=torch.float16)
    if grouped:
        off = torch.tensor([0, 5, M], dtype=torch.int32, device="cuda")
        tg.gemm_fp8_grouped(A, SA, B.view(torch.uint8).expand(2, N, K).contiguous().view(B.dtype),
                            SB.expand(2, 1, 1).contiguous(), off, out=out)
    else:
        tg.gemm_fp8(A, SA, B, SB, out=out)
    del SA
    W = B.float()
    assert torch.equal(out[marks.cuda()].float(),
                       A.view(torch.uint8)[marks.cuda()].view(A.dtype).float() @ W.t())
    row = (f8(ref.encode_e4m3(np.arange(16) % 5 - 2)).float() @ W.t()).half()
    other = 0
    for lo in range(0, M, 1 << 27):
        other += int((out[lo:lo + (1 << 27)] != row).any(dim=1).sum())
    assert other <= len(marks)


# ----------------------------------------------------------------- grouped ----

def grouped_reference(a, sa, b, sb, off):
    return [ref.gemm(a[off[g]:off[g + 1]], sa[off[g]:off[g + 1]], b[g], sb[g])
            for g in range(len(off) - 1)]


@pytest.mark.parametrize("counts,N,K", [
    ([5], 8, 16), ([0, 3, 0, 1, 0], 136, 144), ([1] * 40, 264, 272), ([128, 0, 129, 31, 33], 392, 400),
    ([300, 0, 1, 700, 256, 17], 1000, 528), ([2000], 264, 144), ([0, 0, 0, 513], 4104, 272),
    ([64, 32, 96, 160, 31], 520, 2064)])
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_grouped_parity(tg, counts, N, K, name):
    rng = np.random.default_rng(sum(counts) + N)
    G, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    a, sa = random_operand(rng, M, K, True)
    bs = [random_operand(rng, N, K, False) for _ in range(G)]
    b, sb = np.stack([x[0] for x in bs]), np.stack([x[1] for x in bs])
    d = tg.gemm_fp8_grouped(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                            torch.tensor(off, dtype=torch.int32, device="cuda"), dtype=TYPES[name])
    d = d.double().cpu().numpy()
    for g, (want, size) in enumerate(grouped_reference(a, sa, b, sb, off)):
        bound = ref.gemm_bound(want, size, K, name == "bf16")
        assert np.all(np.abs(d[off[g]:off[g + 1]] - want) <= bound), g


def grouped_integers(rng, G, M, N, K):
    a, sa = integer_operand(rng, M, K, True)
    bs = [integer_operand(rng, N, K, False) for _ in range(G)]
    return a, sa, np.stack([x[0] for x in bs]), np.stack([x[1] for x in bs])


def test_grouped_rows_outside_every_group_are_left(tg):
    rng = np.random.default_rng(7)
    for M, off in ((100, [10, 30, 30, 77]), (1500, [3, 900, 901, 1400])):
        a, sa, b, sb = grouped_integers(rng, 3, M, 264, 272)
        out = torch.full((M, 264), 5.0, device="cuda", dtype=torch.bfloat16)
        tg.gemm_fp8_grouped(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                            torch.tensor(off, dtype=torch.int32, device="cuda"), out=out)
        assert torch.all(out[:off[0]] == 5.0) and torch.all(out[off[-1]:] == 5.0)
        for g, (want, _) in enumerate(grouped_reference(a, sa, b, sb, off)):
            got = out[off[g]:off[g + 1]].double().cpu().numpy()
            assert np.array_equal(got, rounded(want, torch.bfloat16)), g


def test_grouped_offsets_out_of_range_are_clamped(tg):
    """Offsets below 0, past the last row or decreasing: the groups that are
    well formed are right, and nothing outside the result is written."""
    rng = np.random.default_rng(8)
    M, N, K = 60, 136, 144
    a, sa, b, sb = grouped_integers(rng, 4, M, N, K)
    big = torch.full((M + 64, N), 5.0, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([-7, 20, 1 << 30, -(1 << 31), 5], dtype=torch.int32, device="cuda")
    tg.gemm_fp8_grouped(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                        off, out=big[32:32 + M])
    assert torch.all(big[:32] == 5.0) and torch.all(big[32 + M:] == 5.0)
    want, _ = ref.gemm(a[20:60], sa[20:60], b[1], sb[1])
    assert np.array_equal(big[52:92].double().cpu().numpy(), rounded(want, torch.bfloat16))


@pytest.mark.parametrize("M,off", [
    (60, [0, 50, 20, 60]),                          # group 2 starts where group 0 ends
    (60, [-7, 20, 1 << 30, -(1 << 31), 5]),
    (60, [40, 10, -3, 7, 55, 12, 90]),
    (900, [0, 700, 130, 300, 800, 260, 900]),       # rows enough for pair tiles
    (300, None)])                                   # 384 random offsets
def test_grouped_offsets_out_of_order_count_as_the_largest_so_far(tg, M, off):
    """Groups never overlap: each row has one owner, rows without one are left."""
    rng = np.random.default_rng(14)
    if off is None:
        off = rng.integers(-50, M + 50, 385)
        off[:300] = np.sort(off[:300])
    off = np.asarray(off)
    G, N, K = len(off) - 1, 136, 144
    a, sa, b, sb = grouped_integers(rng, G, M, N, K)
    out = torch.full((M, N), 5.0, device="cuda", dtype=torch.bfloat16)
    tg.gemm_fp8_grouped(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                        torch.tensor(off, dtype=torch.int32, device="cuda"), out=out)
    eff = np.clip(np.maximum.accumulate(off), 0, M)
    got = out.double().cpu().numpy()
    for g, (want, _) in enumerate(grouped_reference(a, sa, b, sb, eff)):
        assert np.array_equal(got[eff[g]:eff[g + 1]], rounded(want, torch.bfloat16)), g
    assert np.all(got[:eff[0]] == 5.0) and np.all(got[eff[-1]:] == 5.0)


def test_grouped_most_groups(tg):
    rng = np.random.default_rng(9)
    G, N, K = 384, 136, 144
    counts = rng.integers(0, 4, G)
    off = np.concatenate([[0], np.cumsum(counts)])
    a, sa, b, sb = grouped_integers(rng, G, int(off[-1]), N, K)
    d = tg.gemm_fp8_grouped(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                            torch.tensor(off, dtype=torch.int32, device="cuda"))
    for g, (want, _) in enumerate(grouped_reference(a, sa, b, sb, off)):
        assert np.array_equal(d[off[g]:off[g + 1]].double().cpu().numpy(),
                              rounded(want, torch.bfloat16)), g


def test_grouped_nan_stays_in_its_group(tg):
    rng = np.random.default_rng(10)
    off = [0, 20, 45, 300]
    a, sa, b, sb = grouped_integers(rng, 3, 300, 136, 144)
    a[19, 0] = 0x7f                 # last row of group 0, in the same tile as group 1's rows
    b[1] = 0x7f                     # all of group 1's weights
    d = tg.gemm_fp8_grouped(f8(a), torch.from_numpy(sa).cuda(), f8(b), torch.from_numpy(sb).cuda(),
                            torch.tensor(off, dtype=torch.int32, device="cuda"))
    d = d.double().cpu().numpy()
    assert np.all(np.isfinite(d[:19])) and np.all(np.isnan(d[19:45])) and np.all(np.isfinite(d[45:]))


# ----------------------------------------------- streams, graphs, large sizes ----

def test_other_stream_than_the_current(tg):
    rng = np.random.default_rng(11)
    side = torch.cuda.Stream()
    x = torch.randn((300, 528), device="cuda").bfloat16()
    b, sb = random_operand(rng, 264, 528, False)
    B, SB = f8(b), torch.from_numpy(sb).cuda()
    q, s = tg.quantize_fp8(x)
    want = tg.gemm_fp8(q, s, B, SB)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        q2, s2 = tg.quantize_fp8(x, stream=side)
        got = tg.gemm_fp8(q2, s2, B, SB, stream=side)
        del q2, s2
        torch.empty((300, 528), device="cuda", dtype=torch.uint8).fill_(255)   # reuse freed memory
        side.synchronize()
        assert torch.equal(got, want)


def test_graph_follows_the_offsets_and_the_inputs(tg):
    """A captured quantise + grouped product replayed with other offsets and
    inputs: nothing of the first call is kept."""
    rng = np.random.default_rng(12)
    G, M, N, K = 4, 200, 264, 272
    bs = [random_operand(rng, N, K, False) for _ in range(G)]
    B = f8(np.stack([x[0] for x in bs]))
    SB = torch.from_numpy(np.stack([x[1] for x in bs])).cuda()
    x = torch.randn((M, K), device="cuda").half()
    off = torch.tensor([0, 50, 100, 150, 200], dtype=torch.int32, device="cuda")

    def step():
        q, s = tg.quantize_fp8(x)
        return tg.gemm_fp8_grouped(q, s, B, SB, off, dtype=torch.float16)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for counts in ([50, 50, 50, 50], [0, 199, 0, 1], [200, 0, 0, 0]):
        off.copy_(torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32))
        x.copy_(torch.randn((M, K), device="cuda").half())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


def test_quantize_past_32_bit_offsets(tg):
    M, K = 140000, 16384
    x = torch.zeros((M, K), device="cuda", dtype=torch.bfloat16)
    rows = [0, 65536, 131072, M - 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    for r in rows:
        x[r] = torch.randn(K, device="cuda", generator=g).bfloat16()
    Q, S = tg.quantize_fp8(x)
    want_q, want_s = ref.quantize(x[rows].double().cpu().numpy(), 1)
    assert np.array_equal(codes(Q[rows]), want_q)
    assert np.array_equal(S[rows].cpu().numpy(), want_s)
    assert not Q[1:65536].view(torch.uint8).any()
