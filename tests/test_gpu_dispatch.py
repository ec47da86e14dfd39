"""GPU tests of dispatch_rows, combine_rows and its gradients.  Places are whole numbers
and rows copies or codes: equal.  A sum over k choices is off by half a step of its type
and k + 1 steps of 2^-24 of the terms' magnitudes; a gradient of a weight, summed over C
columns by lanes and warps, by at most C / 32 + 16 such steps."""
import numpy as np
import pytest

from tests import experts_reference as ref
from tests import fp8_reference as ref8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def choices(T, k, E, kind="some", seed=0):
    rng = np.random.default_rng(seed + T + k + E)
    if kind == "one":
        return np.full((T, k), E - 1)
    ids = rng.integers(0, E, (T, k))
    if kind == "padded":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[T // 2:] = rng.choice([-1, E, 1 << 30, -(1 << 31)], (T - T // 2, k))
    if kind == "none":
        ids[:] = -1
    return ids


def on_gpu(ids):
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def random(shape, name, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(TYPES[name])


def same_bytes(a, b):
    if a.dtype == torch.float8_e4m3fn:
        a, b = a.view(torch.uint8), b.view(torch.uint8)
    else:
        a, b = a.view(torch.int16), b.view(torch.int16)
    return torch.equal(a, b)


SIZES = [(1, 1, 1, 8), (1, 8, 64, 4096), (3, 2, 5, 136), (16, 4, 64, 1032), (33, 1, 7, 256),
         (40, 32, 512, 264), (257, 3, 384, 520), (700, 8, 16, 128), (2100, 8, 61, 40)]


@pytest.mark.parametrize("T,k,E,C", SIZES)
@pytest.mark.parametrize("kind", ["some", "one", "padded", "none"])
@pytest.mark.parametrize("name,quantize", [("f16", False), ("bf16", True), ("f16", True),
                                           ("bf16", False)])
def test_rows_by_expert(tg, T, k, E, C, kind, name, quantize):
    ids = choices(T, k, E, kind)
    x = random((T, C), name)
    r = tg.dispatch_rows(x, on_gpu(ids), E, quantize=quantize)
    offsets, row_of, slots = ref.dispatch(ids, E)
    assert r.offsets.dtype == torch.int32 and r.row_of.dtype == torch.int32
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.row_of.cpu().numpy(), row_of)
    token = torch.from_numpy(slots // k).cuda()
    n = len(slots)
    assert r.rows.shape == (T * k, C)
    if quantize:
        q, s = tg.quantize_fp8(x)
        assert r.rows.dtype == torch.float8_e4m3fn
        assert same_bytes(r.rows[:n], q.view(torch.uint8)[token].view(q.dtype))
        assert torch.equal(r.scales[:n], s[token])
    else:
        assert r.scales is None and same_bytes(r.rows[:n], x[token])


@pytest.mark.parametrize("T,k,E,C", [
    (256, 1, 9, 8), (257, 1, 512, 8), (8192, 1, 3, 8), (1025, 8, 33, 8), (5000, 4, 512, 16),
    (4100, 8, 64, 8), (8190, 8, 7, 8), (4096, 32, 500, 8), (4097, 32, 300, 8)])
@pytest.mark.parametrize("kind", ["some", "one", "padded"])
def test_many_slots(tg, T, k, E, C, kind):
    """As many as each way of placing them takes."""
    test_rows_by_expert(tg, T, k, E, C, kind, "bf16", False)


def test_codes_against_the_reference(tg):
    x = random((20, 272), "bf16") * torch.logspace(-6, 6, 20, device="cuda").bfloat16()[:, None]
    x[3] = 0
    ids = choices(20, 2, 4)
    r = tg.dispatch_rows(x, on_gpu(ids), 4, quantize=True)
    codes, scales = ref8.quantize(x.double().cpu().numpy(), 1)
    token = ref.dispatch(ids, 4)[2] // 2
    assert np.array_equal(r.rows.view(torch.uint8).cpu().numpy(), codes[token])
    assert np.array_equal(r.scales.cpu().numpy(), scales[token])


def combine_reference(rows, row_of, w):
    T, k = row_of.shape
    y, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for j in range(k):
        have = (row_of[:, j] >= 0) & (row_of[:, j] < len(rows))
        part = w[have, j, None] * rows[row_of[have, j]]
        y[have] += part
        size[have] += np.abs(part)
    return y, size


@pytest.mark.parametrize("T,k,E,C", SIZES)
@pytest.mark.parametrize("kind", ["some", "padded", "none"])
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_gradients(tg, T, k, E, C, kind, name, weighted):
    _, row_of, slots = ref.dispatch(choices(T, k, E, kind), E)
    rows, dy = random((T * k, C), name, 1), random((T, C), name, 2)
    rows[len(slots):] = float("nan")        # rows of no choice are not read
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(3))
    w[0, 0] = 0.0
    at = on_gpu(row_of)
    got = tg.combine_rows(rows, at, w.cuda() if weighted else None).double().cpu().numpy()
    full = rows.double().cpu().numpy()
    wd = w.double().numpy() if weighted else np.ones((T, k))
    want, size = combine_reference(full, row_of, wd)
    assert np.all(np.abs(got - want) <= HALF[name] * np.abs(want) + (k + 1) * 2.0 ** -24 * size
                  + TINY[name])
    if not weighted:
        return
    d = tg.combine_rows_backward(dy, rows, at, w.cuda())
    g, have = dy.double().cpu().numpy(), row_of >= 0
    drows, dweights = d.drows.double().cpu().numpy(), d.dweights.double().cpu().numpy()
    assert np.all(dweights[~have] == 0.0)
    t, j = np.nonzero(have)
    picked = full[row_of[t, j]]
    want_w = (g[t] * picked).sum(axis=1)
    bound = (C / 32 + 16) * 2.0 ** -24 * np.abs(g[t] * picked).sum(axis=1)
    assert np.all(np.abs(dweights[t, j] - want_w) <= bound)
    want_r = w.double().numpy()[t, j, None] * g[t]
    # (the product is rounded to 32 bits before its type: one step more)
    bound = (HALF[name] + 2.0 ** -24) * np.abs(want_r) + TINY[name]
    assert np.all(np.abs(drows[row_of[t, j]] - want_r) <= bound)


def test_rows_of_no_choice_are_left(tg):
    """Through the C ABI, into buffers of the caller's: rows past the last slot's, and
    memory around the results, keep what they hold."""
    T, k, E, C = 50, 4, 6, 264
    ids = choices(T, k, E, "padded")
    offsets, row_of, slots = ref.dispatch(ids, E)
    x, rows = random((T, C), "f16"), torch.full((T * k + 2, C), 5.0, device="cuda").half()
    off = torch.full((E + 3,), 77, dtype=torch.int32, device="cuda")
    at = torch.full((T + 2, k), 77, dtype=torch.int32, device="cuda")
    idc = on_gpu(ids)
    need = tg.lib().dispatch_rows_workspace_size(T, k, E)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    st = tg.lib().dispatch_rows(T, k, E, C, idc.data_ptr(), x.data_ptr(), 0, rows[1].data_ptr(), None,
                                1, 1, off[1].data_ptr(), at[1].data_ptr(), ws.data_ptr(), need, None)
    assert st == tg.TMAGEMM_OK
    torch.cuda.synchronize()
    assert np.array_equal(off.cpu().numpy(), [77, *offsets, 77])
    assert np.array_equal(at[1:-1].cpu().numpy(), row_of)
    assert (at[[0, -1]] == 77).all() and (rows[0] == 5.0).all()
    assert (rows[1 + len(slots):] == 5.0).all()
    assert torch.equal(rows[1:1 + len(slots)], x[torch.from_numpy(slots // k).cuda()])
    # the gradients of rows likewise
    drows = torch.full((T * k, C), 5.0, device="cuda").half()
    w, dw = torch.ones((T, k), device="cuda"), torch.empty((T, k), device="cuda")
    at = at[1:-1].contiguous()
    st = tg.lib().combine_rows_backward(T, k, C, T * k, x.data_ptr(), x.repeat(k, 1).data_ptr(),
                                        at.data_ptr(), w.data_ptr(), drows.data_ptr(), dw.data_ptr(),
                                        0, None)
    assert st == tg.TMAGEMM_OK
    torch.cuda.synchronize()
    assert (drows[len(slots):] == 5.0).all()


def test_no_tokens(tg):
    r = tg.dispatch_rows(torch.empty((0, 64), device="cuda").half(),
                         torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert r.rows.shape == (0, 64) and r.offsets.tolist() == [0] * 10
    y = tg.combine_rows(r.rows, r.row_of, torch.empty((0, 4), device="cuda"))
    assert y.shape == (0, 64)
    # no rows to read, tokens without choices: zeros
    y = tg.combine_rows(r.rows, torch.full((3, 4), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, torch.zeros_like(y)) and y.shape == (3, 64)


def test_rows_past_32_bit_offsets(tg):
    """2^32 elements of rows: those of the last expert lie past every 32-bit offset."""
    T, k, E, C = 65536, 8, 3, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    ids = np.zeros((T, k), dtype=np.int64)
    ids[5, 3] = ids[T - 1, 7] = 2
    ids[77, 1] = 1
    x = random((T, C), "bf16")
    r = tg.dispatch_rows(x, on_gpu(ids), E)
    n = T * k
    assert r.offsets.tolist() == [0, n - 3, n - 2, n]
    assert torch.equal(r.rows[n - 3:], x[[77, 5, T - 1]])
    assert torch.equal(r.rows[n - 4], x[T - 1]) and torch.equal(r.rows[n - 11], x[T - 2])
    w = torch.zeros((T, k), device="cuda")
    w[5, 3], w[T - 1, 7], w[0, 0] = 2.0, 3.0, 1.0
    y = tg.combine_rows(r.rows, r.row_of, w)
    for t, f in ((5, 2.0), (T - 1, 3.0), (0, 1.0), (77, 0.0)):
        assert torch.equal(y[t], (f * x[t].float()).bfloat16())
    d = tg.combine_rows_backward(x, r.rows, r.row_of, w)
    assert torch.equal(d.drows[n - 1], (3.0 * x[T - 1].float()).bfloat16())
    square = x[T - 1].double().square().sum()
    assert abs(float(d.dweights[T - 1, 7]) - float(square)) <= (C / 32 + 16) * 2.0 ** -24 * float(square)


def test_refusals(tg):
    x, ids = random((4, 256), "f16"), on_gpu(choices(4, 2, 8))
    for error, args in ((TypeError, (x.float(), ids, 8)), (TypeError, (x, ids.long(), 8)),
                        (ValueError, (x, ids[:3], 8)), (ValueError, (x.t(), ids, 8)),
                        (tg.TmaGemmError, (x, ids, 0)), (tg.TmaGemmError, (x, ids, 513)),
                        (tg.TmaGemmError, (x[:, :252].contiguous(), ids, 8))):
        with pytest.raises(error):
            tg.dispatch_rows(*args)
    w = torch.ones((4, 2), device="cuda")
    rows = random((8, 256), "f16")
    for error, args in ((TypeError, (rows, ids, w.half())), (ValueError, (rows, ids, w[:3])),
                        (TypeError, (rows, ids.long(), w)), (ValueError, (rows[:, ::2], ids, w))):
        with pytest.raises(error):
            tg.combine_rows(*args)
    with pytest.raises(ValueError):
        tg.combine_rows_backward(x[:3], rows, ids, w)
    with pytest.raises(TypeError):
        tg.combine_rows_backward(x, rows, ids, None)


# ------------------------------------------------------- streams and graphs ----

def test_other_stream_than_the_current(tg):
    side = torch.cuda.Stream()
    x, logits = random((300, 264), "bf16"), torch.randn((300, 24), device="cuda")

    def step(stream=None):
        r = tg.route_topk(logits, 3, stream=stream)
        d = tg.dispatch_rows(x, r.ids, 24, stream=stream)
        return tg.combine_rows(d.rows, d.row_of, r.weights, stream=stream)

    want = step()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = step(side)
        torch.empty((900, 264), device="cuda", dtype=torch.bfloat16).fill_(255)   # freed memory
        side.synchronize()
        assert torch.equal(got, want)


def test_graph_follows_its_inputs(tg):
    """Route, dispatch, sum and gradients captured once and replayed with other logits:
    nothing of the first call is kept.  Two graphs of the same calls do not share
    workspaces."""
    T, E, C = 1500, 24, 264
    x, dy = random((T, C), "bf16", 4), random((T, C), "bf16", 5)
    logits = torch.randn((T, E), device="cuda")

    def step():
        r = tg.route_topk(logits, 3)
        d = tg.dispatch_rows(x, r.ids, E)
        y = tg.combine_rows(d.rows, d.row_of, r.weights)
        g = tg.combine_rows_backward(dy, d.rows, d.row_of, r.weights)
        return [y, g.drows, tg.combine_rows(g.drows, d.row_of),
                tg.route_topk_backward(logits, r.ids, g.dweights)]

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    side = torch.cuda.Stream()
    for seed in range(3):
        logits.copy_(torch.randn((T, E), generator=torch.Generator().manual_seed(seed)))
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        want = step()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
