"""GPU tests of norm_residual and its gradients against 64-bit references.

Bounds: an output is half a step of its type off for its one rounding (2^-8 of
bf16, 2^-11 of fp16), and each FP32 step before it 2^-24 of the magnitudes that
go into it.  The longest chain is under 64 such steps (about 20 operations and
the tree sums of a row: at most 16 terms per thread, 5 + 5 levels; column sums:
at most 7 rows per thread and 42 partial sums in the sizes here), so 2^-17 of
the magnitudes, twice that, is allowed."""
import numpy as np
import pytest

from tests import fp8_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -140}
STEP = 2.0 ** -17
EPS = 1e-6


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def near(got, want, size, kind, what):
    g = got.double().cpu().numpy().reshape(want.shape)
    bound = HALF[kind] * np.abs(want) + STEP * size + TINY[kind]
    err = np.abs(g - want)
    assert np.all(err <= bound), (what, float((err - bound).max()))


def make(T, C, name, gate, post, pre, seed=0, y=True):
    g = torch.Generator().manual_seed(seed + T + C)
    dt = TYPES[name]
    shape = {None: None, "channel": (C,), "token": (T, 1), "element": (T, C)}[gate]
    v = {"h": torch.randn((T, C), generator=g).to(dt),
         "y": torch.randn((T, C), generator=g).to(dt) if y else None,
         "gate": None if shape is None else torch.randn(shape, generator=g).to(dt),
         "w_post": torch.randn(C, generator=g).to(dt) if post else None,
         "w_pre": torch.randn(C, generator=g).to(dt) if pre else None}
    dev = {k: None if t is None else t.cuda() for k, t in v.items()}
    host = {k: None if t is None else t.double().numpy() for k, t in v.items()}
    if gate == "channel":
        host["gate"] = host["gate"].reshape(1, C)
    return dev, host


def sizes(v, alpha, dh=None, dx=None):
    """Magnitudes that go into each output: the formulas with |.| of every term."""
    f = ref.norm_forward(**v, alpha=alpha, eps=EPS)
    s = {"h2": np.abs(v["h"])}
    g = 1.0 if v["gate"] is None else np.abs(v["gate"])
    if v["y"] is not None:
        s["h2"] = s["h2"] + abs(alpha) * g * np.abs(f["u"])
    if v["w_pre"] is not None:
        s["x"] = s["h2"] * f["rh"] * np.abs(v["w_pre"])
    if dh is None and dx is None:
        return f, s
    t = 0.0 if dh is None else np.abs(dh)
    if dx is not None:
        n, p = s["h2"] * f["rh"], np.abs(dx * v["w_pre"])
        t = t + f["rh"] * (p + n * np.mean(p * n, axis=1, keepdims=True))
        s["dw_pre"] = np.sum(np.abs(dx) * n, axis=0)
    s["dh"] = t + np.zeros_like(v["h"])
    if v["y"] is not None:
        du = abs(alpha) * g * s["dh"]
        s["dy"] = du
        if v["w_post"] is not None:
            m, q = np.abs(v["y"]) * f["ry"], du * np.abs(v["w_post"])
            s["dy"] = f["ry"] * (q + m * np.mean(q * m, axis=1, keepdims=True))
            s["dw_post"] = np.sum(du * m, axis=0)
        dg = abs(alpha) * np.abs(f["u"]) * s["dh"]
        s["dgate"] = {"e": dg, "c": np.sum(dg, axis=0, keepdims=True),
                      "t": np.sum(dg, axis=1, keepdims=True)}
    return f, s


SHAPES = [(1, 8), (1, 4096), (3, 136), (5, 264), (2, 8192), (2, 16384), (40, 1032), (300, 512),
          (700, 2056), (400, 4096), (330, 12304)]


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("gate,post,pre", [(None, False, True), ("channel", True, True),
                                           ("token", False, False), ("element", True, True),
                                           ("token", True, True), (None, True, False)])
def test_forward_and_gradients(tg, T, C, name, gate, post, pre):
    dev, v = make(T, C, name, gate, post, pre)
    alpha = 0.7
    r = tg.norm_residual(**dev, alpha=alpha, eps=EPS, save_rstd=True)
    g = torch.Generator().manual_seed(T)
    dh = torch.randn((T, C), generator=g).to(TYPES[name])
    dx = torch.randn((T, C), generator=g).to(TYPES[name]) if pre else None
    hd, hx = dh.double().numpy(), dx.double().numpy() if pre else None
    f, s = sizes(v, alpha, hd, hx)
    near(r.h, f["h2"], s["h2"], name, "h")
    if pre:
        near(r.x, f["x"], s["x"], name, "x")
        near(r.rstd_pre, f["rh"], f["rh"], "f32", "rstd_pre")
    else:
        assert r.x is None and r.rstd_pre is None
    if post:
        near(r.rstd_post, f["ry"], f["ry"], "f32", "rstd_post")
    d = tg.norm_residual_backward(**dev, dh=dh.cuda(), dx=None if dx is None else dx.cuda(),
                                  alpha=alpha, rstd_post=r.rstd_post, rstd_pre=r.rstd_pre)
    want = ref.norm_backward(v["h"], hd, hx, **{k: v[k] for k in v if k != "h"}, alpha=alpha, eps=EPS)
    near(d.dh, want["dh"], s["dh"], name, "dh")
    near(d.dy, want["dy"], s["dy"], name, "dy")
    if post:
        near(d.dw_post, want["dw_post"], s["dw_post"], "f32", "dw_post")
    if pre:
        near(d.dw_pre, want["dw_pre"], s["dw_pre"], "f32", "dw_pre")
    if gate is not None:
        assert d.dgate.shape == dev["gate"].shape
        kind = name if gate == "element" else "f32"
        near(d.dgate, want["dgate"], s["dgate"][gate[0]], kind, "dgate")
    tg.check()


@pytest.mark.parametrize("T,C", [(1, 256), (700, 1032)])
def test_first_norm_without_a_block(tg, T, C):
    dev, v = make(T, C, "bf16", None, False, True, y=False)
    r = tg.norm_residual(dev["h"], w_pre=dev["w_pre"], eps=EPS, save_rstd=True)
    f, s = sizes(v, 1.0, None, np.ones((T, C)))
    assert r.h is dev["h"]
    near(r.x, f["x"], s["x"], "bf16", "x")
    dx = torch.ones((T, C), dtype=torch.bfloat16, device="cuda")
    d = tg.norm_residual_backward(dev["h"], dx=dx, w_pre=dev["w_pre"], rstd_pre=r.rstd_pre)
    want = ref.norm_backward(v["h"], None, np.ones((T, C)), w_pre=v["w_pre"], eps=EPS)
    near(d.dh, want["dh"], s["dh"], "bf16", "dh")
    near(d.dw_pre, want["dw_pre"], s["dw_pre"], "f32", "dw_pre")
    assert d.dy is None and d.dgate is None and d.dw_post is None


@pytest.mark.parametrize("T,C", [(1, 8), (1, 4096), (5, 136), (33, 1032), (700, 520), (400, 8192)])
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_quantised_output(tg, T, C, name):
    """Codes times scales are x to within half an e4m3 step (2^-4 of the value,
    2^-10 of the scale below the normal range) of the FP32 x; the scale is the
    block's largest magnitude / 448."""
    dev, v = make(T, C, name, "channel", True, True)
    r = tg.norm_residual(**dev, alpha=0.5, eps=EPS, quantize=True)
    f, s = sizes(v, 0.5)
    near(r.h, f["h2"], s["h2"], name, "h")
    blocks = -(-C // 128)
    pad = lambda a: np.pad(a, ((0, 0), (0, blocks * 128 - C))).reshape(T, blocks, 128)  # noqa: E731
    amax, size = pad(np.abs(f["x"])).max(axis=2), pad(s["x"]).max(axis=2)
    got = r.scales.double().cpu().numpy()
    assert r.scales.shape == (T, blocks)
    assert np.all(np.abs(got - amax / 448) <= 2.0 ** -23 * got + STEP * size / 448)
    q = r.x.double().cpu().numpy()
    scale = np.repeat(got, 128, axis=1)[:, :C]
    bound = 2.0 ** -4 * np.abs(f["x"]) + 2.0 ** -10 * scale + 2 * STEP * s["x"]
    assert np.all(np.abs(q * scale - f["x"]) <= bound)
    # and the codes are those of quantising the same x, but where it is near a tie
    want_q, _ = ref.quantize(f["x"], 1)
    assert np.mean(r.x.view(torch.uint8).cpu().numpy() != want_q) < 1e-2
    tg.check()


def test_zero_rows_and_masked_values(tg):
    """A row of zeros has x = 0 and finite gradients; NaN and infinities stay in
    their rows."""
    T, C = 6, 264
    dev, _ = make(T, C, "bf16", "token", True, True)
    dev["h"][1] = 0
    dev["y"][1] = 0
    dev["y"][2, 5] = float("nan")
    dev["h"][3, 7] = float("inf")
    dev["gate"][4] = 0
    r = tg.norm_residual(**dev, eps=EPS, save_rstd=True)
    assert torch.all(r.h[1] == 0) and torch.all(r.x[1] == 0)
    assert torch.isnan(r.h[2]).all() and torch.isnan(r.x[2]).all()
    assert torch.isinf(r.h[3, 7]) and torch.isnan(r.x[3, 7])
    assert torch.equal(r.h[4], dev["h"][4])
    good = [0, 1, 4, 5]
    assert torch.isfinite(r.x[good]).all()
    dh = torch.ones((T, C), dtype=torch.bfloat16, device="cuda")
    d = tg.norm_residual_backward(**dev, dh=dh, dx=dh, rstd_post=r.rstd_post, rstd_pre=r.rstd_pre)
    assert torch.isfinite(d.dh[good]).all() and torch.isfinite(d.dy[good]).all()
    assert torch.all(d.dy[4] == 0) and torch.isfinite(d.dgate[good]).all()
    tg.check()


def test_no_rows(tg):
    C = 264
    w = torch.ones(C, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, C), dtype=torch.bfloat16, device="cuda")
    r = tg.norm_residual(e, e, gate=w, w_post=w, w_pre=w, save_rstd=True)
    assert r.h.shape == (0, C) and r.x.shape == (0, C)
    q = tg.norm_residual(e, e, w_pre=w, quantize=True)
    assert q.x.shape == (0, C) and q.scales.shape == (0, 3)
    d = tg.norm_residual_backward(e, e, dh=e, dx=e, gate=w, w_post=w, w_pre=w,
                                  rstd_post=r.rstd_post, rstd_pre=r.rstd_pre)
    for t in (d.dgate, d.dw_post, d.dw_pre):
        assert torch.all(t == 0)      # sums over no rows


@pytest.mark.parametrize("cols", [1, 264])
@pytest.mark.parametrize("post,pre", [(True, True), (False, False)])
def test_no_rows_with_a_gate_per_row(tg, cols, post, pre):
    C = 264
    w = torch.ones(C, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, C), dtype=torch.bfloat16, device="cuda")
    gate = torch.empty((0, cols), dtype=torch.bfloat16, device="cuda")
    args = {"gate": gate, "w_post": w if post else None, "w_pre": w if pre else None}
    r = tg.norm_residual(e, e, save_rstd=True, **args)
    d = tg.norm_residual_backward(e, e, dh=e, dx=e if pre else None, rstd_post=r.rstd_post,
                                  rstd_pre=r.rstd_pre, **args)
    assert d.dgate.shape == gate.shape and d.dh.shape == d.dy.shape == (0, C)
    assert not post or torch.all(d.dw_post == 0)
    assert not pre or torch.all(d.dw_pre == 0)
    tg.check()


def test_sums_over_no_rows_are_zero_whatever_the_weights(tg):
    C = 264
    w = torch.full((C,), float("nan"), dtype=torch.bfloat16, device="cuda")
    gate = torch.full((C,), float("inf"), dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, C), dtype=torch.bfloat16, device="cuda")
    n = torch.empty(0, device="cuda")
    d = tg.norm_residual_backward(e, e, dh=e, dx=e, gate=gate, w_post=w, w_pre=w, rstd_post=n,
                                  rstd_pre=n)
    for t in (d.dgate, d.dw_post, d.dw_pre):
        assert torch.all(t == 0)


@pytest.mark.parametrize("T", [1, 2, 5])
def test_gate_gradient_type_goes_by_the_gates_shape(tg, T):
    """Whatever the number of tokens; (1, C) names a gate per element of one token."""
    C = 264
    dt = torch.bfloat16
    h = torch.randn((T, C), device="cuda").to(dt)
    for shape, kind in (((C,), torch.float32), ((T, 1), torch.float32), ((T, C), dt)):
        d = tg.norm_residual_backward(h, h, dh=h, gate=torch.ones(shape, device="cuda", dtype=dt))
        assert d.dgate.dtype == kind and d.dgate.shape == shape, shape
    if T > 1:
        row = torch.ones((1, C), device="cuda", dtype=dt)
        for call in (lambda: tg.norm_residual(h, h, gate=row),
                     lambda: tg.norm_residual_backward(h, h, dh=h, gate=row)):
            with pytest.raises(ValueError, match="gate must be"):
                call()


def test_gradients_repeat_their_bits(tg):
    dev, _ = make(2000, 1032, "f16", "channel", True, True)
    r = tg.norm_residual(**dev, save_rstd=True)
    dh = torch.randn((2000, 1032), device="cuda").half()
    runs = [tg.norm_residual_backward(**dev, dh=dh, dx=dh, rstd_post=r.rstd_post,
                                      rstd_pre=r.rstd_pre) for _ in range(4)]
    for d in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(d, runs[0]))


def test_backward_refuses_a_small_workspace(tg):
    import ctypes
    dev, _ = make(10, 264, "bf16", None, True, True)
    r = tg.norm_residual(**dev, save_rstd=True)
    need = tg.lib().norm_residual_backward_workspace_size(10, 264)
    t = torch.zeros((10, 264), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(264, device="cuda")
    p = tg.TmagemmNorm(10, 264, 1, 0, 1.0, 1e-6, dev["h"].data_ptr(), dev["y"].data_ptr(), None,
                       dev["w_post"].data_ptr(), dev["w_pre"].data_ptr(), r.rstd_post.data_ptr(),
                       r.rstd_pre.data_ptr())
    p.dh_out = p.dx = p.dh = p.dy = t.data_ptr()
    p.dw_post = p.dw_pre = w.data_ptr()
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for ptr, size in ((None, need), (ws.data_ptr(), need - 1), (ws.data_ptr() + 4, need)):
        s = tg.lib().norm_residual_backward(ctypes.byref(p), ptr, size, None)
        assert s == tg.TMAGEMM_ERR_WORKSPACE


def test_rows_past_32_bit_offsets(tg):
    T, C = 140000, 16384
    h = torch.zeros((T, C), device="cuda", dtype=torch.bfloat16)
    rows = [0, 65536, 131072, T - 1]
    g = torch.Generator(device="cuda").manual_seed(2)
    for r in rows:
        h[r] = torch.randn(C, device="cuda", generator=g).bfloat16()
    w = torch.ones(C, device="cuda", dtype=torch.bfloat16)
    r = tg.norm_residual(h, h, w_pre=w, alpha=1.0, eps=EPS)
    hv = h[rows].double().cpu().numpy()
    f = ref.norm_forward(hv, hv, w_pre=np.ones(C), eps=EPS)
    near(r.h[rows], f["h2"], np.abs(f["h2"]), "bf16", "h")
    near(r.x[rows], f["x"], np.abs(f["x"]), "bf16", "x")
    assert not r.x[1:65536].any()


def test_other_stream_than_the_current(tg):
    dev, _ = make(300, 1032, "bf16", "element", True, True)
    dh = torch.randn((300, 1032), device="cuda").bfloat16()
    want = tg.norm_residual(**dev, save_rstd=True)
    grads = tg.norm_residual_backward(**dev, dh=dh, dx=dh, rstd_post=want.rstd_post,
                                      rstd_pre=want.rstd_pre)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        r = tg.norm_residual(**dev, save_rstd=True, stream=side)
        d = tg.norm_residual_backward(**dev, dh=dh, dx=dh, rstd_post=r.rstd_post,
                                      rstd_pre=r.rstd_pre, stream=side)
        torch.empty((300, 1032), device="cuda", dtype=torch.bfloat16).fill_(9.0)
        side.synchronize()
        assert torch.equal(r.x, want.x) and all(torch.equal(a, b) for a, b in zip(d, grads))


@pytest.mark.parametrize("T,C", [(1, 264), (300, 1032)])
@pytest.mark.parametrize("gate,post,pre", [(None, True, False), ("token", True, False),
                                           ("channel", True, True), ("element", False, True)])
def test_gradients_without_one_of_the_residual_stream(tg, T, C, gate, post, pre):
    """No dh (the residual stream ends here): with w_pre the gradients are those of x
    alone, without it they are all zero."""
    dev, v = make(T, C, "bf16", gate, post, pre)
    r = tg.norm_residual(**dev, alpha=0.7, eps=EPS, save_rstd=True)
    g = torch.Generator().manual_seed(T)
    dx = torch.randn((T, C), generator=g).to(torch.bfloat16) if pre else None
    hx = dx.double().numpy() if pre else None
    d = tg.norm_residual_backward(**dev, dx=dx.cuda() if pre else None, alpha=0.7,
                                  rstd_post=r.rstd_post, rstd_pre=r.rstd_pre)
    if not pre:
        assert all(t is None or torch.all(t == 0) for t in d)
        return
    _, s = sizes(v, 0.7, None, hx)
    want = ref.norm_backward(v["h"], None, hx, **{k: v[k] for k in v if k != "h"}, alpha=0.7, eps=EPS)
    near(d.dh, want["dh"], s["dh"], "bf16", "dh")
    near(d.dy, want["dy"], s["dy"], "bf16", "dy")
    near(d.dw_pre, want["dw_pre"], s["dw_pre"], "f32", "dw_pre")
    if post:
        near(d.dw_post, want["dw_post"], s["dw_post"], "f32", "dw_post")
    near(d.dgate, want["dgate"], s["dgate"][gate[0]], "bf16" if gate == "element" else "f32", "dgate")


def test_graph_follows_its_inputs(tg):
    """A captured forward and backward replayed on other inputs give what calls give."""
    dev, _ = make(300, 1032, "bf16", "channel", True, True)
    dh = torch.randn((300, 1032), device="cuda").bfloat16()

    def step():
        r = tg.norm_residual(**dev, save_rstd=True)
        q = tg.norm_residual(**dev, quantize=True)
        d = tg.norm_residual_backward(**dev, dh=dh, dx=dh, rstd_post=r.rstd_post,
                                      rstd_pre=r.rstd_pre)
        return [r.h, r.x, q.x.view(torch.uint8), q.scales, *d]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in (dev["h"], dev["y"], dev["gate"], dh):
            t.copy_(torch.randn_like(t))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_gradients_past_32_bit_offsets(tg):
    """Six operands of 2.3e9 values; only a few rows, some past 2^31 values, are not zero,
    so the column sums are those rows' sums."""
    T, C = 140000, 16384
    rows = [0, 65536, 131072, T - 1]
    g = torch.Generator(device="cuda").manual_seed(3)

    def sparse():
        t = torch.zeros((T, C), device="cuda", dtype=torch.bfloat16)
        for r in rows:
            t[r] = torch.randn(C, device="cuda", generator=g).bfloat16()
        return t

    h, y, dh, dx = (sparse() for _ in range(4))
    w = torch.randn((2, C), device="cuda", generator=g).bfloat16()
    r = tg.norm_residual(h, y, w_post=w[0], w_pre=w[1], eps=EPS, save_rstd=True)
    d = tg.norm_residual_backward(h, y, dh=dh, dx=dx, w_post=w[0], w_pre=w[1],
                                  rstd_post=r.rstd_post, rstd_pre=r.rstd_pre)
    host = lambda t: t[rows].double().cpu().numpy()  # noqa: E731
    v = {"h": host(h), "y": host(y), "gate": None, "w_post": w[0].double().cpu().numpy(),
         "w_pre": w[1].double().cpu().numpy()}
    _, s = sizes(v, 1.0, host(dh), host(dx))
    want = ref.norm_backward(v["h"], host(dh), host(dx), y=v["y"], w_post=v["w_post"],
                             w_pre=v["w_pre"], eps=EPS)
    near(d.dh[rows], want["dh"], s["dh"], "bf16", "dh")
    near(d.dy[rows], want["dy"], s["dy"], "bf16", "dy")
    near(d.dw_post, want["dw_post"], s["dw_post"], "f32", "dw_post")
    near(d.dw_pre, want["dw_pre"], s["dw_pre"], "f32", "dw_pre")
    assert not d.dh[1:65536].any() and not d.dy[131073:T - 1].any()
