"""GPU tests of route_topk and its gradient against 64-bit references.

Bounds: a weight is a quotient of exponentials, whose arguments (differences of logits)
are rounded by 2^-24 of their size, which is a relative error of that many steps times the
size; expf, sums in trees, quotient and products add under 40 steps of 2^-24.  Gradients
have the magnitudes of their terms in the place of the weight, and a rounding to the
logits' type."""
import numpy as np
import pytest

from tests import experts_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -140}


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def spread(logits):
    finite = np.where(np.isfinite(logits), logits, np.nan)
    with np.errstate(all="ignore"):
        wide = np.nanmax(finite, axis=1) - np.nanmin(finite, axis=1) + np.nanmax(np.abs(finite), axis=1)
    return np.nan_to_num(wide)[:, None]


def check(tg, logits, k, seed=0, gradient=True, **kw):
    """Forward and backward of torch logits against the references."""
    l = logits.double().cpu().numpy()
    bias = kw.pop("bias", None)
    r = tg.route_topk(logits, k, bias=bias, **kw)
    ids, weights = ref.route(l, k, bias=None if bias is None else bias.double().cpu().numpy(), **kw)
    assert r.ids.dtype == torch.int32 and r.weights.dtype == torch.float32
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    steps = (40 + 2 * spread(l)) * 2.0 ** -24
    got = r.weights.double().cpu().numpy()
    assert np.all(np.abs(got - weights) <= steps * np.abs(weights) + 2.0 ** -140)
    if not gradient:
        return r
    g = torch.Generator().manual_seed(seed)
    dw = torch.randn((l.shape[0], k), generator=g)
    same = {n: kw[n] for n in ("score", "renormalize", "scale") if n in kw}
    d = tg.route_topk_backward(logits, r.ids, dw.cuda(), **same)
    assert d.dtype == logits.dtype and d.shape == logits.shape
    want, size = ref.route_gradient(l, ids, dw.double().numpy(), same.get("score", "softmax"),
                                    same.get("renormalize", True), same.get("scale", 1.0))
    kind = {v: n for n, v in TYPES.items()}[logits.dtype]
    bound = HALF[kind] * np.abs(want) + 2 * steps * size + TINY[kind]
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= bound)
    return r


def make(T, E, name, seed=0, size=1.5):
    g = torch.Generator().manual_seed(seed + 31 * T + E)
    return (size * torch.randn((T, E), generator=g)).to(TYPES[name]).cuda()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 2, 2), (7, 33, 5), (20, 122, 6),
                                   (9, 128, 1), (40, 256, 8), (5, 511, 32), (8, 512, 10)])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize,scale", [(True, 2.5), (False, 1.0)])
def test_route_and_gradient(tg, T, E, k, name, score, renormalize, scale):
    check(tg, make(T, E, name), k, score=score, renormalize=renormalize, scale=scale)


@pytest.mark.parametrize("E,k,groups,top_groups", [
    (256, 8, 8, 4), (64, 6, 8, 3), (160, 6, 8, 3), (12, 4, 6, 3), (8, 2, 8, 2), (330, 8, 3, 2),
    (510, 20, 17, 5), (512, 32, 32, 2), (62, 4, 31, 30), (16, 16, 1, 1), (40, 9, 5, 5)])
@pytest.mark.parametrize("group_sum", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_and_bias(tg, E, k, groups, top_groups, group_sum, score, biased):
    g = torch.Generator().manual_seed(E + k)
    bias = (0.1 * torch.randn(E, generator=g)).cuda() if biased else None
    for name in ("f32", "bf16"):
        check(tg, make(50, E, name), k, score=score, bias=bias, groups=groups,
              top_groups=top_groups, group_sum=group_sum, gradient=False)


@pytest.mark.parametrize("T", [1, 8, 9, 4100])
def test_token_counts(tg, T):
    check(tg, make(T, 60, "bf16"), 4)
    check(tg, make(T, 60, "f32"), 4, score="sigmoid", bias=torch.linspace(-1, 1, 60).cuda(),
          groups=4, top_groups=2, group_sum=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(tg, score):
    logits = torch.zeros((6, 96), device="cuda")
    logits[1, 50:] = 1.0
    logits[2, ::3] = -0.0
    logits[3, [95, 4, 40]] = 2.0
    logits[4] = -30.0
    logits[5, 7] = 5.0
    for kw in ({}, dict(bias=torch.zeros(96, device="cuda")),
               dict(groups=8, top_groups=3, group_sum=2), dict(groups=8, top_groups=8, group_sum=1)):
        check(tg, logits, 7, score=score, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
def test_values_that_32_bits_cannot_tell_apart(tg, score, groups, top_groups):
    """Biases that make all of p + bias nearly equal: the order is that of 64 bits."""
    T, E = 24, 128
    logits = make(1, E, "f32", size=2.0).expand(T, E).contiguous()
    p = ref.scores(logits.double().cpu().numpy(), score)
    bias = torch.from_numpy((0.7 - p[0]).astype(np.float32)).cuda()
    far = torch.arange(T, device="cuda")[:, None] * 1e-9 * torch.randn((T, E), device="cuda")
    logits = logits + far.float()
    v = ref.scores(logits.double().cpu().numpy(), score) + bias.double().cpu().numpy()
    assert np.ptp(v, axis=1).max() < 1e-6
    check(tg, logits, 8, score=score, bias=bias, groups=groups, top_groups=top_groups, group_sum=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups", [(64, 8), (512, 8), (512, 32)])
def test_equal_values_across_groups(tg, score, biased, E, groups):
    """Logits of a few values only: groups whose best are equal, and more equal experts in a
    group than count for its value; with biases of two values, and next to each other's."""
    g = torch.Generator().manual_seed(E + groups)
    logits = torch.randint(0, 3, (300, E), generator=g).float()
    logits[100:200] *= 2.0 ** -22       # next to each other's in FP32
    logits[200:] = 14 + logits[200:] / 8     # sigmoid: the same FP32 score
    bias = 2.0 ** -24 * torch.randint(0, 2, (E,), generator=g).float() if biased else None
    for kind in (logits, logits.bfloat16()):
        check(tg, kind.cuda(), 6, score=score, bias=None if bias is None else bias.cuda(),
              groups=groups, top_groups=groups // 2, group_sum=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_sum,top_groups", [(0, 0), (1, 3), (2, 3), (2, 5)])
def test_pairs_that_32_bits_cannot_tell_apart(tg, score, group_sum, top_groups):
    """Runs of eight experts in pairs whose values are equal to FP32 rounding, one run far
    from the next: neighbours in doubt, and groups, with the rest well apart."""
    T, E = 200, 64
    logits = make(1, E, "f32", seed=3).expand(T, E).contiguous()
    p = ref.scores(logits.double().cpu().numpy(), score)[0]
    v = p + 0.25 * np.arange(E) / E
    for g in range(1, 8, 2):
        v[8 * g:8 * g + 8] = v[8 * g - 8:8 * g]
    bias = torch.from_numpy((v - p).astype(np.float32)).cuda()
    logits = logits + (1e-7 * torch.randn((T, E), device="cuda"))
    kw = dict(groups=8, top_groups=top_groups, group_sum=group_sum) if group_sum else {}
    check(tg, logits, 7, score=score, bias=bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_closed_experts(tg, score, renormalize):
    """-inf closes an expert, whatever its bias; a token without any gets ids of -1."""
    logits = make(6, 40, "f32")
    inf = float("inf")
    logits[0] = -inf
    logits[1, 3:] = -inf
    logits[2, ::2] = -inf
    logits[3, 20:] = -inf
    logits[4, 1:] = torch.finfo(torch.float32).min
    for kw in ({}, dict(bias=torch.arange(40, device="cuda").float()),
               dict(groups=4, top_groups=2, group_sum=2)):
        r = check(tg, logits, 5, score=score, renormalize=renormalize, **kw)
        assert (r.ids[0] == -1).all() and (r.weights[0] == 0).all()
        assert (r.ids[1, 3:] == -1).all() and (r.weights[1, 3:] == 0).all()


def test_scores_below_the_smallest_float(tg):
    """Renormalised weights of scores that FP32 cannot hold."""
    logits = make(5, 20, "f32", size=3.0) - 200.0
    logits[0, 0] = 100.0
    bias = torch.zeros(20, device="cuda")
    bias[5:9] = 10.0
    for score in ("softmax", "sigmoid"):
        check(tg, logits, 4, score=score, bias=bias)


def test_nan_shows_in_the_weights(tg):
    logits = make(3, 30, "f32")
    logits[1, 17] = float("nan")
    for kw in ({}, dict(bias=torch.zeros(30, device="cuda")), dict(score="sigmoid"),
               dict(groups=5, top_groups=2, group_sum=2)):
        r = tg.route_topk(logits, 4, **kw)
        assert torch.isnan(r.weights[1]).all() and not torch.isnan(r.weights[[0, 2]]).any()
        ids = r.ids[1].tolist()
        assert len(set(ids)) == 4 and all(0 <= i < 30 for i in ids)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False),
                                               ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(tg, score, renormalize):
    """Central differences of the 64-bit weights: h^2 of the third derivative (under 1 for
    scores) and rounding 2^-52 / h, with h = 1e-4, are under 1e-7."""
    l = make(4, 24, "f32")
    dw = torch.randn((4, 3), generator=torch.Generator().manual_seed(1))
    kw = dict(score=score, renormalize=renormalize, scale=1.5)
    r = tg.route_topk(l, 3, **kw)
    got = tg.route_topk_backward(l, r.ids, dw.cuda(), **kw).double().cpu().numpy()
    x, ids = l.double().cpu().numpy(), r.ids.cpu().numpy()
    for e in range(24):
        f = []
        for h in (1e-4, -1e-4):
            moved = x.copy()
            moved[:, e] += h
            c = np.take_along_axis(ref.scores(moved, score), ids, axis=1)
            w = 1.5 * (c / c.sum(axis=1, keepdims=True) if renormalize else c)
            f.append((w * dw.double().numpy()).sum(axis=1))
        assert np.all(np.abs((f[0] - f[1]) / 2e-4 - got[:, e]) < 1e-6)


def test_gradient_of_choices_outside_the_experts(tg):
    logits = make(2, 16, "f32")
    ids = torch.tensor([[3, -1, 16], [-1, -1, 1 << 30]], dtype=torch.int32, device="cuda")
    dw = torch.ones((2, 3), device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            d = tg.route_topk_backward(logits, ids, dw, score=score, renormalize=renormalize)
            want, size = ref.route_gradient(logits.double().cpu().numpy(), ids.cpu().numpy(),
                                            np.ones((2, 3)), score, renormalize, 1.0)
            assert np.all(np.abs(d.double().cpu().numpy() - want) <= 100 * 2.0 ** -24 * size)


def test_no_tokens(tg):
    r = tg.route_topk(torch.empty((0, 8), device="cuda"), 2)
    assert r.ids.shape == (0, 2) and r.weights.shape == (0, 2)
    d = tg.route_topk_backward(torch.empty((0, 8), device="cuda"), r.ids, r.weights)
    assert d.shape == (0, 8)


def test_refusals(tg):
    l = make(4, 8, "f32")
    bad = [(ValueError, dict(k=0)), (ValueError, dict(k=9)), (ValueError, dict(groups=3)),
           (ValueError, dict(groups=4, top_groups=5)), (ValueError, dict(groups=8, top_groups=1)),
           (ValueError, dict(group_sum=3)), (TypeError, dict(bias=torch.zeros(8, device="cuda").half())),
           (ValueError, dict(bias=torch.zeros(7, device="cuda"))), (TypeError, dict(bias=torch.zeros(8)))]
    for error, kw in bad:
        with pytest.raises(error):
            tg.route_topk(l, **{"k": 2, **kw})
    with pytest.raises(TypeError):
        tg.route_topk(l.double(), 2)
    with pytest.raises(ValueError):
        tg.route_topk(make(8, 4, "f32").t(), 2)
    with pytest.raises(ValueError):
        tg.route_topk(l[0], 2)
    r = tg.route_topk(l, 2)
    with pytest.raises(TypeError):
        tg.route_topk_backward(l, r.ids.long(), r.weights)
    with pytest.raises(ValueError):
        tg.route_topk_backward(l, r.ids, r.weights[:3])
    with pytest.raises(tg.TmaGemmError):
        tg.route_topk(make(2, 513, "f32"), 2)
