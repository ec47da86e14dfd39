"""GPU tests of renormalised weights where one choice has all of the sum: the weight is the
scale and its gradient zero, exactly (a number divided by itself is 1)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("k", [1, 4])
def test_one_choice(tg, score, name, k):
    """k = 1, and tokens with one open expert for more."""
    T, E = 5000, 20
    g = torch.Generator().manual_seed(k)
    logits = 6.0 * torch.randn((T, E), generator=g)
    if k > 1:
        logits[:, 1:] = -float("inf")
    logits = logits.to(getattr(torch, name)).cuda()
    dw = torch.randn((T, k), generator=g).cuda()
    for bias in (None, torch.linspace(-1, 1, E).cuda()):
        r = tg.route_topk(logits, k, score=score, bias=bias, scale=2.5)
        assert (r.ids[:, 0] >= 0).all() and (r.ids[:, 1:] == -1).all()
        assert (r.weights[:, 0] == 2.5).all() and (r.weights[:, 1:] == 0.0).all()
        d = tg.route_topk_backward(logits, r.ids, dw, score=score, scale=2.5)
        assert (d == 0.0).all()
