"""GPU tests of route_topk's order where FP32 cannot tell values apart, where they are
infinite, and where scores are all but 1: the ids are those of 64 bits."""
import itertools

import numpy as np
import pytest

from tests import experts_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def tg():
    import tma_pipelined_tensor_tn_gb300 as m
    m.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def ordered(values, count):
    """The lowest indices of the largest values that are not None, largest first."""
    open_ = [i for i, v in enumerate(values) if v is not None]
    return sorted(open_, key=lambda i: (-values[i], i))[:count]


def choose(logits, values, k, groups=1, top_groups=1, group_sum=1):
    """ids (T, k) by float64 values; a logit of -inf closes, a value of -inf does not."""
    T, E = logits.shape
    ids, size = np.full((T, k), -1), E // groups
    for t in range(T):
        v = [None if np.isneginf(l) else float(x) for l, x in zip(logits[t], values[t])]
        if groups > 1:
            sums = []
            for g in range(groups):
                part = v[g * size:(g + 1) * size]
                best = ordered(part, group_sum)
                sums.append(sum(part[i] for i in best) if best else None)
            keep = ordered(sums, top_groups)
            v = [x if e // size in keep else None for e, x in enumerate(v)]
        best = ordered(v, k)
        ids[t, :len(best)] = best
    return ids


def check(tg, logits, k, score, bias, values=None, **groups):
    """The ids against those of 64 bits (or by the values given), and the weights."""
    l = logits.double().cpu().numpy()
    if values is None:
        values = ref.scores(l, score) + (0.0 if bias is None else bias.double().cpu().numpy())
    want = choose(l, values, k, **groups)
    r = tg.route_topk(logits, k, score=score, bias=bias, **groups)
    ids = r.ids.cpu().numpy()
    assert np.array_equal(ids, want), np.flatnonzero((ids != want).any(axis=1))[:10]
    have = want >= 0
    c = np.where(have, np.take_along_axis(ref.scores(l, score), np.maximum(want, 0), axis=1), 0.0)
    # (Scores of these tests are far from the smallest numbers; the bound is that of
    # test_gpu_route.py with logits up to 100 apart.)
    share = c / np.where(have.any(axis=1), c.sum(axis=1), 1.0)[:, None]
    assert np.all(np.abs(r.weights.double().cpu().numpy() - share) <= 300 * 2.0 ** -24 * share)


# ------------------------------------------- ties in front of a larger value ----

@pytest.mark.parametrize("score,logits,bias,k,expect", [
    ("sigmoid", (20.0, 20.0, 21.0, -5.0), 0.0, 1, [2]),
    ("sigmoid", (-17.0, -17.0, -16.5, -20.0), 0.5, 1, [2]),
    ("sigmoid", (20.0, 20.0, 20.0, 20.0, 21.0, 20.5), 0.0, 2, [4, 5]),
    ("sigmoid", (30.0, 20.0, 20.0, 20.0, 21.0, 30.0), 0.0, 3, [0, 5, 4]),
    ("softmax", (0.0, -17.0, -17.0, -16.5, -20.0), 0.5, 2, [0, 3]),
    ("softmax", (0.0, -17.0, -17.0, -17.0, -16.5, -16.0), 0.5, 3, [0, 5, 4])])
def test_ties_across_the_last_choice(tg, score, logits, bias, k, expect):
    """The k-th and the next are equal, and one behind them is larger by less than FP32
    shows."""
    l = torch.tensor([logits], device="cuda")
    b = torch.full((len(logits),), bias, device="cuda")
    assert tg.route_topk(l, k, score=score, bias=b).ids.tolist() == [expect]
    check(tg, l, k, score, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [(6, 1, 1), (20, 1, 1), (64, 1, 1), (64, 8, 3),
                                                 (330, 1, 1)])
@pytest.mark.parametrize("k", [1, 2, 5])
def test_runs_of_ties(tg, score, E, groups, top_groups, k):
    """Logits of a few values whose scores FP32 cannot tell apart next to the bias."""
    g = torch.Generator().manual_seed(E + k)
    logits = -17.0 + 0.25 * torch.randint(0, 6, (400, E), generator=g).float()
    logits[200:, ::7] = -1.0           # a few that stand out
    if score == "softmax":
        logits[:, 3] = 0.0             # so that the others stay small
    bias = torch.full((E,), 0.5)
    bias[E // 2] += 2.0 ** -24
    kw = dict(groups=groups, top_groups=top_groups, group_sum=1) if groups > 1 else {}
    for kind in (logits, logits.bfloat16()):
        check(tg, kind.cuda(), k, score, bias.cuda(), **kw)


# ------------------------------------------------------------ infinite biases ----

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k,forced", [(1, 1), (1, 5), (4, 1), (4, 3), (4, 4), (4, 5), (4, 40),
                                      (8, 64), (32, 33), (32, 32)])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_biases(tg, score, k, forced, sign):
    """+inf on fewer than, exactly and more than k experts puts these first, -inf on any
    number of them last, in the order of their indices."""
    E, rng = 64, np.random.default_rng(k + forced)
    logits = torch.from_numpy(rng.normal(size=(20, E))).float().cuda()
    logits[3, 1:] = -INF
    bias = torch.from_numpy(0.1 * rng.normal(size=E)).float()
    bias[torch.from_numpy(rng.permutation(E)[:forced])] = sign * INF
    for group in ({}, dict(groups=8, top_groups=4, group_sum=1)):
        check(tg, logits, k, score, bias.cuda(), **group)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_sum", [1, 2])
def test_infinite_biases_of_some_groups(tg, score, group_sum):
    """Groups with one, two or only experts at +inf or at -inf (never both in one)."""
    E, rng = 48, np.random.default_rng(group_sum)
    logits = torch.from_numpy(rng.normal(size=(50, E))).float().cuda()
    for high, low in itertools.product(((), (7,), (7, 9), (40, 41, 42), (7, 21, 40)),
                                       ((), (25,), tuple(range(24, 32)), tuple(range(25, 32)))):
        bias = 0.1 * torch.from_numpy(rng.normal(size=E)).float()
        bias[list(high)] = INF
        bias[list(low)] = -INF
        for top_groups in (1, 2, 5):
            check(tg, logits, 4, score, bias.cuda(), groups=6, top_groups=top_groups,
                  group_sum=group_sum)


# --------------------------------------------- groups whose two best cancel out ----

def test_sum_that_cancels(tg):
    l = torch.tensor([[1.4e-5, 0.0, 1.65e-5, -1.4e-5]], device="cuda")
    b = torch.tensor([100.0, -100.0, 100.0, -100.0], device="cuda")
    kw = dict(groups=2, top_groups=1, group_sum=2)
    assert tg.route_topk(l, 1, score="sigmoid", bias=b, **kw).ids.tolist() == [[0]]
    check(tg, l, 1, "sigmoid", b, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 32.0, 100.0, 1000.0])
@pytest.mark.parametrize("E,groups", [(16, 4), (512, 8), (256, 32)])
def test_group_sums_of_opposite_biases(tg, score, size, E, groups):
    """The two best of each group have biases of +-size, so that the groups' sums hold the
    scores' differences and the rounding of the biases' size: a few 1e-6 apart."""
    T, g = 300, torch.Generator().manual_seed(E)
    per = E // groups
    logits = 1e-5 * torch.randn((T, E), generator=g)
    if score == "softmax":
        logits *= E                    # scores of 1 / E: the same differences
    bias = torch.full((E,), -4.0 * size)
    bias[0::per], bias[per - 1::per] = size, -size
    for top_groups in (1, groups // 2):
        check(tg, logits.cuda(), 2, score, bias.cuda(), groups=groups, top_groups=top_groups,
              group_sum=2)


# -------------------------------------------------------------- scores near 1 ----

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_without_a_bias_by_logits(tg, score, name):
    """Without a bias experts are in the order of their logits, also where their scores are
    the same number in 64 bits, and whatever the groups are valued by."""
    T, E, groups = 100, 64, 4
    g = torch.Generator().manual_seed(0)
    logits = 40.0 + 20.0 * torch.rand((T, E), generator=g)
    logits[50:] -= 800.0 * torch.rand((50, E), generator=g)
    logits = logits.to(getattr(torch, name)).cuda()
    l = logits.double().cpu().numpy()
    check(tg, logits[:50], 4, score, None, values=l[:50])
    # (All groups are kept, so that their order does not matter.)
    for group_sum in (1, 2):
        r = tg.route_topk(logits, 4, score=score, groups=groups, top_groups=groups,
                          group_sum=group_sum)
        assert np.array_equal(r.ids.cpu().numpy(), choose(l, l, 4))
    # One group ahead of the others: the order within it.
    logits[:, :16] -= 100.0
    logits[:, 32:] -= 100.0
    l = logits.double().cpu().numpy()
    sums = np.sort(ref.scores(l, score).reshape(T, groups, -1), axis=2)[:, :, -2:].sum(axis=2)
    others = np.delete(sums, 1, axis=1).max(axis=1)
    rows = np.flatnonzero(sums[:, 1] > others + 1e-6)
    r = tg.route_topk(logits, 3, score=score, groups=groups, top_groups=1, group_sum=2)
    want = 16 + choose(l[:, 16:32], l[:, 16:32], 3)
    assert len(rows) >= 40 and np.array_equal(r.ids.cpu().numpy()[rows], want[rows])
