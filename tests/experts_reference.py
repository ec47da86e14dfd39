"""Plain references of the router, the rows of experts and the 4-bit products, in 64
bits (numpy), written from their definitions and sharing no code with the library."""
import numpy as np


def scores(logits, score):
    """softmax or sigmoid of float64 logits (closed experts, -inf, get 0)."""
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "softmax":
            e = np.exp(logits - logits.max(axis=1, keepdims=True))
            p = e / e.sum(axis=1, keepdims=True)
            return np.where(np.isneginf(logits).all(axis=1, keepdims=True), 0.0, p)
        return 1.0 / (1.0 + np.exp(-logits))


def best(values, count):
    """Indices of the largest values, largest first, ties to the lowest index; those at
    -inf are left out."""
    order = [i for i in np.argsort(-values, kind="stable") if values[i] != -np.inf]
    return order[:count]


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_sum=1,
          renormalize=True, scale=1.0):
    """(ids, weights) of float64 logits without NaN."""
    T, E = logits.shape
    p = scores(logits, score)
    v = np.where(np.isneginf(logits), -np.inf, p + (0.0 if bias is None else bias))
    ids, weights = np.full((T, k), -1), np.zeros((T, k))
    size = E // groups
    for t in range(T):
        values = v[t].copy()
        if groups > 1:
            sums = np.full(groups, -np.inf)
            for g in range(groups):
                part = values[g * size:(g + 1) * size]
                top = best(part, group_sum)
                if top:
                    sums[g] = part[top].sum()
            keep = best(sums, top_groups)
            for g in range(groups):
                if g not in keep:
                    values[g * size:(g + 1) * size] = -np.inf
        chosen = best(values, k)
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if renormalize:
            # score ratios by logits, so that none of them vanishes
            l = logits[t, chosen]
            if score == "sigmoid":
                l = -np.logaddexp(0.0, -l)
            c = np.exp(l - l.max())
            c /= c.sum()
        else:
            c = p[t, chosen]
        weights[t, :len(chosen)] = scale * c
    return ids, weights


def route_gradient(logits, ids, dweights, score, renormalize, scale):
    """(dlogits, size): the gradient with the choice held fixed, and the sum of the
    magnitudes of its terms."""
    T, E = logits.shape
    p = scores(logits, score)
    d, s = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not at:
            continue
        e = ids[t, at]
        if renormalize:
            l = logits[t, e]
            if score == "sigmoid":
                l = -np.logaddexp(0.0, -l)
            share = np.exp(l - l.max())
            share /= share.sum()
        else:
            share = p[t, e]
        part = scale * dweights[t, at] * share          # dw_j w_j
        dt, st = np.zeros(E), np.zeros(E)
        dt[e] += part
        st[e] += np.abs(part)
        if score == "softmax" and not renormalize:
            dt -= p[t] * part.sum()
            st += p[t] * np.abs(part).sum()
        elif renormalize:
            dt[e] -= share * part.sum()
            st[e] += share * np.abs(part).sum()
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                f = np.where(np.isneginf(logits[t]), 1.0, 1.0 / (1.0 + np.exp(logits[t])))
            dt, st = dt * f, st * f
        d[t], s[t] = dt, st
    return d, s


def dispatch(ids, experts):
    """(offsets, row_of, slots): slots in the order of their rows."""
    flat = ids.ravel()
    slots = [s for e in range(experts) for s in np.flatnonzero(flat == e)]
    row_of = np.full(len(flat), -1)
    row_of[slots] = np.arange(len(slots))
    counts = [int((flat == e).sum()) for e in range(experts)]
    return (np.concatenate([[0], np.cumsum(counts)]).astype(np.int64), row_of.reshape(ids.shape),
            np.asarray(slots, dtype=np.int64))


def weights_w4(codes, scales, zeros, group):
    """(N, K) float64 weights of packed codes (N, K / 2)."""
    N, half = codes.shape
    q = np.empty((N, 2 * half))
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    at = np.arange(2 * half) // group
    return (q - (8.0 if zeros is None else zeros.astype(np.float64)[:, at])) * scales[:, at]


def w4_bound(ref, size, K, group, bf16):
    """What a 4-bit product may be off: half a step of its type (2^-8 of a bf16 value,
    2^-11 of an fp16 one), and for each addition of partial sums in FP32 -- 16 k at a
    time, a group, up to 16 parts of K and 4 of a cluster -- 2^-23 of the terms'
    magnitudes (the tensor cores may truncate), doubled for the additions within."""
    half = 2.0 ** -8 if bf16 else 2.0 ** -11
    steps = -(-K // 16) + -(-K // group) + 20
    return half * np.abs(ref) + steps * 2.0 ** -22 * size + (2.0 ** -134 if bf16 else 2.0 ** -25)
