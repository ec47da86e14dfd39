"""Performance cases of what stands around the products of routed experts, and of
linear layers with 4-bit weights: the router's choice and its gradient, rows laid
out by expert and summed back with their gradients, and products of a few tokens
with 4-bit weights (dense and by expert).

Each case is one pass through one operator, either in its plain form (torch
operations in 32 bits, one rounding at the end) or, with ``own`` set, through
the library's entry points.  ``exact`` gives the results from the operators'
definitions in 64 bits.

Definitions:
  route     p = softmax(l) or sigmoid(l) over a token's E logits l.  Experts are
            chosen by p + bias, best first, ties to the lowest index: with groups,
            only out of the ``top_groups`` groups whose ``group_sum`` best values of
            p + bias have the largest sum.  w_j = scale p_j, divided by the sum of
            the chosen p with ``renormalize``.  Gradient: of the weights with respect
            to the logits, the choice held fixed.
  dispatch  choice j of token t (slot t k + j) goes to expert ids[t, j].  Rows are
            laid out by expert, slots of one expert in order; offsets[e] is the
            first row of expert e and row_of[t, j] the row of a slot.  A row is its
            token's x, in 16 bits or as e4m3 codes with a scale per 128 columns
            (a = max(max |x|, 2^-100), S = fl32(a / 448), Q = e4m3(fl32(x fl32(448 / a)))).
  combine   y[t] = sum_j w[t, j] rows[row_of[t, j]].
  w4        D[m, n] = sum_k A[m, k] (q[n, k] - z[n, g]) s[n, g] with g = k // group;
            q in 0 .. 15, two to a byte, the even k in the low half; z = 8 where no
            zero points are given.
"""
import math

import numpy as np
import torch

own = False

_BLOCK = 128
_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # One token decoded, a softmax over a few dozen experts: latency only.
        {"name": "route_decode", "op": "route", "T": 1, "E": 64, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_sum": 1, "renormalize": True,
         "grad": False, "type": "f32"},
        # A prompt: sigmoid scores, a bias that balances the experts, groups of them.
        {"name": "route_prompt", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_sum": 2, "renormalize": True,
         "grad": False, "type": "f32"},
        # A training step with an odd number of experts, not renormalised, so that every
        # logit has a gradient.
        {"name": "route_train", "op": "route", "T": 16384, "E": 122, "k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_sum": 1, "renormalize": False,
         "grad": True, "type": "bf16"},
        # A decode batch into the codes that the 8-bit products read.
        {"name": "dispatch_decode", "op": "dispatch", "T": 16, "C": 4096, "E": 64, "k": 4,
         "quantize": True, "skew": 1.0, "grad": False, "type": "bf16"},
        # A prompt of an odd length, quantised on the way.
        {"name": "dispatch_prompt", "op": "dispatch", "T": 4099, "C": 4096, "E": 64, "k": 8,
         "quantize": True, "skew": 0.5, "grad": False, "type": "f16"},
        # A training step: rows in 16 bits, and the gradient back to the tokens.
        {"name": "dispatch_train", "op": "dispatch", "T": 8192, "C": 2048, "E": 16, "k": 2,
         "quantize": False, "skew": 0.5, "grad": True, "type": "bf16"},
        # A decode batch summed back.
        {"name": "combine_decode", "op": "combine", "T": 16, "C": 4096, "E": 64, "k": 4,
         "skew": 1.0, "grad": False, "type": "bf16"},
        # A training step: forward, then the gradients of the rows and of the weights.
        {"name": "combine_train", "op": "combine", "T": 8192, "C": 2048, "E": 64, "k": 8,
         "skew": 0.5, "grad": True, "type": "bf16"},
        # One token decoded against a down projection: bound by reading the weights once.
        {"name": "w4_decode_1", "op": "w4", "M": 1, "N": 4096, "K": 14336, "group": 128,
         "zeros": False, "type": "bf16"},
        # A decode batch against an up projection, with zero points.
        {"name": "w4_decode_27", "op": "w4", "M": 27, "N": 14336, "K": 4096, "group": 64,
         "zeros": True, "type": "f16"},
        # Odd sizes and small groups.
        {"name": "w4_odd", "op": "w4", "M": 5, "N": 5003, "K": 2080, "group": 32, "zeros": True,
         "type": "f16"},
        # A decode batch over many experts: most get a few tokens, some none.
        {"name": "w4_experts_decode", "op": "w4_experts", "G": 64, "R": 128, "N": 4096, "K": 2048,
         "group": 128, "zeros": False, "skew": 1.0, "type": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, (v + step - 1) // step * step)


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "w4", "w4_experts"])
    t = rng.choice(["f16", "bf16"])
    if op == "route":
        grad = rng.random() < 0.4
        groups = 1 if grad else rng.choice([1, 1, 4, 8])
        E = groups * _log_int(rng, max(2, 8 // groups), 384 // groups)
        top_groups = groups if groups == 1 else rng.randint(1, groups)
        k = rng.randint(1, min(10, E // groups * top_groups))
        return {"op": op, "T": _log_int(rng, 1, 16384 * 122 // max(E, 122)), "E": E, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "top_groups": top_groups,
                "group_sum": 1 if groups == 1 else rng.choice([1, 2]),
                "renormalize": rng.random() < 0.6, "grad": grad,
                "type": rng.choice(["f32", "f32", t])}
    if op in ("dispatch", "combine"):
        E = _log_int(rng, 2, 384)
        k = rng.randint(1, min(E, 8))
        C = _log_int(rng, 256, 8192, 16)
        top = min(16384, 8192 * 8 * 2048 // (k * C))
        case = {"op": op, "T": _log_int(rng, 1, top), "C": C, "E": E, "k": k,
                "skew": rng.choice([0.0, 0.5, 1.0]), "grad": rng.random() < 0.5, "type": t}
        if op == "dispatch":
            case["quantize"] = not case["grad"] and rng.random() < 0.6
        return case
    case = {"op": op, "group": rng.choice([32, 64, 128, 128]), "zeros": rng.random() < 0.5,
            "type": t}
    if op == "w4":
        case.update(M=_log_int(rng, 1, 32), N=_log_int(rng, 128, 14336),
                    K=_log_int(rng, 256, 14336, 32))
        if case["N"] * case["K"] > 4096 * 14336:
            case["K"] = 4096
        return case
    case.update(G=_log_int(rng, 2, 64), R=_log_int(rng, 1, 128), N=_log_int(rng, 256, 4096),
                K=_log_int(rng, 256, 2048, 32), skew=rng.choice([0.0, 0.5, 1.0]))
    return case


def _share(count, skew):
    """The probability with which a slot goes to each expert."""
    p = (1.0 + np.arange(count)) ** -skew
    return p / p.sum()


def _blocks(n, size=_BLOCK):
    return -(-n // size)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["type"] == "f32" else 2
        total = T * E * size + 8 * T * k + (4 * E if case["bias"] else 0)
        if case["grad"]:
            total += T * E * size + 4 * T * k           # dlogits, dweights
        return {"bytes": total, "flops": (10.0 if case["grad"] else 4.0) * T * E}
    if op in ("dispatch", "combine"):
        T, C, k = case["T"], case["C"], case["k"]
        if op == "dispatch":
            row = C + 4 * _blocks(C) if case["quantize"] else 2 * C
            total = 2 * T * C + 8 * T * k + T * k * row + 4 * (case["E"] + 1)
            if case["grad"]:
                total += 2 * T * k * C + 2 * T * C      # gradient of the rows, of x
            return {"bytes": total, "flops": float(T * C * (3 if case["quantize"] else 1)
                                                   + (T * k * C if case["grad"] else 0))}
        total = 2 * T * k * C + 8 * T * k + 2 * T * C
        if case["grad"]:
            total += 2 * T * C + 2 * T * k * C + 4 * T * k   # dy, drows, dweights
        return {"bytes": total, "flops": (5.0 if case["grad"] else 2.0) * T * k * C}
    N, K = case["N"], case["K"]
    weights = N * K / 2 + N * _blocks(K, case["group"]) * (3 if case["zeros"] else 2)
    if op == "w4":
        M = case["M"]
        return {"bytes": weights + 2 * M * (K + N), "flops": 2.0 * M * N * K}
    R = case["R"]
    busy = float(np.sum(1.0 - (1.0 - _share(case["G"], case["skew"])) ** R))
    return {"bytes": busy * weights + 2 * R * (K + N) + 4 * (case["G"] + 1),
            "flops": 2.0 * R * N * K}


# ----------------------------------------------------------------- inputs ----

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(shape, g):
    """Zero-mean values whose channels differ in size, as hidden states do."""
    size = torch.exp(0.5 * torch.randn(shape[-1], device="cuda", generator=g))
    return torch.randn(shape, device="cuda", generator=g) * size


def _choices(case, g):
    """k different experts for each token, some of them wanted more than others."""
    E = case["E"]
    p = torch.from_numpy(_share(E, case["skew"])).float().cuda()
    p = p[torch.randperm(E, device="cuda", generator=g)]
    u = torch.rand((case["T"], E), device="cuda", generator=g).clamp_(1e-6, 1.0 - 1e-6)
    return torch.topk(p.log() - (-u.log()).log(), case["k"], dim=1).indices.int()


def _weights4(N, K, group, zeros, dt, g):
    """Codes (N, K / 2), scales and zero points of a weight matrix, as a 4-bit
    checkpoint holds them: groups of each row scaled to the codes' range."""
    kg = _blocks(K, group)
    w = torch.randn((N, K), device="cuda", generator=g) * 0.02
    w = torch.nn.functional.pad(w, (0, kg * group - K)).view(N, kg, group)
    lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
    s = ((hi - lo) / 15.0 if zeros else torch.maximum(hi / 7.0, -lo / 8.0)).to(dt)
    z = torch.round(-lo / s.float()).clamp(0, 15) if zeros else torch.full_like(lo, 8.0)
    q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp_(0, 15)
    q = q.to(torch.uint8).view(N, kg * group)[:, :K]
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return packed, s, z.to(torch.uint8) if zeros else None


def prepare(case, seed):
    g = _generator(seed)
    dt = _TYPES[case["type"]]
    s = {"case": case}
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        liking = 0.5 * torch.randn(E, device="cuda", generator=g)
        s["logits"] = (1.5 * torch.randn((T, E), device="cuda", generator=g) + liking).to(dt)
        s["bias"] = None
        if case["bias"]:
            s["bias"] = -0.05 * liking + 0.01 * torch.randn(E, device="cuda", generator=g)
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        if case["grad"]:
            s["dweights"] = torch.randn((T, case["k"]), device="cuda", generator=g)
        return s
    if op in ("dispatch", "combine"):
        T, C, k = case["T"], case["C"], case["k"]
        s["ids"] = _choices(case, g)
        if op == "dispatch":
            s["x"] = _activations((T, C), g).to(dt)
            if case["grad"]:
                s["drows"] = torch.randn((T * k, C), device="cuda", generator=g).to(dt)
            return s
        s["row_of"] = _plan(s["ids"], case["E"])[1]
        s["rows"] = _activations((T * k, C), g).to(dt)
        s["weights"] = torch.softmax(torch.randn((T, k), device="cuda", generator=g), 1)
        if case["grad"]:
            s["dy"] = torch.randn((T, C), device="cuda", generator=g).to(dt)
        return s
    N, K = case["N"], case["K"]
    if op == "w4":
        s["A"] = _activations((case["M"], K), g).to(dt)
        s["B"], s["SB"], s["ZB"] = _weights4(N, K, case["group"], case["zeros"], dt, g)
        return s
    G, R, kg = case["G"], case["R"], _blocks(K, case["group"])
    rng = np.random.RandomState(seed % (1 << 32))
    counts = rng.multinomial(R, _share(G, case["skew"])[rng.permutation(G)])
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32,
                                device="cuda")
    s["most"] = int(counts.max())       # for the plain form's padding only
    s["A"] = _activations((R, K), g).to(dt)
    s["B"] = torch.empty((G, N, K // 2), device="cuda", dtype=torch.uint8)
    s["SB"] = torch.empty((G, N, kg), device="cuda", dtype=dt)
    s["ZB"] = torch.empty((G, N, kg), device="cuda", dtype=torch.uint8) if case["zeros"] else None
    for i in range(G):
        s["B"][i], s["SB"][i], z = _weights4(N, K, case["group"], case["zeros"], dt, g)
        if z is not None:
            s["ZB"][i] = z
    return s


# ------------------------------------------------------------ plain forms ----

def _plain_route(s):
    case = s["case"]
    l, k, n = s["logits"], case["k"], case["groups"]
    T, E = l.shape
    # The choice in 64 bits: values next to each other are told apart.
    l64 = l.double()
    p64 = torch.softmax(l64, 1) if case["score"] == "softmax" else torch.sigmoid(l64)
    v = p64 if s["bias"] is None else p64 + s["bias"].double()
    if n > 1:
        best = torch.topk(v.view(T, n, E // n), min(case["group_sum"], E // n), dim=2).values.sum(2)
        chosen = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, n), dtype=torch.bool, device="cuda")
        keep.scatter_(1, chosen[:, :case["top_groups"]], True)
        v = torch.where(keep.repeat_interleave(E // n, 1), v, -math.inf)
    ids = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]
    # The weights in 32 bits.
    l = l.float()
    p = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    chosen = p.gather(1, ids)
    total = chosen.sum(1, keepdim=True) if case["renormalize"] else torch.ones_like(chosen[:, :1])
    out = {"ids": ids.int(), "weights": s["scale"] * (chosen / total)}
    if case["grad"]:
        dw = s["scale"] * s["dweights"]
        if case["renormalize"]:
            dw = (dw - (dw * (chosen / total)).sum(1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_(1, ids, dw)
        if case["score"] == "softmax":
            dl = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            dl = dp * p * (1.0 - p)
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _plan(ids, experts):
    """(offsets, row_of): the rows of each slot, sorted by expert."""
    flat = ids.flatten().long()
    expert, slot = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(expert, torch.arange(experts + 1, device="cuda"))
    row_of = torch.empty_like(slot)
    row_of[slot] = torch.arange(len(slot), device="cuda")
    return offsets.int(), row_of.view(ids.shape).int()


def _quantize(x):
    """Codes and scales of float32 rows by blocks of 128 columns."""
    M, K = x.shape
    v = torch.nn.functional.pad(x, (0, _blocks(K) * _BLOCK - K)).view(M, _blocks(K), _BLOCK)
    a = v.abs().amax(dim=2).clamp(min=2.0 ** -100)
    # Tensor by tensor: a division by a Python number is a multiplication in torch.
    top = torch.full_like(a, 448.0)
    q = (v * (top / a)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(M, _blocks(K) * _BLOCK)[:, :K].contiguous(), a / top


def _gather(t, at):
    """Rows of t; 8-bit ones as bytes."""
    return t.view(torch.uint8)[at].view(t.dtype) if t.element_size() == 1 else t[at]


def _plain_dispatch(s):
    case = s["case"]
    offsets, row_of = _plan(s["ids"], case["E"])
    token = torch.empty(row_of.numel(), dtype=torch.long, device="cuda")
    token[row_of.flatten().long()] = torch.arange(row_of.numel(), device="cuda") // case["k"]
    out = {"offsets": offsets, "row_of": row_of}
    if case["quantize"]:
        q, scales = _quantize(s["x"].float())
        out["rows"], out["scales"] = _gather(q, token), scales[token]
    else:
        out["rows"] = s["x"][token]
    if case["grad"]:
        dx = torch.zeros((case["T"], case["C"]), device="cuda")
        for j in range(case["k"]):
            dx += s["drows"][row_of[:, j].long()].float()
        out["dx"] = dx.to(s["x"].dtype)
    return out


def _plain_combine(s):
    case = s["case"]
    row_of, w = s["row_of"].long(), s["weights"]
    y = torch.zeros((case["T"], case["C"]), device="cuda")
    for j in range(case["k"]):
        y += w[:, j, None] * s["rows"][row_of[:, j]].float()
    out = {"y": y.to(s["rows"].dtype)}
    if case["grad"]:
        dy = s["dy"].float()
        out["drows"] = torch.empty_like(s["rows"])
        out["dweights"] = torch.empty_like(w)
        for j in range(case["k"]):
            out["drows"][row_of[:, j]] = (w[:, j, None] * dy).to(s["rows"].dtype)
            out["dweights"][:, j] = (dy * s["rows"][row_of[:, j]].float()).sum(1)
    return out


def _weights32(B, SB, ZB, group, K):
    q = torch.stack((B & 15, B >> 4), dim=-1).flatten(-2).float()
    spread = lambda t: t.float().repeat_interleave(group, dim=-1)[..., :K]  # noqa: E731
    return (q - (8.0 if ZB is None else spread(ZB))) * spread(SB)


def _plain_w4(s):
    case = s["case"]
    w = _weights32(s["B"], s["SB"], s["ZB"], case["group"], case["K"])
    if case["op"] == "w4":
        return (s["A"].float() @ w.t()).to(s["A"].dtype)
    # Rows padded to the largest group, one batched product, rows taken back.
    R, K = s["A"].shape
    G, N, _ = s["B"].shape
    row = torch.arange(R, device="cuda")
    group = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    place = group * s["most"] + row - s["offsets"].long()[group]
    padded = torch.zeros((G * s["most"], K), device="cuda")
    padded = padded.index_copy_(0, place, s["A"].float()).view(G, s["most"], K)
    d = torch.bmm(padded, w.transpose(1, 2))
    return d.view(G * s["most"], N)[place].to(s["A"].dtype)


# ---------------------------------------------------- the library's calls ----

def _own_route(s):
    import tma_pipelined_tensor_tn_gb300 as tg
    case = s["case"]
    r = tg.route_topk(s["logits"], case["k"], score=case["score"], bias=s["bias"],
                      groups=case["groups"], top_groups=case["top_groups"],
                      group_sum=case["group_sum"], renormalize=case["renormalize"],
                      scale=s["scale"])
    out = {"ids": r.ids, "weights": r.weights}
    if case["grad"]:
        out["dlogits"] = tg.route_topk_backward(s["logits"], r.ids, s["dweights"],
                                                score=case["score"],
                                                renormalize=case["renormalize"],
                                                scale=s["scale"])
    return out


def _own_dispatch(s):
    import tma_pipelined_tensor_tn_gb300 as tg
    case = s["case"]
    r = tg.dispatch_rows(s["x"], s["ids"], case["E"], quantize=case["quantize"])
    out = {"offsets": r.offsets, "row_of": r.row_of, "rows": r.rows}
    if case["quantize"]:
        out["scales"] = r.scales
    if case["grad"]:
        out["dx"] = tg.combine_rows(s["drows"], r.row_of)
    return out


def _own_combine(s):
    import tma_pipelined_tensor_tn_gb300 as tg
    out = {"y": tg.combine_rows(s["rows"], s["row_of"], s["weights"])}
    if s["case"]["grad"]:
        d = tg.combine_rows_backward(s["dy"], s["rows"], s["row_of"], s["weights"])
        out["drows"], out["dweights"] = d.drows, d.dweights
    return out


def _own_w4(s):
    import tma_pipelined_tensor_tn_gb300 as tg
    case = s["case"]
    if case["op"] == "w4":
        return tg.gemm_w4(s["A"], s["B"], s["SB"], s["ZB"], group=case["group"])
    return tg.gemm_w4_grouped(s["A"], s["B"], s["SB"], s["offsets"], s["ZB"],
                              group=case["group"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "dispatch": _own_dispatch, "combine": _own_combine,
                "w4": _own_w4, "w4_experts": _own_w4}[op](state)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "w4": _plain_w4, "w4_experts": _plain_w4}[op](state)


# ------------------------------------------------------ results in 64 bits ----

def _e4m3(v):
    """The nearest e4m3 value (ties to even) of float64 numbers up to 448 in size:
    three fraction bits down to 2^-6, steps of 2^-9 below."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_route(s):
    case = s["case"]
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    if case["score"] == "softmax":
        p = np.exp(l - l.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-l))
    v = p + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    if case["groups"] > 1:
        size = E // case["groups"]
        part = -np.sort(-v.reshape(T, case["groups"], size), axis=2)
        score = part[:, :, :min(case["group_sum"], size)].sum(axis=2)
        order = np.argsort(-score, axis=1, kind="stable")
        out_of = np.ones((T, case["groups"]), dtype=bool)
        np.put_along_axis(out_of, order[:, :case["top_groups"]], False, axis=1)
        v = np.where(np.repeat(out_of, size, axis=1), -np.inf, v)
    ids = np.argsort(-v, axis=1, kind="stable")[:, :case["k"]]
    c = np.take_along_axis(p, ids, axis=1)
    total = c.sum(axis=1, keepdims=True)
    w = s["scale"] * (c / total if case["renormalize"] else c)
    out = {"ids": torch.from_numpy(ids.astype(np.int32)), "weights": torch.from_numpy(w)}
    if case["grad"]:
        # dl[t, i] = sum_j dweights[t, j] d w[t, j] / d l[t, i]
        dw = s["dweights"].double().cpu().numpy()
        full = np.zeros((T, E))
        if case["score"] == "softmax":
            # d w_j / d l_i = w_j ([i = j] - share_i), over all experts or the chosen ones
            np.put_along_axis(full, ids, dw * w, axis=1)
            share = p
            if case["renormalize"]:
                share = np.zeros((T, E))
                np.put_along_axis(share, ids, c / total, axis=1)
            full -= share * (dw * w).sum(axis=1, keepdims=True)
        else:
            # d w_j / d l_i = w_j (1 - p_i) ([i = j] - c_i / total)
            part = dw * w
            if case["renormalize"]:
                part = part - c / total * part.sum(axis=1, keepdims=True)
            np.put_along_axis(full, ids, part * (1.0 - c), axis=1)
        out["dlogits"] = torch.from_numpy(full)
    return out


def _exact_plan(ids, experts):
    flat = ids.cpu().numpy().ravel()
    order = np.argsort(flat, kind="stable")
    row_of = np.empty(len(flat), dtype=np.int32)
    row_of[order] = np.arange(len(flat), dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=experts))])
    return offsets.astype(np.int32), row_of.reshape(ids.shape), order


def _exact_dispatch(s):
    case = s["case"]
    offsets, row_of, order = _exact_plan(s["ids"], case["E"])
    token = torch.from_numpy(order // case["k"]).cuda()
    out = {"offsets": torch.from_numpy(offsets), "row_of": torch.from_numpy(row_of)}
    if case["quantize"]:
        values, scales = [], []
        for lo in range(0, case["C"], _BLOCK):
            part = s["x"][:, lo:lo + _BLOCK].double()
            a = part.abs().amax(1).clamp(min=2.0 ** -100)
            # the scale, its reciprocal and the product are rounded to 32 bits
            r = (448.0 / a).float().double()
            values.append(_e4m3((part * r[:, None]).float().double()))
            scales.append((a / 448.0).float().double())
        out["rows"] = torch.cat(values, 1)[token]
        out["scales"] = torch.stack(scales, 1)[token]
    else:
        out["rows"] = s["x"].double()[token]
    if case["grad"]:
        out["dx"] = s["drows"].double()[torch.from_numpy(row_of).cuda().long()].sum(1)
    return out


def _exact_combine(s):
    case = s["case"]
    at = s["row_of"].long()
    w = s["weights"].double()
    out = {"y": torch.empty((case["T"], case["C"]), dtype=torch.float64, device="cuda")}
    if case["grad"]:
        out["drows"] = torch.empty(s["rows"].shape, dtype=torch.float64, device="cuda")
        out["dweights"] = torch.empty_like(w)
    for lo in range(0, case["T"], 1024):
        t = slice(lo, lo + 1024)
        picked = s["rows"][at[t]].double()
        out["y"][t] = torch.einsum("tk,tkc->tc", w[t], picked)
        if case["grad"]:
            dy = s["dy"][t].double()
            out["drows"][at[t]] = w[t][:, :, None] * dy[:, None, :]
            out["dweights"][t] = torch.einsum("tc,tkc->tk", dy, picked)
    return out


def _exact_w4(s):
    case = s["case"]
    N, K, group = case["N"], case["K"], case["group"]
    if case["op"] == "w4":
        spans = [(0, case["M"], s["B"], s["SB"], s["ZB"])]
    else:
        off = s["offsets"].tolist()
        spans = [(off[i], off[i + 1], s["B"][i], s["SB"][i],
                  None if s["ZB"] is None else s["ZB"][i]) for i in range(case["G"])]
    d = torch.zeros((s["A"].shape[0], N), dtype=torch.float64, device="cuda")
    for lo, hi, B, SB, ZB in spans:
        if hi == lo:
            continue
        # even and odd columns apart: they are the low and high halves of the bytes
        at = torch.arange(0, K, 2, device="cuda") // group
        scale = SB.double()[:, at]
        zero = 8.0 if ZB is None else ZB.double()[:, at]
        a = s["A"][lo:hi].double()
        low, high = (B % 16).double() - zero, torch.div(B, 16, rounding_mode="floor").double() - zero
        d[lo:hi] = a[:, 0::2] @ (low * scale).t() + a[:, 1::2] @ (high * scale).t()
    return d


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine,
            "w4": _exact_w4, "w4_experts": _exact_w4}[case["op"]](s)
