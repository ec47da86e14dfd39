"""Performance cases of the 8-bit linear layers: block-scaled quantisation, the
block-scaled products (dense and grouped by expert) and the fused norms around
a block.

Each case is one pass through one operator, either in its plain form (torch
operations in 32 bits, one rounding at the end) or, with ``own`` set, through
the library's entry points.  ``exact`` gives the results from the operators'
definitions in 64 bits.

Definitions (B = 128, the block length along K; e4m3 with largest value 448):
  quantise   a = max(max |x| over a block, 2^-100); scale S = fl32(a / 448);
             Q = e4m3(fl32(x * fl32(448 / a))), to nearest even.
  product    D[m, n] = sum_b SA[m, b] SB[n // B, b] sum_{k in b} A[m, k] W[n, k].
  norms      u = y * rsqrt(mean y^2 + eps) * w_post (u = y without w_post),
             h' = h + alpha * gate * u,
             x  = h' * rsqrt(mean h'^2 + eps) * w_pre.
"""
import math

import numpy as np
import torch

own = False

_BLOCK = 128
_EPS = 1e-6
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # One token decoded against a down projection: bound by reading the weights once.
        {"name": "linear_decode_1", "op": "gemm", "M": 1, "N": 4096, "K": 14336, "type": "bf16"},
        # A decode batch against an up projection.
        {"name": "linear_decode_32", "op": "gemm", "M": 32, "N": 14336, "K": 4096, "type": "f16"},
        # A prompt of an odd length, output and inner sizes that end inside a block.
        {"name": "linear_odd", "op": "gemm", "M": 1237, "N": 5000, "K": 2064, "type": "f16"},
        # A long prompt (or a batch of them): bound by the tensor cores.
        {"name": "linear_8192", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "type": "bf16"},
        # A decode batch over many experts: most get a few tokens, some none.
        {"name": "experts_decode", "op": "grouped", "G": 64, "R": 128, "N": 4096, "K": 2048,
         "skew": 1.0, "type": "bf16"},
        # A prompt over few experts, unevenly routed.
        {"name": "experts_prompt", "op": "grouped", "G": 8, "R": 8192, "N": 4096, "K": 2048,
         "skew": 1.0, "type": "bf16"},
        # Ragged sizes throughout.
        {"name": "experts_odd", "op": "grouped", "G": 21, "R": 1999, "N": 1544, "K": 1040,
         "skew": 0.5, "type": "f16"},
        # Activations of a long prompt, one scale per row and block.
        {"name": "quantize_rows", "op": "quantize", "M": 8192, "K": 14336, "block_rows": 1,
         "type": "bf16"},
        # A weight matrix with an odd number of rows, one scale per 128 x 128.
        {"name": "quantize_weight", "op": "quantize", "M": 4100, "K": 4096, "block_rows": 128,
         "type": "f16"},
        # Between two blocks while decoding one token: latency only.
        {"name": "norm_decode", "op": "norm", "T": 1, "C": 4096, "post": True, "gate": "channel",
         "quantize": True, "grad": False, "type": "bf16"},
        # Between two blocks of a prompt, feeding an 8-bit product; no norm after the block.
        {"name": "norm_prompt", "op": "norm", "T": 4096, "C": 8192, "post": False, "gate": "none",
         "quantize": True, "grad": False, "type": "f16"},
        # A training step: forward, then every gradient.
        {"name": "norm_train", "op": "norm", "T": 8192, "C": 4096, "post": True,
         "gate": "element", "quantize": False, "grad": True, "type": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, (v + step - 1) // step * step)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "grouped", "quantize", "norm"])
    t = rng.choice(["f16", "bf16"])
    if op == "gemm":
        M = _log_int(rng, 1, 8192)
        return {"op": op, "M": M, "N": _log_int(rng, 128, 14336, 8),
                "K": _log_int(rng, 256, 14336 if M <= 4096 else 8192, 16), "type": t}
    if op == "grouped":
        return {"op": op, "G": _log_int(rng, 2, 64), "R": _log_int(rng, 8, 8192),
                "N": _log_int(rng, 256, 4096, 8), "K": _log_int(rng, 256, 2048, 16),
                "skew": rng.choice([0.0, 0.5, 1.0]), "type": t}
    if op == "quantize":
        return {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 128, 14336, 8),
                "block_rows": rng.choice([1, 1, 128]), "type": t}
    grad = rng.random() < 0.5
    return {"op": op, "T": _log_int(rng, 1, 8192), "C": _log_int(rng, 256, 8192, 8),
            "post": rng.random() < 0.5,
            "gate": rng.choice(["none", "channel", "token", "element"]),
            "quantize": not grad and rng.random() < 0.5, "grad": grad, "type": t}


def _share(case):
    """The probability with which a row goes to each expert."""
    p = (1.0 + np.arange(case["G"])) ** -case["skew"]
    return p / p.sum()


def work(case):
    blocks = lambda n: -(-n // _BLOCK)  # noqa: E731
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * blocks(K) * (M + blocks(N)),
                "flops": 2.0 * M * N * K}
    if case["op"] == "grouped":
        R, N, K = case["R"], case["N"], case["K"]
        # experts that get at least one row, on average
        busy = float(np.sum(1.0 - (1.0 - _share(case)) ** R))
        return {"bytes": R * K + busy * N * K + 2 * R * N + 4 * blocks(K) * (R + busy * blocks(N)),
                "flops": 2.0 * R * N * K}
    if case["op"] == "quantize":
        M, K, br = case["M"], case["K"], case["block_rows"]
        return {"bytes": 3 * M * K + 4 * (-(-M // br)) * blocks(K), "flops": 3.0 * M * K}
    T, C = case["T"], case["C"]
    gate = {"none": 0, "channel": C, "token": T, "element": T * C}[case["gate"]]
    weights = C * (2 if case["post"] else 1)
    # forward: read h, y, gate and weights; write h', x
    total = 2 * (2 * T * C + gate + weights) + 2 * T * C
    total += T * C + 4 * T * blocks(C) if case["quantize"] else 2 * T * C
    if case["grad"]:
        # both directions' outputs, and the gradients' own inputs
        total += 4 * T * (2 if case["post"] else 1)
        total += 2 * 2 * T * C                       # dh', dx
        total += 2 * 2 * T * C + 4 * weights         # dh, dy, weight gradients
        total += 2 * gate if case["gate"] == "element" else 4 * gate
    return {"bytes": total, "flops": (30.0 if case["grad"] else 12.0) * T * C}


# ----------------------------------------------------------------- inputs ----

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(shape, g):
    """Zero-mean values whose channels differ in size, as hidden states do."""
    size = torch.exp(0.5 * torch.randn(shape[-1], device="cuda", generator=g))
    return torch.randn(shape, device="cuda", generator=g) * size


def _quantize_blocks(x, block_rows):
    """Codes and scales of a float32 matrix by blocks of block_rows x 128."""
    M, K = x.shape
    rows, cols = -(-M // block_rows), -(-K // _BLOCK)
    padded = torch.nn.functional.pad(x, (0, cols * _BLOCK - K, 0, rows * block_rows - M))
    v = padded.view(rows, block_rows, cols, _BLOCK)
    a = v.abs().amax(dim=(1, 3)).clamp(min=2.0 ** -100)
    # Tensor by tensor: a division by a Python number is a multiplication in torch.
    top = torch.full_like(a, 448.0)
    q = (v * (top / a)[:, None, :, None]).to(torch.float8_e4m3fn)
    q = q.view(rows * block_rows, cols * _BLOCK)[:M, :K].contiguous()
    return q, a / top


def prepare(case, seed):
    g = _generator(seed)
    dt = _TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "gemm":
        s["A"], s["SA"] = _quantize_blocks(_activations((case["M"], case["K"]), g), 1)
        # the quantiser's layout of row scales: consecutive rows next to each other
        s["SA"] = s["SA"].t().contiguous().t()
        w = torch.randn((case["N"], case["K"]), device="cuda", generator=g) * 0.02
        s["B"], s["SB"] = _quantize_blocks(w, _BLOCK)
    elif case["op"] == "grouped":
        G, R, N, K = case["G"], case["R"], case["N"], case["K"]
        rng = np.random.RandomState(seed % (1 << 32))
        counts = rng.multinomial(R, _share(case)[rng.permutation(G)])
        offsets = np.concatenate([[0], np.cumsum(counts)])
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["most"] = int(counts.max())       # for the plain form's padding only
        s["A"], s["SA"] = _quantize_blocks(_activations((R, K), g), 1)
        s["SA"] = s["SA"].t().contiguous().t()
        s["B"] = torch.empty((G, N, K), device="cuda", dtype=torch.float8_e4m3fn)
        s["SB"] = torch.empty((G, -(-N // _BLOCK), -(-K // _BLOCK)), device="cuda")
        for i in range(G):
            w = torch.randn((N, K), device="cuda", generator=g) * 0.02
            s["B"][i], s["SB"][i] = _quantize_blocks(w, _BLOCK)
    elif case["op"] == "quantize":
        x = _activations((case["M"], case["K"]), g)
        s["X"] = (x if case["block_rows"] == 1 else x * 0.02).to(dt)
    else:
        T, C = case["T"], case["C"]
        s["h"] = (2.0 * _activations((T, C), g)).to(dt)
        s["y"] = _activations((T, C), g).to(dt)
        shape = {"none": None, "channel": (C,), "token": (T, 1), "element": (T, C)}[case["gate"]]
        s["gate"] = None
        if shape is not None:
            s["gate"] = torch.sigmoid(torch.randn(shape, device="cuda", generator=g)).to(dt)
        weight = lambda: (1.0 + 0.1 * torch.randn(C, device="cuda", generator=g)).to(dt)  # noqa: E731
        s["w_pre"] = weight()
        s["w_post"] = weight() if case["post"] else None
        s["alpha"] = 0.5
        if case["grad"]:
            s["dh"] = torch.randn((T, C), device="cuda", generator=g).to(dt)
            s["dx"] = torch.randn((T, C), device="cuda", generator=g).to(dt)
    return s


# ------------------------------------------------------------ plain forms ----

def _spread(scales, block, size, dim):
    return scales.repeat_interleave(block, dim=dim).narrow(dim, 0, size)


def _weights32(B, SB):
    N, K = B.shape[-2:]
    return B.float() * _spread(_spread(SB, _BLOCK, N, -2), _BLOCK, K, -1)


def _plain_gemm(s):
    a = s["A"].float() * _spread(s["SA"], _BLOCK, s["A"].shape[1], 1)
    return (a @ _weights32(s["B"], s["SB"]).t()).to(_TYPES[s["case"]["type"]])


def _plain_grouped(s):
    # Rows padded to the largest group, one batched product, rows taken back.
    R, K = s["A"].shape
    G, N, _ = s["B"].shape
    a = s["A"].float() * _spread(s["SA"], _BLOCK, K, 1)
    row = torch.arange(R, device="cuda")
    group = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    place = group * s["most"] + row - s["offsets"].long()[group]
    padded = a.new_zeros((G * s["most"], K)).index_copy_(0, place, a).view(G, s["most"], K)
    d = torch.bmm(padded, _weights32(s["B"], s["SB"]).transpose(1, 2))
    return d.view(G * s["most"], N)[place].to(_TYPES[s["case"]["type"]])


def _plain_quantize(s):
    return _quantize_blocks(s["X"].float(), s["case"]["block_rows"])


def _plain_norm(s):
    case = s["case"]
    dt = _TYPES[case["type"]]
    h, y = s["h"].float(), s["y"].float()
    g = 1.0 if s["gate"] is None else s["gate"].float()
    u, ry = y, None
    if case["post"]:
        ry = torch.rsqrt(y.square().mean(1, keepdim=True) + _EPS)
        u = y * ry * s["w_post"].float()
    h2 = h + s["alpha"] * (g * u)
    rh = torch.rsqrt(h2.square().mean(1, keepdim=True) + _EPS)
    x = h2 * rh * s["w_pre"].float()
    if case["quantize"]:
        q, scales = _quantize_blocks(x, 1)
        return {"h": h2.to(dt), "x": q, "scales": scales}
    out = {"h": h2.to(dt), "x": x.to(dt)}
    if not case["grad"]:
        return out
    dx, dh = s["dx"].float(), s["dh"].float()
    n = h2 * rh
    p = dx * s["w_pre"].float()
    dt_h = dh + rh * (p - n * (p * n).mean(1, keepdim=True))
    out["dw_pre"] = (dx * n).sum(0)
    out["dh"] = dt_h.to(dt)
    du = s["alpha"] * (g * dt_h)
    if case["post"]:
        ny = y * ry
        out["dw_post"] = (du * ny).sum(0)
        q = du * s["w_post"].float()
        out["dy"] = (ry * (q - ny * (q * ny).mean(1, keepdim=True))).to(dt)
    else:
        out["dy"] = du.to(dt)
    if case["gate"] == "element":
        out["dgate"] = (s["alpha"] * (u * dt_h)).to(dt)
    elif case["gate"] == "channel":
        out["dgate"] = s["alpha"] * (u * dt_h).sum(0)
    elif case["gate"] == "token":
        out["dgate"] = s["alpha"] * (u * dt_h).sum(1, keepdim=True)
    return out


def _own_norm(s):
    import tma_pipelined_tensor_tn_gb300 as tg
    case = s["case"]
    r = tg.norm_residual(s["h"], s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
                         alpha=s["alpha"], eps=_EPS, quantize=case["quantize"],
                         save_rstd=case["grad"])
    if case["quantize"]:
        return {"h": r.h, "x": r.x, "scales": r.scales}
    out = {"h": r.h, "x": r.x}
    if case["grad"]:
        d = tg.norm_residual_backward(s["h"], s["y"], dh=s["dh"], dx=s["dx"], gate=s["gate"],
                                      w_post=s["w_post"], w_pre=s["w_pre"], alpha=s["alpha"],
                                      rstd_post=r.rstd_post, rstd_pre=r.rstd_pre)
        out.update({"dw_pre": d.dw_pre, "dh": d.dh, "dy": d.dy})
        if case["post"]:
            out["dw_post"] = d.dw_post
        if case["gate"] != "none":
            out["dgate"] = d.dgate
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"gemm": _plain_gemm, "grouped": _plain_grouped, "quantize": _plain_quantize,
                "norm": _plain_norm}[op](state)
    import tma_pipelined_tensor_tn_gb300 as tg
    dt = _TYPES[state["case"]["type"]]
    if op == "gemm":
        return tg.gemm_fp8(state["A"], state["SA"], state["B"], state["SB"], dtype=dt)
    if op == "grouped":
        return tg.gemm_fp8_grouped(state["A"], state["SA"], state["B"], state["SB"],
                                   state["offsets"], dtype=dt)
    if op == "quantize":
        return tg.quantize_fp8(state["X"], block_rows=state["case"]["block_rows"])
    return _own_norm(state)


# ------------------------------------------------------ results in 64 bits ----

def _e4m3(v):
    """The nearest e4m3 value (ties to even) of float64 numbers up to 448 in size:
    three fraction bits down to 2^-6, steps of 2^-9 below."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    # log2 may round up to the next power just below it
    e = np.where(np.ldexp(1.0, e.astype(int)) > np.maximum(np.abs(v), 2.0 ** -6), e - 1, e)
    step = np.ldexp(1.0, e.astype(int) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def _exact_quantize(x, block_rows):
    """Quantisation of float64 x; the scale, its reciprocal and the product are
    rounded to 32 bits, as the definition says."""
    M, K = x.shape
    q = np.empty((M, K))
    scales = np.empty((-(-M // block_rows), -(-K // _BLOCK)))
    for b in range(scales.shape[1]):
        part = x[:, b * _BLOCK:(b + 1) * _BLOCK]
        a = np.abs(part).max(axis=1)
        a = np.maximum.reduceat(a, np.arange(0, M, block_rows))
        a = np.maximum(a.astype(np.float32), np.float32(2.0 ** -100))
        scales[:, b] = a / np.float32(448.0)
        r = (np.float32(448.0) / a).astype(np.float64).repeat(block_rows)[:M, None]
        q[:, b * _BLOCK:(b + 1) * _BLOCK] = _e4m3((part * r).astype(np.float32).astype(np.float64))
    return q, scales


def _exact_norm(s):
    case = s["case"]
    d = lambda k: s[k].double()  # noqa: E731
    C = case["C"]
    h, y, wq = d("h"), d("y"), d("w_pre")
    g = torch.ones((), dtype=torch.float64, device="cuda") if s["gate"] is None else d("gate")
    inv = lambda v: ((v * v).sum(1, keepdim=True) / C + _EPS) ** -0.5  # noqa: E731
    ny = y * inv(y) if case["post"] else y
    u = ny * d("w_post") if case["post"] else y
    h2 = h + s["alpha"] * g * u
    n = h2 * inv(h2)
    x = n * wq
    if case["quantize"]:
        q, scales = _exact_quantize(x.cpu().numpy(), 1)
        return {"h": h2, "x": torch.from_numpy(q), "scales": torch.from_numpy(scales)}
    out = {"h": h2, "x": x}
    if case["grad"]:
        p = d("dx") * wq
        t = d("dh") + inv(h2) * (p - n * ((p * n).sum(1, keepdim=True) / C))
        out["dh"], out["dw_pre"] = t, (d("dx") * n).sum(0)
        du = s["alpha"] * g * t
        if case["post"]:
            q = du * d("w_post")
            out["dy"] = inv(y) * (q - ny * ((q * ny).sum(1, keepdim=True) / C))
            out["dw_post"] = (du * ny).sum(0)
        else:
            out["dy"] = du
        dg = s["alpha"] * u * t
        if case["gate"] != "none":
            out["dgate"] = {"channel": dg.sum(0), "token": dg.sum(1, keepdim=True),
                            "element": dg}[case["gate"]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        q, scales = _exact_quantize(s["X"].double().cpu().numpy(), case["block_rows"])
        return torch.from_numpy(q), torch.from_numpy(scales)
    if case["op"] == "norm":
        return _exact_norm(s)
    # Products: block by block along K, each block's sum scaled and added.
    if case["op"] == "gemm":
        spans = [(0, case["M"], s["B"], s["SB"])]
    else:
        off = s["offsets"].tolist()
        spans = [(off[i], off[i + 1], s["B"][i], s["SB"][i]) for i in range(case["G"])]
    K, N = case["K"], case["N"]
    d = torch.zeros((s["A"].shape[0], N), dtype=torch.float64, device="cuda")
    n_block = torch.arange(N, device="cuda") // _BLOCK
    for lo, hi, B, SB in spans:
        if hi == lo:
            continue
        for b in range(-(-K // _BLOCK)):
            k = slice(b * _BLOCK, min(K, (b + 1) * _BLOCK))
            part = s["A"][lo:hi, k].double() @ B[:, k].double().t()
            part *= s["SA"][lo:hi, b].double()[:, None]
            part *= SB[:, b].double()[n_block][None, :]
            d[lo:hi] += part
    return d
