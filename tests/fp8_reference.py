"""Plain references of the 8-bit operators and the norms, in 64 bits (numpy),
written from their definitions and sharing no code with the library."""
import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)
TOP = np.float32(448.0)


def e4m3_values():
    """The value of each of the 256 e4m3 codes (sign, 4 exponent bits of bias 7,
    3 fraction bits; exponent 0 is subnormal; 0x7f and 0xff are NaN)."""
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


VALUES = e4m3_values()


def encode_e4m3(v):
    """Codes of float64 values in [-448, 448], to nearest, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    grid = VALUES[:127]                                     # 0 .. 448, ascending
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = grid[hi] - a, a - grid[lo]
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= grid[126], 126, code)
    return np.where(np.signbit(v), code | 128, code).astype(np.uint8)


def quantize(x, block_rows):
    """(codes, scales) of a float array, block by block, with the definition's
    roundings to 32 bits."""
    M, K = x.shape
    rows, blocks = -(-M // block_rows), -(-K // BLOCK)
    codes = np.zeros((M, K), dtype=np.uint8)
    scales = np.zeros((rows, blocks), dtype=np.float32)
    for i in range(rows):
        for b in range(blocks):
            r = slice(i * block_rows, min(M, (i + 1) * block_rows))
            c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
            part = x[r, c].astype(np.float32)
            a = np.maximum(np.max(np.abs(part)), FLOOR)
            scales[i, b] = a / TOP
            codes[r, c] = encode_e4m3((part * (TOP / a)).astype(np.float32).astype(np.float64))
    return codes, scales


def gemm(a_codes, sa, b_codes, sb):
    """(D, S): the block-scaled product in 64 bits, and the sum of the
    magnitudes of its terms (what rounding errors are measured by)."""
    A, B = VALUES[a_codes], VALUES[b_codes]
    M, K = A.shape
    N = B.shape[0]
    d, s = np.zeros((M, N)), np.zeros((M, N))
    with np.errstate(invalid="ignore"):
        for b in range(-(-K // BLOCK)):
            c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
            scale = (sa[:, b].astype(np.float64)[:, None]
                     * sb[np.arange(N) // BLOCK, b].astype(np.float64)[None, :])
            d += (A[:, c] @ B[:, c].T) * scale
            s += (np.abs(A[:, c]) @ np.abs(B[:, c]).T) * np.abs(scale)
    return d, s


def gemm_bound(ref, s, K, bf16):
    """What a product may be off: half a step of its type (at most 2^-8 of a bf16
    value with its 8 significant bits, 2^-11 of an fp16 one), and one FP32 rounding
    (2^-23, the tensor cores may truncate) of the terms' magnitudes for each
    addition of partial sums -- an MMA every 32 k, a scaled block every 128 --
    doubled for the additions within an MMA."""
    half = 2.0 ** -8 if bf16 else 2.0 ** -11
    steps = -(-K // 32) + -(-K // BLOCK) + 2
    tiny = 2.0 ** -134 if bf16 else 2.0 ** -25            # half the smallest step
    return half * np.abs(ref) + steps * 2.0 ** -22 * s + tiny


def norm_forward(h, y=None, gate=None, w_post=None, w_pre=None, alpha=1.0, eps=1e-6):
    """dict of u, h2, x, rstd_post, rstd_pre in 64 bits."""
    out = {"u": None, "h2": h, "x": None, "ry": None, "rh": None}
    if y is not None:
        u = y
        if w_post is not None:
            out["ry"] = (np.mean(y * y, axis=1, keepdims=True) + eps) ** -0.5
            u = y * out["ry"] * w_post
        out["u"] = u
        out["h2"] = h + alpha * (1.0 if gate is None else gate) * u
    if w_pre is not None:
        out["rh"] = (np.mean(out["h2"] ** 2, axis=1, keepdims=True) + eps) ** -0.5
        out["x"] = out["h2"] * out["rh"] * w_pre
    return out


def norm_backward(h, dh, dx, y=None, gate=None, w_post=None, w_pre=None, alpha=1.0, eps=1e-6):
    """dict of gradients of sum(dh * h') + sum(dx * x)."""
    f = norm_forward(h, y, gate, w_post, w_pre, alpha, eps)
    t = np.zeros_like(h) if dh is None else dh.copy()
    out = {}
    if w_pre is not None:
        n = f["h2"] * f["rh"]
        p = dx * w_pre
        t = t + f["rh"] * (p - n * np.mean(p * n, axis=1, keepdims=True))
        out["dw_pre"] = np.sum(dx * n, axis=0)
    out["dh"] = t
    if y is None:
        return out
    g = np.ones((1, 1)) if gate is None else gate
    du = alpha * g * t
    if w_post is not None:
        m = y * f["ry"]
        q = du * w_post
        out["dy"] = f["ry"] * (q - m * np.mean(q * m, axis=1, keepdims=True))
        out["dw_post"] = np.sum(du * m, axis=0)
    else:
        out["dy"] = du
    if gate is not None:
        dg = alpha * f["u"] * t
        if gate.shape == h.shape:
            out["dgate"] = dg
        elif gate.shape[-1] == h.shape[1]:
            out["dgate"] = np.sum(dg, axis=0).reshape(gate.shape)
        else:
            out["dgate"] = np.sum(dg, axis=1, keepdims=True)
    return out
