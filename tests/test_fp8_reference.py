"""The references of the 8-bit operators and the norms, against independent
facts: torch's own e4m3 casts, exact integer products, and differences."""
import numpy as np
import pytest

from tests import fp8_reference as ref

torch = pytest.importorskip("torch")


def test_e4m3_values_and_encoding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.VALUES, want, equal_nan=True)
    v = np.concatenate([np.linspace(-448, 448, 20001), ref.VALUES[:127], -ref.VALUES[:127],
                        (ref.VALUES[:126] + ref.VALUES[1:127]) / 2])
    v = v.astype(np.float32).astype(np.float64)
    want = torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode_e4m3(v), want)


def test_gemm_reference_on_integers():
    rng = np.random.default_rng(0)
    a, b = rng.integers(-8, 9, (5, 300)), rng.integers(-8, 9, (140, 300))
    sa, sb = 2.0 ** rng.integers(-3, 3, (5, 3)), 2.0 ** rng.integers(-3, 3, (2, 3))
    d, _ = ref.gemm(ref.encode_e4m3(a), sa, ref.encode_e4m3(b), sb)
    full = (a * np.repeat(sa, 128, 1)[:, :300]) @ (
        b * np.repeat(np.repeat(sb, 128, 0)[:140], 128, 1)[:, :300]).T
    assert np.array_equal(d, full)


@pytest.mark.parametrize("gate_shape", [None, "channel", "token", "element"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_norm_gradients_against_differences(gate_shape, post, pre):
    rng = np.random.default_rng(1)
    T, C = 3, 16
    shape = {None: None, "channel": (1, C), "token": (T, 1), "element": (T, C)}[gate_shape]
    v = {"h": rng.normal(size=(T, C)), "y": rng.normal(size=(T, C)),
         "gate": None if shape is None else rng.normal(size=shape),
         "w_post": rng.normal(size=C) if post else None,
         "w_pre": rng.normal(size=C) if pre else None}
    dh, dx = rng.normal(size=(T, C)), rng.normal(size=(T, C)) if pre else None

    def loss(v):
        f = ref.norm_forward(**v, alpha=0.7, eps=1e-3)
        return np.sum(dh * f["h2"]) + (np.sum(dx * f["x"]) if pre else 0.0)

    g = ref.norm_backward(v["h"], dh, dx, **{k: v[k] for k in v if k != "h"}, alpha=0.7, eps=1e-3)
    for name in v:
        if v[name] is None:
            continue
        grad = g["d" + name]
        for at in np.ndindex(v[name].shape):
            step = 1e-5
            up, down = dict(v), dict(v)
            up[name], down[name] = v[name].copy(), v[name].copy()
            up[name][at] += step
            down[name][at] -= step
            num = (loss(up) - loss(down)) / (2 * step)
            # central differences: step^2 times a third derivative of order 10
            assert abs(num - grad.reshape(v[name].shape)[at]) < 1e-7, (name, at)
