"""The oracles of the gated linear recurrence and of the layer norm: closed forms, and gradients against differences."""
import numpy as np
import pytest

from oracle import layer_norm as N
from oracle import recurrence as R


def inputs(B=1, H=2, T=7, D=3, seed=0, decay="log"):
    r = np.random.default_rng(seed)
    x, g, i, gy = (r.standard_normal((B, H, T, D)) for _ in range(4))
    g = -np.abs(g) - 0.05 if decay == "log" else g
    return x, g, i, 0.1 + r.random((H, D)), r.standard_normal((B, H, D)), gy, r.standard_normal((B, H, D))


@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("scale", ["none", "sqrt", "complement"])
@pytest.mark.parametrize("gate", [True, False])
def test_gradients_against_differences(decay, scale, gate):
    x, g, i, rate, h0, gy, ghT = inputs(decay=decay)
    if not gate:
        i = None
    if decay != "rate":
        rate = None

    def loss(**kw):
        a = {"x": x, "g": g, "i": i, "rate": rate, "h0": h0, **kw}
        f = R.forward(**a, decay=decay, scale=scale)
        return (f["y"] * gy).sum() + (f["hT"] * ghT).sum()

    got = R.backward(x, g, i, rate, h0, gy, ghT, decay, scale)
    r = np.random.default_rng(1)
    for n, v in (("x", x), ("g", g), ("i", i), ("rate", rate), ("h0", h0)):
        if v is None:
            continue
        d = r.standard_normal(v.shape)
        step = 1e-5
        diff = (loss(**{n: v + step * d}) - loss(**{n: v - step * d})) / (2 * step)
        assert abs(diff - (got["g" + n] * d).sum()) < 1e-7 * (1 + abs(diff)), n


def test_closed_forms():
    x = np.ones((1, 1, 5, 2))
    half = np.full(x.shape, np.log(0.5))
    y = R.forward(x, half)["y"][0, 0, :, 0]
    assert np.allclose(y, 2 - 0.5 ** np.arange(5))
    assert np.allclose(R.forward(x, half, scale="complement")["y"][0, 0, :, 0], 1 - 0.5 ** (np.arange(5) + 1))
    g = half.copy()
    g[:, :, 3] = -np.inf  # a reset
    assert np.allclose(R.forward(x, g)["y"][0, 0, 3:, 0], [1, 1.5])
    # with unit white noise the state's variance stays at one
    r = np.random.default_rng(0)
    h = R.forward(r.standard_normal((1, 1, 400, 500)), np.full((1, 1, 400, 500), -0.02), scale="sqrt",
                  h0=r.standard_normal((1, 1, 500)))["y"]
    assert abs((h ** 2).mean() - 1) < 0.05


def test_layer_norm_gradients_against_differences():
    r = np.random.default_rng(2)
    x, gy, gt = (r.standard_normal((4, 9)) for _ in range(3))
    w, b = r.standard_normal(9), r.standard_normal(9)
    got = N.backward(x, w, gy, gt)
    loss = lambda x=x, w=w, b=b: (N.forward(x, w, b)[0] * gy).sum() + (x * gt).sum()
    for n, v in (("x", x), ("w", w), ("b", b)):
        d, step = r.standard_normal(v.shape), 1e-6
        diff = (loss(**{n: v + step * d}) - loss(**{n: v - step * d})) / (2 * step)
        want = (got[{"x": "gx", "w": "gweight", "b": "gbias"}[n]] * d).sum()
        assert abs(diff - want) < 1e-7 * (1 + abs(diff)), n
    y = N.forward(x)[0]
    assert np.allclose(y.mean(-1), 0) and np.allclose(y.var(-1), 1, atol=1e-4)
