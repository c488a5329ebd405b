"""The recurrence by rates on both sides of 0.375, up to which all of a block's rates take the path of decays near one.

The oracle's bounds hold for any rate in the states: a decay's relative error is y (7 + 1.5 |g|) + 4 units of 2^-24, with
y = rate σ(g) its logarithm, and y a <= 1 - a, so that 7 + 1.5 |g| <= c covers it. In the gradients, where a stands by
itself, y <= 4 keeps 4 (7 + 1.5 |g|) + 4 below the bound's 2 c + 8."""
import numpy as np
import pytest
import torch
from test_recurrence_gpu import DEV, f64, make, near

from bayesian_filtering_linear_gb300 import kla
from oracle import recurrence as R

pytestmark = pytest.mark.gpu


def check(B, H, T, D, io, scale, rate, gate=True, backward=True, seed=0):
    x, g, i, _, h0, gy, ghT = make(B, H, T, D, io, "rate", gate, heads_last=True, seed=seed)
    how = {"decay": "rate", "scale": scale}
    args = [f64(t) for t in (x, g, i, rate, h0)]
    y, hT, kept = kla.recurrence_forward(x, g, i, rate, h0, checkpoints=True, **how)
    f = R.forward(*args, **how)
    near(y, f["y"], f["y_err"], io, "y")
    near(hT, f["hT"], f["hT_err"], "f32", "hT")
    state = h0.clone()
    step = kla.recurrence_step(*(None if z is None else z[:, :, 0].contiguous() for z in (x, g, i)), rate, state, **how)
    near(step, f["y"][:, :, 0], f["y_err"][:, :, 0], io, "step")
    if not backward:
        return
    d = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, checkpoints=kept, **how)
    want = R.backward(*args, f64(gy), f64(ghT), **how)
    for n, t in d.items():
        near(t, want[n], want[n + "_err"], "f32" if n in ("grate", "gh0") else io, n)


def rates(H, D, lo, hi, seed=0):
    r = torch.Generator().manual_seed(seed)
    return (lo * (hi / lo) ** torch.rand(H, D, generator=r)).to(DEV)


@pytest.mark.parametrize("scale", ["none", "sqrt", "complement"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T", [1, 37, 64, 129, 700])
def test_rates_on_both_sides(scale, io, gate, T):
    check(2, 3, T, 40, io, scale, rates(3, 40, 0.02, 4.0, T), gate, seed=T)


@pytest.mark.parametrize("scale", ["none", "sqrt", "complement"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_blocks_on_each_path(scale, io):
    """Some blocks' rates are all at most 0.375, some have one above, and some lie around it."""
    H, D = 6, 64
    rate = rates(H, D, 0.01, 0.374)
    rate[1, 7] = 0.376
    rate[2] = 0.375
    rate[3] = rates(1, D, 0.374, 0.376, 1)
    rate[4, 63] = 3.0
    check(3, H, 1031, D, io, scale, rate, seed=3)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T", [(1, 1, 2500), (1, 16, 1500), (20, 16, 400), (40, 16, 200)])
def test_clusters(io, B, H, T):
    check(B, H, T, 64, io, "sqrt", rates(H, 64, 0.05, 4.0), seed=B)


@pytest.mark.parametrize("scale", ["none", "sqrt", "complement"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rates_that_forget_at_once(scale, io):
    check(2, 2, 300, 64, io, scale, rates(2, 64, 4.0, 200.0), backward=False)


def test_gradients_against_differences():
    """Central differences of the fp64 oracle's loss along random directions, against the kernels' fp32 gradients: the
    oracle's second order is 1e-4^2 of the loss's third derivative, below 1e-5 of the sums here."""
    x, g, i, _, h0, gy, ghT = make(1, 2, 130, 16, "f32", "rate")
    rate = rates(2, 16, 0.05, 4.0)
    how = {"decay": "rate", "scale": "sqrt"}
    d = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, **how)
    args = {n: f64(t) for n, t in (("x", x), ("g", g), ("i", i), ("rate", rate), ("h0", h0))}

    def loss(**kw):
        f = R.forward(**{**args, **kw}, **how)
        return (f["y"] * f64(gy)).sum() + (f["hT"] * f64(ghT)).sum()

    r = np.random.default_rng(0)
    for n, v in args.items():
        way, step = r.standard_normal(v.shape), 1e-4
        got = (f64(d["g" + n]) * way).sum()
        want = (loss(**{n: v + step * way}) - loss(**{n: v - step * way})) / (2 * step)
        assert abs(got - want) <= 1e-4 * np.abs(f64(d["g" + n]) * way).sum(), n
