"""Infinities in the recurrence: a state that is infinite stays so (a ∞ + b = ∞ for every decay above zero), whatever way
the tokens are shared out, and gradients are infinite where their formulas are, and nowhere else. The oracle goes token by
token in 64 bits and says where values are infinite or NaN; finite ones keep its bounds."""
import itertools

import numpy as np
import pytest
import torch
from test_recurrence_gpu import DEV, DT, f64

from bayesian_filtering_linear_gb300 import kla
from oracle import recurrence as R

pytestmark = pytest.mark.gpu
KINDS = list(itertools.product(["log", "sigmoid", "rate"], ["none", "sqrt", "complement"]))
INF = float("inf")


def same(got, want, err, io, what):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf]), what
    rest = np.isfinite(want)
    tol = err[rest] + (2.0 ** -8 * (np.abs(want[rest]) + err[rest]) if io == "bf16" else 0) + 1e-36
    assert (np.abs(got[rest] - want[rest]) <= tol).all(), what


def make(B, H, T, D, io, decay, far=False, seed=0):
    """Decays from near one to (`far`) e^-20, whose product over a few tokens is below every float."""
    r = torch.Generator().manual_seed(seed)
    x, g, i, gy = (torch.randn(B, H, T, D, generator=r) for _ in range(4))
    rate = None
    if decay == "log":
        g = -(20.0 if far else 1.0) * torch.rand(B, H, T, D, generator=r)
    elif decay == "sigmoid":
        g = g - 18 if far else g + 1
    else:
        rate = (30.0 if far else 0.5) * torch.rand(H, D, generator=r)
    x, g, i, gy = (t.to(DT[io]).to(DEV) for t in (x, g, i, gy.abs() + 0.1))
    h0, ghT = torch.randn(B, H, D, generator=r).to(DEV), torch.rand(B, H, D, generator=r).to(DEV) + 0.1
    return x, g, i, None if rate is None else rate.to(DEV), h0, gy, ghT


@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_step_from_an_infinite_state(decay, io):
    """Decays of one, next to one, where 1 - a begins to be exact, and far ones; 0 · ∞ has no value."""
    D = 64
    values = {"log": [0.0, -1e-8, -0.01, -0.2, -0.375, -0.4, -1.0, -20.0, -80.0], "sigmoid": [80.0, 9.0, 1.0, 0.0, -1.0, -70.0],
              "rate": [30.0, 3.0, 1.0, 0.0, -1.0, -30.0]}[decay]
    g = torch.tensor(values).repeat(D)[:D].to(DT[io]).to(DEV).expand(2, 1, D).contiguous()
    rates = torch.tensor([0.0, 1e-6, 0.3, 0.7, 5.0, 60.0, 0.05]).repeat(D)[:D].to(DEV).view(1, D)
    state = torch.full((2, 1, D), INF, device=DEV)
    state[1] = -INF
    want = state.clone()
    x = torch.randn(2, 1, D, device=DEV).to(DT[io])
    y = kla.recurrence_step(x, g, None, rates if decay == "rate" else None, state, decay=decay)
    assert torch.equal(state, want) and torch.equal(y.float(), want)
    y = kla.recurrence_step(torch.full_like(x, -INF), g, None, rates if decay == "rate" else None, state, decay=decay)
    assert bool(y[0].isnan().all()) and bool((y[1] == -INF).all())
    if decay == "log":
        reset = torch.full_like(g, -INF)
        assert bool(kla.recurrence_step(x, reset, None, None, want, decay=decay).isnan().all())
        finite = torch.full_like(want, 3e38)
        assert torch.equal(kla.recurrence_step(x, reset, None, None, finite, decay=decay), x)


@pytest.mark.parametrize("decay,scale", KINDS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("far", [False, True])
def test_infinite_states_stay(decay, scale, io, far):
    """From the first state on, from an x on, and until an x of the other sign; the other channels' bits stay."""
    B, H, T, D = 2, 2, 333, 64
    x, g, i, rate, h0, _, _ = make(B, H, T, D, io, decay, far)
    how = {"decay": decay, "scale": scale}
    want = kla.recurrence_forward(x, g, i, rate, h0, checkpoints=True, **how)
    h0[0, 0, 3], h0[0, 1, 8] = INF, -INF
    x[1, 0, 77, 5], x[1, 0, 100, 6], x[1, 0, 250, 6], x[0, 1, 200, 8] = INF, -INF, INF, INF
    y, hT, kept = kla.recurrence_forward(x, g, i, rate, h0, checkpoints=True, **how)
    with np.errstate(all="ignore"):
        f = R.forward(*[f64(t) for t in (x, g, i, rate, h0)], **how)
    assert np.isinf(f["y"][0, 0, :, 3]).all() and np.isnan(f["y"][1, 0, 250:, 6]).all()
    same(y, f["y"], f["y_err"], io, "y")
    same(hT, f["hT"], f["hT_err"], "f32", "hT")
    before = np.concatenate([f64(h0)[:, :, None], f["y"][:, :, 63::64]], 2)[:, :, :kept.shape[0]]
    zero = np.zeros_like(f["y_err"][:, :, :1])
    before_err = np.concatenate([zero, f["y_err"][:, :, 63::64]], 2)[:, :, :kept.shape[0]]
    same(kept, np.moveaxis(before, 2, 0), np.moveaxis(before_err, 2, 0), "f32", "checkpoints")
    clean = torch.ones(B, H, D, dtype=torch.bool, device=DEV)
    for c in ((0, 0, 3), (0, 1, 8), (1, 0, 5), (1, 0, 6)):
        clean[c] = False
    tokens = clean[:, :, None].expand_as(y)
    assert torch.equal(y[tokens], want[0][tokens]) and torch.equal(hT[clean], want[1][clean])
    # and token by token
    state = h0.clone()
    for t in range(90):
        step = kla.recurrence_step(*(z[:, :, t].contiguous() for z in (x, g, i)), rate, state, **how)
        same(step, f["y"][:, :, t], f["y_err"][:, :, t], io, t)


@pytest.mark.parametrize("B,H,T,D", [(1, 1, 1300, 64), (1, 4, 1100, 64), (2, 16, 300, 64), (40, 16, 150, 64), (1, 1, 17, 8)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_infinite_states_in_clusters_of_every_size(B, H, T, D, io):
    x, g, i, rate, h0, gy, ghT = make(B, H, T, D, io, "log")
    h0[0, 0, 1] = INF
    x[-1, -1, T // 2, 2] = -INF
    ghT[0, 0, 3] = INF
    check(x, g, i, rate, h0, gy, ghT, io, {"decay": "log", "scale": "sqrt"})


def check(x, g, i, rate, h0, gy, ghT, io, how):
    y, hT, kept = kla.recurrence_forward(x, g, i, rate, h0, checkpoints=True, **how)
    d = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, checkpoints=kept, **how)
    args = [f64(t) for t in (x, g, i, rate, h0)]
    with np.errstate(all="ignore"):
        f = R.forward(*args, **how)
        want = R.backward(*args, f64(gy), f64(ghT), **how)
    same(y, f["y"], f["y_err"], io, "y")
    same(hT, f["hT"], f["hT_err"], "f32", "hT")
    for n, t in d.items():
        same(t, want[n], want[n + "_err"], "f32" if n in ("grate", "gh0") else io, n)
    again = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, **how)
    assert all(torch.equal(torch.nan_to_num(d[n]), torch.nan_to_num(again[n])) for n in d)


@pytest.mark.parametrize("decay,scale", KINDS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
def test_gradients_with_infinite_states(decay, scale, io, gate):
    """gy and ghT are positive, so that every G is and an infinite dL/dlog a has the state's sign. (An infinite x under
    "none": the oracle multiplies it by the derivative zero of s, a term that is not there.)"""
    x, g, i, rate, h0, gy, ghT = make(2, 2, 201, 64, io, decay)
    h0[0, 0, 3], h0[0, 1, 8] = INF, -INF
    if scale != "none":
        x[1, 0, 77, 5], x[1, 1, 130, 6] = INF, -INF
    gy[0, 1, 150, 9], ghT[1, 1, 10] = INF, INF
    check(x, g, i if gate else None, rate, h0, gy, ghT, io, {"decay": decay, "scale": scale})


def test_infinite_states_in_place_and_in_parts_of_wider_tensors():
    """The last state over the first, outputs between another tensor's columns, and channels that no block fills."""
    B, H, T, D = 1, 3, 130, 24
    wide, out = torch.randn(B, T, 3, H * D, device=DEV), torch.zeros(B, T, 2, H * D, device=DEV)
    x, g, i = (wide[:, :, n].unflatten(-1, (H, D)).transpose(1, 2) for n in range(3))
    g.copy_(-g.abs())
    h0 = torch.randn(B, H, D, device=DEV)
    h0[0, 0, 0], h0[0, 2, 23] = INF, -INF
    x[0, 1, 128, 4] = INF
    how = {"decay": "log", "scale": "complement"}
    with np.errstate(all="ignore"):
        f = R.forward(*[f64(t) for t in (x, g, i)], h0=f64(h0), **how)
    y = out[:, :, 1].unflatten(-1, (H, D)).transpose(1, 2)
    state = h0.clone()
    kla.recurrence_forward(x, g, i, None, state, y=y, hT=state, **how)
    same(y, f["y"], f["y_err"], "f32", "y")
    same(state, f["hT"], f["hT_err"], "f32", "hT")
    assert not bool(out[:, :, 0].any())


def test_a_channel_of_which_one_half_is_nan():
    """Two channels share a thread: one NaN from the start, the other infinite later, forward and backward."""
    x, g, i, rate, h0, gy, ghT = make(1, 1, 300, 64, "f32", "rate")
    x[0, 0, 0, 10], x[0, 0, 200, 11] = float("nan"), INF
    ghT[0, 0, 20], gy[0, 0, 100, 21] = float("nan"), INF
    check(x, g, i, rate, h0, gy, ghT, "f32", {"decay": "rate", "scale": "sqrt"})
