"""fp64 oracle of the gated linear recurrence (numpy), token by token from its
definition, with bounds of what arithmetic in 24 bits may be off by.

    h_t = a_t h_{t-1} + s(a_t) σ(i_t) x_t
    a = e^g ("log"), σ(g) ("sigmoid"), exp(-rate σ(g)) ("rate")
    s = 1 ("none"), sqrt(1 - a²) ("sqrt"), 1 - a ("complement")

Every function takes x, g, i ``[B,H,T,D]`` (i may be None), rate ``[H,D]``, h0
``[B,H,D]`` or None. The ``*_err`` entries are bounds: |h| <= ĥ, the recursion on
absolute values, and with u = 2^-24 a token adds to the state's error
  6 ĥ_t u               the roundings of its own update, and its share of those of the maps it is composed into
  (1 - a) c ĥ_{t-1} u   from the decay: 1 - a is known to c u of itself
  c s σ |x| u           from what is written
with c = 24 + 3 |g| + 3 |i|: a few roundings and special functions of 2 u each, and the argument of an exponential,
rounded, moves it by |argument| u.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def sigmoid(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def gates(g, i, rate, decay, scale):
    """a, 1 - a, s, ds/dlog a, σ(i), dlog a/dg, and σ(g)."""
    sg = sigmoid(g)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        la = {"log": lambda: g, "sigmoid": lambda: -np.logaddexp(0, -g), "rate": lambda: -rate[:, None] * sg}[decay]()
        a, less = np.exp(la), -np.expm1(la)
        size = {"none": lambda: np.ones_like(a), "sqrt": lambda: np.sqrt(np.maximum(less * (1 + a), 0)),
                "complement": lambda: less}[scale]()
        by_log = {"none": lambda: 0 * a, "sqrt": lambda: np.where(size > 0, -a * a / np.where(size > 0, size, 1), 0),
                  "complement": lambda: -a}[scale]()
    open_ = np.ones_like(a) if i is None else sigmoid(i)
    by_g = {"log": lambda: np.ones_like(a), "sigmoid": lambda: sigmoid(-g),
            "rate": lambda: -rate[:, None] * sg * sigmoid(-g)}[decay]()
    return a, less, size, by_log, open_, by_g, sg


def _coefficient(g, i):
    c = 24 + 3 * np.abs(np.where(np.isfinite(g), g, 0))
    return c if i is None else c + 3 * np.abs(i)


def forward(x, g, i=None, rate=None, h0=None, decay="log", scale="none"):
    """y, hT, and the bounds y_err, hT_err (all [B,H,T,D] or [B,H,D])."""
    a, less, size, _, open_, _, _ = gates(g, i, rate, decay, scale)
    c = _coefficient(g, i)
    h = np.zeros(x.shape[:2] + x.shape[3:]) if h0 is None else h0.astype(np.float64)
    top, err = np.abs(h), np.zeros_like(h)
    y, y_err, tops = np.empty(x.shape), np.empty(x.shape), np.empty(x.shape)
    for t in range(x.shape[2]):
        b = size[:, :, t] * open_[:, :, t] * x[:, :, t]
        err = a[:, :, t] * err + (np.abs(less[:, :, t]) * c[:, :, t] * top + c[:, :, t] * np.abs(b)) * U
        h = a[:, :, t] * h + b
        top = a[:, :, t] * top + np.abs(b)
        err = err + 6 * U * top
        y[:, :, t], y_err[:, :, t], tops[:, :, t] = h, err, top
    return {"y": y, "hT": h, "y_err": y_err, "hT_err": err, "top": tops}


def backward(x, g, i=None, rate=None, h0=None, gy=None, ghT=None, decay="log", scale="none"):
    """gx, gg, gi, grate, gh0, each with its bound *_err."""
    a, less, size, by_log, open_, by_g, sg = gates(g, i, rate, decay, scale)
    c = _coefficient(g, i)
    f = forward(x, g, i, rate, h0, decay, scale)
    start = np.zeros(x.shape[:2] + (1,) + x.shape[3:]) if h0 is None else h0[:, :, None].astype(np.float64)
    before = np.concatenate([start, f["y"][:, :, :-1]], 2)
    before_err = np.concatenate([0 * start, f["y_err"][:, :, :-1]], 2)
    Z = np.zeros(start[:, :, 0].shape) if ghT is None else ghT.astype(np.float64)
    top, err = np.abs(Z), np.zeros_like(Z)
    G, G_err, G_top = (np.empty(x.shape) for _ in range(3))
    for t in reversed(range(x.shape[2])):
        y = 0 if gy is None else gy[:, :, t]
        G[:, :, t], G_top[:, :, t] = Z + y, top + np.abs(y)
        G_err[:, :, t] = err + 6 * U * G_top[:, :, t]
        Z = a[:, :, t] * G[:, :, t]
        top = a[:, :, t] * G_top[:, :, t]
        err = a[:, :, t] * G_err[:, :, t] + np.abs(less[:, :, t]) * c[:, :, t] * G_top[:, :, t] * U
    xo = open_ * x
    inner, inner_top = a * before + by_log * xo, a * np.abs(before) + np.abs(by_log * xo)
    inner_err = a * before_err + (2 * c + 8) * U * inner_top
    log_, log_err = G * inner, G_err * np.abs(inner) + np.abs(G) * inner_err + G_err * inner_err
    out = {"gx": G * size * open_, "gx_err": np.abs(size * open_) * (G_err + c * U * np.abs(G)),
           "gg": log_ * by_g, "gg_err": np.abs(by_g) * (log_err + (c + 8) * U * np.abs(log_)), "gh0": Z, "gh0_err": err}
    if i is not None:
        p = size * open_ * x * sigmoid(-i)
        out["gi"], out["gi_err"] = G * p, np.abs(p) * (G_err + (2 * c + 8) * U * np.abs(G))
    if rate is not None:  # a sum over B and T: a thread adds up an eighth of a sequence, then come the blocks and the batch
        out["grate"] = -(log_ * sg).sum((0, 2))
        depth = x.shape[2] / 8 + 8 * x.shape[0] + 32
        out["grate_err"] = (sg * (log_err + (c + depth) * U * np.abs(log_))).sum((0, 2))
    return out
