"""fp64 oracle of the layer norm (numpy) and its gradients, from the definition,
with bounds of what arithmetic in 24 bits may be off by (u = 2^-24).

A row's sum is added up in at most 64 steps and eight levels of exchanges, 80 u
of the sum of its absolute values with what is around it."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def _row_sum_err(x):
    return 80 * U * np.abs(x).mean(-1, keepdims=True)


def normalised(x, eps):
    """The normalised rows n, 1/sqrt(var + eps), and bounds of n's error and of the other's relative error."""
    mean = x.mean(-1, keepdims=True)
    d = x - mean
    r = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n = d * r
    mean_err = _row_sum_err(x)
    # the differences' common error adds its square to the variance, the sums and the root 100 u
    r_err = 100 * U + 0.5 * (mean_err * r) ** 2 + 4 * U * (np.abs(x) * r).mean(-1, keepdims=True)
    return n, r, r * (mean_err + 2 * U * (np.abs(x) + np.abs(mean))) + np.abs(n) * r_err, r_err


def forward(x, weight=None, bias=None, eps=1e-5):
    """y of rows x ``[N,D]`` and the bound of its error."""
    n, _, n_err, _ = normalised(x, eps)
    w = 1.0 if weight is None else weight
    y = n * w + (0.0 if bias is None else bias)
    return y, n_err * np.abs(w) + 3 * U * (np.abs(n * w) + np.abs(y))


def backward(x, weight=None, gy=None, gtotal=None, eps=1e-5):
    """gx, gweight, gbias with their bounds."""
    n, r, n_err, r_err = normalised(x, eps)
    g = np.zeros_like(x) if gy is None else gy
    rows = 160 + x.shape[0] / 64  # roundings in a row when rows are added up
    out = {"gweight": (g * n).sum(0), "gweight_err": (np.abs(g) * n_err + rows * U * np.abs(g * n)).sum(0),
           "gbias": g.sum(0), "gbias_err": rows * U * np.abs(g).sum(0)}
    if weight is not None:
        g = g * weight
    s1, s2 = g.mean(-1, keepdims=True), (g * n).mean(-1, keepdims=True)
    s1_err = _row_sum_err(g) + U * np.abs(g).mean(-1, keepdims=True)
    s2_err = _row_sum_err(g * n) + (np.abs(g) * n_err).mean(-1, keepdims=True)
    inner = g - s1 - n * s2
    out["gx"] = r * inner + (0.0 if gtotal is None else gtotal)
    out["gx_err"] = (r * (s1_err + np.abs(n) * s2_err + n_err * (np.abs(s2) + s2_err)
                          + 4 * U * (np.abs(g) + np.abs(s1) + np.abs(n * s2)) + r_err * np.abs(inner))
                     + 2 * U * np.abs(out["gx"]))
    return out
