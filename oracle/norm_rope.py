"""fp64 oracle of the per-head norm with the position rotation (numpy): the
rotation as a matrix, the norm from its definition, gradients from both."""
from __future__ import annotations

import numpy as np


def rotation(pos, inv_freq, D, layout, rot_scale=1.0):
    """The matrix that turns a row of D entries at one position: y = R x."""
    half = len(inv_freq)
    R = np.eye(D)
    for i, f in enumerate(inv_freq):
        p, q = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = np.cos(pos * float(f)), np.sin(pos * float(f))
        R[p, p] = R[q, q] = c * rot_scale
        R[p, q], R[q, p] = -s * rot_scale, s * rot_scale
    return R


def _sizes(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    m = (x * x).sum(-1, keepdims=True)
    return np.sqrt((m / x.shape[-1] if norm == "rms" else m) + eps)


def _matrices(positions, inv_freq, D, layout, rot_scale):
    B, T = positions.shape
    return np.stack([[rotation(int(positions[b, t]), inv_freq, D, layout, rot_scale) for t in range(T)]
                     for b in range(B)]).reshape(B, T, D, D)


def forward(x, w, positions, inv_freq, norm="rms", layout="half", eps=1e-6, rot_scale=1.0):
    """x ``[B,H,T,D]``, w ``[D]``, positions ``[B,T]``."""
    R = _matrices(positions, inv_freq, x.shape[-1], layout, rot_scale)
    return np.einsum("btij,bhtj->bhti", R, x / _sizes(x, norm, eps) * w)


def backward(x, w, gy, positions, inv_freq, norm="rms", layout="half", eps=1e-6, rot_scale=1.0):
    """(gx, gw)."""
    D = x.shape[-1]
    R = _matrices(positions, inv_freq, D, layout, rot_scale)
    gn = np.einsum("btij,bhti->bhtj", R, gy)
    z = _sizes(x, norm, eps)
    g = gn * w
    gx = g / z
    if norm != "none":
        gx = gx - x * (g * x).sum(-1, keepdims=True) / z ** 3 / (D if norm == "rms" else 1)
    return gx, (gn * x / z).sum((0, 1, 2))
