"""fp64 oracle of the gated delta rule and its gradients, token by token, in
the definition's own order (numpy; nothing shared with the CUDA path):

    u = β (v − a Sᵀk),   S ← a S + k uᵀ,   o = scale · Sᵀq,   a = e^g

q, k ``[B,Hk,T,dk]``, v ``[B,H,T,dv]``, g, beta ``[B,H,T]``; value head h reads
key head h // (H // Hk). ``mistake`` plants an error for the pins.
"""
from __future__ import annotations

import numpy as np


def _heads(x, H):
    return np.repeat(x, H // x.shape[1], axis=1) if x.shape[1] else x


def forward(q, k, v, g, beta, state0=None, scale=1.0, mistake: str = ""):
    """``(o, stateT, history)``; history holds S before every token and what
    each token found missing, v − a Sᵀk."""
    H = v.shape[1]
    q, k = _heads(q, H), _heads(k, H)
    B, _, T, dk = k.shape
    dv = v.shape[-1]
    S = np.zeros((B, H, dk, dv)) if state0 is None else state0.astype(np.float64).copy()
    o, before, missed = np.zeros((B, H, T, dv)), [], []
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(T):
            a = np.exp(g[:, :, t])[..., None, None]
            before.append(S)
            if mistake == "read before write":
                o[:, :, t] = scale * np.einsum("bhij,bhi->bhj", S, q[:, :, t])
            seen = S if mistake == "undecayed prediction" else a * S
            m = v[:, :, t] - np.einsum("bhij,bhi->bhj", seen, k[:, :, t])
            missed.append(m)
            S = a * S + k[:, :, t][..., None] * (beta[:, :, t][..., None] * m)[..., None, :]
            if mistake != "read before write":
                o[:, :, t] = scale * np.einsum("bhij,bhi->bhj", S, q[:, :, t])
    return o, S, (before, missed)


def backward(q, k, v, g, beta, state0=None, go=None, gstateT=None, scale=1.0, mistake: str = ""):
    """Reverse mode of :func:`forward`: a dict of gradients."""
    Hk, H = k.shape[1], v.shape[1]
    _, last, (before, missed) = forward(q, k, v, g, beta, state0, scale)
    qh, kh = _heads(q, H), _heads(k, H)
    B, _, T, dk = kh.shape
    Z = np.zeros_like(last) if gstateT is None else gstateT.astype(np.float64).copy()
    gq, gk, gv = np.zeros_like(qh), np.zeros_like(kh), np.zeros_like(v)
    gg, gb = np.zeros_like(g), np.zeros_like(beta)
    after = last
    for t in reversed(range(T)):
        a, b = np.exp(g[:, :, t])[..., None, None], beta[:, :, t][..., None]
        kt, qt, S = kh[:, :, t], qh[:, :, t], before[t]
        if go is not None:
            gq[:, :, t] = scale * np.einsum("bhij,bhj->bhi", after, go[:, :, t])
            Z = Z + qt[..., None] * (scale * go[:, :, t])[..., None, :]
        gu = np.einsum("bhij,bhi->bhj", Z, kt)
        gb[:, :, t] = (gu * missed[t]).sum(-1)
        gm = b * gu
        gv[:, :, t] = gm
        gk[:, :, t] = np.einsum("bhij,bhj->bhi", Z, b * missed[t])
        if mistake != "no gradient through the prediction":
            gk[:, :, t] -= np.einsum("bhij,bhj->bhi", a * S, gm)
            Z = Z - kt[..., None] * gm[..., None, :]
        Z = a * Z
        gg[:, :, t] = (Z * S).sum((-2, -1)) if mistake != "decay of the written state" else (Z * after).sum((-2, -1))
        after = S
    gq, gk = (x.reshape(B, Hk, H // max(Hk, 1), T, dk).sum(2) for x in (gq, gk))
    return {"gq": gq, "gk": gk, "gv": gv, "gg": gg, "gbeta": gb, "gstate0": Z}
