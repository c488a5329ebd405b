"""Pins of the fp64 oracles of the gated delta rule (oracle/delta.py) and of
the norm with rotation (oracle/norm_rope.py): closed forms, invariances and
central differences, each of which a planted mistake must fail."""
import numpy as np
import pytest

from oracle import delta as O
from oracle import norm_rope as N


def problem(seed=0, B=1, Hk=2, H=4, T=6, dk=4, dv=3):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, Hk, T, dk))
    return {"q": r.standard_normal((B, Hk, T, dk)), "k": k / np.linalg.norm(k, axis=-1, keepdims=True),
            "v": r.standard_normal((B, H, T, dv)), "g": -r.random((B, H, T)), "beta": r.random((B, H, T)),
            "state0": r.standard_normal((B, H, dk, dv))}


def test_full_writes_of_unit_keys_are_read_back():
    """β = 1 and no decay: after the write, the state holds v under k exactly;
    orthogonal keys hold all of them (an associative memory)."""
    r = np.random.default_rng(0)
    keys = np.linalg.qr(r.standard_normal((4, 4)))[0][None, None]
    v = r.standard_normal((1, 1, 4, 3))
    zero, one = np.zeros((1, 1, 4)), np.ones((1, 1, 4))
    o, S, _ = O.forward(keys, keys, v, zero, one)
    assert np.allclose(o, v) and np.allclose(np.einsum("bhij,bhti->bhtj", S, keys), v)
    again = np.concatenate([keys, keys], 2)  # written again with other values: those replace the first
    w = r.standard_normal((1, 1, 4, 3))
    _, S, _ = O.forward(again, again, np.concatenate([v, w], 2), np.zeros((1, 1, 8)), np.ones((1, 1, 8)))
    assert np.allclose(np.einsum("bhij,bhti->bhtj", S, keys), w)


def test_product_form_of_the_state():
    """S_T = (Π a_t (I − β_t k_t k_tᵀ)) S_0 + Σ ... as matrices, one token at a time."""
    p = problem(Hk=4)
    S = p["state0"].copy()
    for t in range(6):
        for h in range(4):
            k, b = p["k"][0, h, t][:, None], p["beta"][0, h, t]
            S[0, h] = np.exp(p["g"][0, h, t]) * (np.eye(4) - b * k @ k.T) @ S[0, h] + b * k @ p["v"][0, h, t][None]
    assert np.allclose(O.forward(**p)[1], S)
    assert not np.allclose(O.forward(**p, mistake="undecayed prediction")[1], S)


def test_a_cut_sequence_equals_one_pass_and_a_reset_forgets():
    p = problem(T=7)
    o, S, _ = O.forward(**p)
    cut = {n: (x[:, :, :3] if n != "state0" else x) for n, x in p.items()}
    o1, S1, _ = O.forward(**cut)
    rest = {n: (x[:, :, 3:] if n != "state0" else S1) for n, x in p.items()}
    o2, S2, _ = O.forward(**rest)
    assert np.allclose(np.concatenate([o1, o2], 2), o) and np.allclose(S2, S)
    p["g"][:, :, 4] = -np.inf
    o, S, _ = O.forward(**p)
    tail = {n: (x[:, :, 4:] if n != "state0" else None) for n, x in p.items()}
    o2, S2, _ = O.forward(**tail)
    assert np.allclose(o[:, :, 4:], o2) and np.allclose(S, S2)
    assert not np.allclose(O.forward(**p, mistake="read before write")[0][:, :, 4:], o2)


def differences(f, x, h=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        out[i] = (up - f()) / (2 * h)
        x[i] = keep
    return out


def delta_error(mistake=""):
    p = problem(1, T=4)
    r = np.random.default_rng(2)
    go, gs = r.standard_normal(p["v"].shape), r.standard_normal(p["state0"].shape)

    def loss():
        o, S, _ = O.forward(**p, scale=0.7)
        return (o * go).sum() + (S * gs).sum()

    got = O.backward(**p, go=go, gstateT=gs, scale=0.7, mistake=mistake)
    worst = 0.0
    for n, x in p.items():
        want = differences(loss, x)
        worst = max(worst, np.abs(got["g" + n] - want).max() / np.abs(want).max())
    return worst


def test_delta_gradients_match_differences():
    assert delta_error() < 1e-7


@pytest.mark.parametrize("mistake", ["no gradient through the prediction", "decay of the written state"])
def test_planted_gradient_mistakes_are_caught(mistake):
    assert delta_error(mistake) > 1e-3


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_orthogonal_relative_and_partial(layout):
    f = np.array([1.0, 0.3])
    R = [N.rotation(p, f, 6, layout) for p in (0, 5, 9)]
    assert np.allclose(R[0], np.eye(6)) and np.allclose(R[1] @ R[1].T, np.eye(6))
    assert np.allclose(R[1].T @ R[2], N.rotation(4, f, 6, layout))  # the product of q and k sees 9 − 5
    assert np.allclose(R[1][4:], np.eye(6)[4:])
    pair = (0, 2) if layout == "half" else (0, 1)
    assert np.isclose(R[1][pair[1], pair[0]], np.sin(5.0)) and np.isclose(R[1][pair], -np.sin(5.0))


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_rope_gradients_match_differences(norm, layout):
    r = np.random.default_rng(3)
    x, w, gy = r.standard_normal((1, 2, 2, 6)), r.standard_normal(6), r.standard_normal((1, 2, 2, 6))
    pos, f = np.array([[3, 700]]), np.array([1.0, 0.3])

    def loss():
        return (N.forward(x, w, pos, f, norm, layout, 1e-3, 1.3) * gy).sum()

    gx, gw = N.backward(x, w, gy, pos, f, norm, layout, 1e-3, 1.3)
    assert np.allclose(gx, differences(loss, x), atol=1e-7) and np.allclose(gw, differences(loss, w), atol=1e-7)
    if norm != "none":  # the norm takes the row's length out
        small = N.forward(1e3 * x, np.ones(6), pos, f, norm, layout, 0.0)
        assert np.allclose((small ** 2).sum(-1), 1 if norm == "l2" else 6)
