"""A CPU model of the delta rule's chunked form with its operands held as bf16
parts: three parts leave outputs and states far inside 2^-20 of the 64-bit values
(2-norm), the bound that the GPU tests hold fp32 results to on the same problem;
with two parts in any one place they are outside it."""
import numpy as np
import pytest

C = 64


def bf16(x):
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32).reshape(np.shape(x))


def parts(x, n):
    """x as the sum of n bf16 values."""
    rest, out = np.asarray(x, np.float32), np.zeros(np.shape(x))
    for _ in range(n):
        p = bf16(rest)
        out, rest = out + p.astype(np.float64), rest - p
    return out


def problem(T, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    return (unit(r.standard_normal((T, dk))), unit(r.standard_normal((T, dk)) + 0.5 * r.standard_normal(dk)),
            r.standard_normal((T, dv)), -0.002 * r.random(T) ** 3, 2 / (1 + np.exp(-r.standard_normal(T))),
            r.standard_normal((dk, dv)))


def by_tokens(q, k, v, g, b, S):
    o = np.zeros_like(v)
    for t in range(len(q)):
        S = np.exp(g[t]) * S
        S = S + np.outer(k[t], b[t] * (v[t] - S.T @ k[t]))
        o[t] = S.T @ q[t]
    return o, S


def by_chunks(q, k, v, g, b, S, n):
    """n: the parts of each of W, X, U, P (states and updates in fp32, products of parts exact)."""
    f32 = lambda x: np.asarray(x, np.float32).astype(np.float64)
    o = []
    for i in range(0, len(q), C):
        Q, K, V, B = (parts(x[i:i + C], 3) for x in (q, k, v, b[:, None]))
        c = np.cumsum(g[i:i + C])
        D = np.tril(np.exp(c[:, None] - c[None, :]))
        G, E = np.exp(c)[:, None], np.exp(c[-1] - c)[:, None]
        M = np.linalg.inv(np.eye(len(c)) + np.tril(B * D * (K @ K.T), -1))
        W = parts(-M @ (B * G * K), n["W"])
        U = f32(f32(M @ (B * V)) + W @ parts(S, n["X"]))
        o.append(G * (Q @ parts(S, n["S"])) + parts(D * (Q @ K.T), n["P"]) @ parts(U, n["U"]))
        S = f32(G[-1] * S + K.T @ parts(E * U, n["EU"]))
    return np.concatenate(o), S


def errors(less=""):
    p = problem(640, 64, 64)
    p = tuple(np.asarray(x, np.float32).astype(np.float64) for x in p)
    n = {x: 2 if x == less else 3 for x in ("W", "X", "S", "P", "U", "EU")}
    got, want = by_chunks(*p, n), by_tokens(*p)
    return [np.linalg.norm(x - y) / np.linalg.norm(y) for x, y in zip(got, want)]


def test_three_parts_are_within_the_bound():
    assert max(errors()) <= 2.0 ** -20 / 4


@pytest.mark.parametrize("less", ["W", "X", "S", "P", "U", "EU"])
def test_two_parts_are_not(less):
    assert max(errors(less)) > 2.0 ** -20
