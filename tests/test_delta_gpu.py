"""The gated delta rule on the GPU against the fp64 oracle (oracle/delta.py).

Tolerances. For ‖k‖ ≤ 1, 0 ≤ β ≤ 2 and g ≤ 0 a token's map is a contraction,
so roundings do not grow: each token adds sums of dk terms, off by about
√dk · 2^-24 of the largest value, T of them add in quadrature, and the worst of
a tensor's elements is taken as sixteen times the typical one:
16 · 2^-24 · √(dk · max(T, 16)) of the largest value for fp32. The decay's
gradient sums dk · dv products more per token. bf16 outputs are off by another
half step, 2^-8 of the value, and may come from operands kept to 16 bits:
2^-10 of the largest value (2^-16, eight for the sums' growth, eight for the
worst element)."""
import numpy as np
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from oracle import delta as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def problem(B, Hk, H, T, dk, dv, io, seed=0, state=True, correlated=0.5, decay=1.0):
    r = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=r)

    k = randn(B, Hk, T, dk) + correlated * randn(B, Hk, 1, dk)
    q = randn(B, Hk, T, dk)
    p = {"q": q / q.norm(dim=-1, keepdim=True).clamp_min(1e-6), "k": 0.996 * k / k.norm(dim=-1, keepdim=True).clamp_min(1e-6),
         "v": randn(B, H, T, dv), "g": -decay * torch.rand(B, H, T, generator=r) ** 3,
         "beta": torch.sigmoid(randn(B, H, T))}
    p = {n: x.to(DT[io]) for n, x in p.items()}
    p["state0"] = randn(B, H, dk, dv) if state else None
    return p


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def to_dev(p):
    return {n: None if x is None else x.to(DEV) for n, x in p.items()}


def near(got, want, io, dk, T, what, extra=0):
    got = f64(got)
    assert got.shape == want.shape, what
    if want.size == 0:
        return
    top = np.abs(want).max()
    tol = 16 * 2.0 ** -24 * np.sqrt(dk * max(T, 16) + extra) * top
    err = np.abs(got - want)
    if io == "bf16":
        err = err - 2.0 ** -8 * np.abs(want)
        tol = tol + 2.0 ** -10 * top
    assert err.max() <= tol + 1e-30, f"{what}: {err.max():.3g} > {tol:.3g} (largest {top:.3g})"


def check_forward(p, io, scale=0.3, **kw):
    d = to_dev(p)
    o, S = kla.delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state0"], scale=scale, **kw)
    n = {x: f64(y) for x, y in p.items()}
    wo, wS, _ = O.forward(n["q"], n["k"], n["v"], n["g"], n["beta"], n["state0"], scale)
    dk, T = p["k"].shape[-1], p["k"].shape[2]
    near(o, wo, io, dk, T, "o")
    near(S, wS, "f32", dk, T, "stateT")
    return o, S


def check_backward(p, io, scale=0.3, go=True, gs=True, seed=9):
    r = torch.Generator().manual_seed(seed)
    B, H, T, dv = p["v"].shape
    dk = p["k"].shape[-1]
    go = torch.randn(B, H, T, dv, generator=r).to(DT[io]) if go else None
    gs = torch.randn(B, H, dk, dv, generator=r) if gs else None
    d = to_dev(p)
    got = kla.delta_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state0"],
                             go=None if go is None else go.to(DEV), gstateT=None if gs is None else gs.to(DEV),
                             scale=scale)
    n = {x: f64(y) for x, y in p.items()}
    want = O.backward(n["q"], n["k"], n["v"], n["g"], n["beta"], n["state0"], f64(go), f64(gs), scale)
    for x, y in got.items():
        near(y, want[x], "f32" if x == "gstate0" else io, dk, T, x, dk * dv if x == "gg" else 0)
    return got


SHAPES = [(1, 1, 1, 1, 16, 16), (2, 1, 2, 2, 16, 32), (1, 2, 2, 15, 32, 16), (1, 1, 3, 16, 64, 64),
          (1, 2, 4, 17, 32, 64), (2, 2, 2, 63, 64, 64), (1, 1, 1, 64, 128, 128), (1, 2, 4, 65, 64, 128),
          (1, 1, 2, 129, 128, 64), (1, 1, 2, 200, 64, 16), (1, 1, 1, 257, 16, 128), (1, 1, 1, 150, 128, 32)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, io):
    check_forward(problem(*shape, io, seed=sum(shape)), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_forward_long(io):
    check_forward(problem(1, 1, 2, 1500, 64, 64, io, seed=4, decay=0.05), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, io):
    check_backward(problem(*shape, io, seed=sum(shape)), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_backward_long(io):
    check_backward(problem(1, 1, 2, 700, 64, 64, io, seed=4, decay=0.05), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 2, 513, 128, 128), (1, 2, 2, 640, 128, 64), (2, 1, 1, 705, 128, 16)])
def test_wide_keys_over_many_chunks(shape, io):
    """Few heads of d_k = 128 and more than eight chunks, forward and from the end."""
    p = problem(*shape, io, seed=sum(shape), decay=0.05)
    p["g"][:, :, 100:102] = -float("inf")
    p["g"][:, :, 448] = -60.0
    check_forward(p, io)
    check_backward(p, io)
    p["state0"] = None
    check_forward(p, io)
    check_backward(p, io, gs=False)


def hard(name, p):
    if name == "resets":            # decays of exactly zero, alone and side by side, at chunk borders too
        for t in (0, 5, 15, 16, 63, 64, 65, 99):
            p["g"][:, :, t] = -float("inf")
    elif name == "strong decay":
        p["g"].fill_(-30.0)
    elif name == "mixed decay":     # strong and none in turn: differences of large sums
        p["g"].zero_()
        p["g"][:, :, ::7] = -90.0
    elif name == "no decay":
        p["g"].zero_()
    elif name == "no writes":
        p["beta"].zero_()
    elif name == "zero keys":
        p["k"][:, :, ::3] = 0
    elif name == "one key":         # every token writes over the last one
        p["k"].copy_(p["k"][:, :, :1].expand_as(p["k"]).clone())
        p["beta"].fill_(1.0)
        p["g"].zero_()
    elif name == "reflections":     # β = 2: eigenvalues of −1
        p["beta"].fill_(2.0)
        p["k"] /= 1.001
    elif name == "orthogonal keys":
        p["k"].zero_()
        for t in range(p["k"].shape[2]):
            p["k"][:, :, t, t % p["k"].shape[3]] = 1
        p["beta"].fill_(1.0)
    return p


HARD = ["resets", "strong decay", "mixed decay", "no decay", "no writes", "zero keys", "one key", "reflections",
        "orthogonal keys"]


@pytest.mark.parametrize("name", HARD)
@pytest.mark.parametrize("io,dk,dv", [("f32", 64, 64), ("bf16", 64, 64), ("bf16", 128, 128), ("f32", 32, 64)])
def test_hard_inputs(name, io, dk, dv):
    p = hard(name, problem(1, 1, 2, 130, dk, dv, io, seed=8))
    check_forward(p, io)
    check_backward(p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_without_states_and_with_parts_of_the_gradient(io):
    p = problem(1, 2, 2, 70, 64, 64, io, state=False)
    check_forward(p, io)
    d = to_dev(p)
    o, S = kla.delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.3, final_state=False)
    assert S is None
    assert torch.equal(o, kla.delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.3)[0])
    check_backward(p, io)
    check_backward(p, io, go=False)
    check_backward(p, io, gs=False)
    z = check_backward(p, io, go=False, gs=False)
    assert all(float(x.abs().max()) == 0 for x in z.values())


def test_default_scale_and_given_outputs():
    p = to_dev(problem(1, 1, 1, 20, 64, 32, "f32"))
    o, S = torch.empty_like(p["v"]), p["state0"].clone()
    a = kla.delta_forward(p["q"], p["k"], p["v"], p["g"], p["beta"], S, o=o, stateT=S)  # the state in place
    b = kla.delta_forward(p["q"], p["k"], p["v"], p["g"], p["beta"], p["state0"], scale=64 ** -0.5)
    assert a[0] is o and a[1] is S and torch.equal(o, b[0]) and torch.equal(S, b[1])


def test_state_in_place_over_a_long_sequence():
    p = to_dev(problem(1, 1, 3, 300, 128, 128, "bf16"))
    S = p["state0"].clone()
    a = kla.delta_forward(p["q"], p["k"], p["v"], p["g"], p["beta"], S, stateT=S)
    b = kla.delta_forward(p["q"], p["k"], p["v"], p["g"], p["beta"], p["state0"])
    assert torch.equal(a[0], b[0]) and torch.equal(S, b[1])


@pytest.mark.parametrize("T", [0, 1])
def test_empty_and_single(T):
    p = to_dev(problem(2, 1, 2, T, 64, 64, "bf16"))
    o, S = kla.delta_forward(p["q"], p["k"], p["v"], p["g"], p["beta"], p["state0"])
    assert o.shape == (2, 2, T, 64)
    if T == 0:
        assert torch.equal(S, p["state0"])
        z = kla.delta_forward(p["q"], p["k"], p["v"], p["g"], p["beta"])[1]
        assert float(z.abs().max()) == 0
        g = kla.delta_backward(p["q"], p["k"], p["v"], p["g"], p["beta"], p["state0"], gstateT=S)
        assert torch.equal(g["gstate0"], S) and g["gk"].shape == p["k"].shape
        assert float(kla.delta_backward(p["q"], p["k"], p["v"], p["g"], p["beta"])["gstate0"].abs().max()) == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("cuts", [(1,), (64,), (50, 51), (16, 64, 128)])
def test_pieces_equal_one_pass(io, cuts):
    p = problem(1, 1, 2, 140, 64, 64, io, seed=3)
    want, last = check_forward(p, io)
    d = to_dev(p)
    S, parts, at = d["state0"], [], 0
    for t in (*cuts, 140):
        x = {n: d[n][:, :, at:t].contiguous() for n in ("q", "k", "v", "g", "beta")}
        o, S = kla.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], S, scale=0.3)
        parts.append(o)
        at = t
    near(torch.cat(parts, 2), f64(want), io, 64, 140, "pieces")
    near(S, f64(last), "f32", 64, 140, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,H,dk,dv", [(1, 1, 1, 16, 16), (3, 2, 4, 32, 64), (2, 1, 2, 64, 128), (5, 2, 2, 128, 32),
                                          (1, 4, 8, 128, 128)])
def test_step(B, Hk, H, dk, dv, io):
    p = problem(B, Hk, H, 5, dk, dv, io, seed=dk + dv)
    if H > 1:
        p["g"][0, 0, 3] = -float("inf")
    n = {x: f64(y) for x, y in p.items()}
    want, last, _ = O.forward(n["q"], n["k"], n["v"], n["g"], n["beta"], n["state0"], 0.3)
    d = to_dev(p)
    S = d["state0"]
    for t in range(5):
        x = {m: d[m][:, :, t].contiguous() for m in ("q", "k", "v", "g", "beta")}
        x = {m: (y.clone() if m in ("q", "k", "v") else y) for m, y in x.items()}
        o = kla.delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], S, scale=0.3)
        near(o, want[:, :, t], io, dk, 5, f"o of token {t}")
    near(S, last, "f32", dk, 5, "state")


def test_a_value_that_is_no_number_stays_in_its_column_and_chunk():
    """Not before the 64 tokens around it, not in other columns or heads."""
    p = problem(1, 1, 2, 200, 64, 64, "bf16")
    clean = to_dev(p)
    a = kla.delta_forward(*(clean[n] for n in ("q", "k", "v", "g", "beta", "state0")))
    p["v"][0, 1, 130, 7] = float("nan")
    d = to_dev(p)
    b = kla.delta_forward(*(d[n] for n in ("q", "k", "v", "g", "beta", "state0")))
    assert torch.equal(a[0][0, 0], b[0][0, 0]) and torch.equal(a[0][:, :, :128], b[0][:, :, :128])
    assert bool(b[0][0, 1, 130:, 7].isnan().all()) and bool(b[1][0, 1, :, 7].isnan().all())
    other = [j for j in range(64) if j != 7]
    assert torch.equal(a[0][..., other], b[0][..., other]) and torch.equal(a[1][..., other], b[1][..., other])


def test_repeated_backward_gives_identical_bits():
    p = problem(2, 1, 4, 300, 64, 64, "bf16")
    a, b = check_backward(p, "bf16"), check_backward(p, "bf16")
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_autograd_and_another_stream():
    p = problem(1, 1, 2, 90, 64, 64, "f32")
    leaves = {n: x.to(DEV).requires_grad_() for n, x in p.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, S = kla.delta_rule(*(leaves[n] for n in ("q", "k", "v", "g", "beta", "state0")), scale=0.3)
        w, u = torch.randn_like(o), torch.randn_like(S)
        ((o * w).sum() + (S * u).sum()).backward()
    torch.cuda.current_stream().wait_stream(side)
    d = {n: x.detach() for n, x in leaves.items()}
    g = kla.delta_backward(*(d[n] for n in ("q", "k", "v", "g", "beta", "state0")), go=w, gstateT=u, scale=0.3)
    for n, x in leaves.items():
        assert torch.equal(x.grad, g["g" + n]), n


def test_gradient_against_differences():
    p = to_dev(problem(1, 1, 1, 70, 16, 16, "f32", decay=0.2))
    names = ("q", "k", "v", "g", "beta", "state0")
    r = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randn(p["v"].shape, generator=r, device=DEV)

    def loss(q):
        return float((kla.delta_forward(*(q[n] for n in names), scale=1.0)[0].double() * w).sum())

    g = kla.delta_backward(*(p[n] for n in names), go=w, scale=1.0)
    for n in names:
        x = torch.randn(p[n].shape, generator=r, device=DEV)
        x = x / x.norm()
        h = 2.0 ** -7
        up, down = ({**p, n: p[n] + s * h * x} for s in (1, -1))
        d = (loss(up) - loss(down)) / (2 * h)
        want = float((g["g" + n].double() * x).sum())
        # the difference: fp32 sums of ~1e3 terms over 2h, and the third derivative's h²
        assert abs(d - want) <= 2e-3 * max(1.0, float(g["g" + n].norm())), (n, d, want)


def test_captured_calls_replay():
    p = to_dev(problem(1, 2, 4, 100, 64, 64, "bf16"))
    names = ("q", "k", "v", "g", "beta", "state0")
    go = torch.randn_like(p["v"])
    nbytes = kla.LIB.kla_delta_backward_workspace_size(1, 2, 4, 100, 64, 64)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    S = p["state0"].clone()
    tok = {n: p[n][:, :, 0].contiguous() for n in names[:5]}

    def calls():
        o, last = kla.delta_forward(*(p[n] for n in names))
        g = kla.delta_backward(*(p[n] for n in names), go=go, workspace=ws)
        y = kla.delta_step(*(tok[n] for n in names[:5]), S)
        return [o, last, y, *g.values()]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    S.copy_(p["state0"])
    p["v"].copy_(torch.randn_like(p["v"]))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in out]
    S.copy_(p["state0"])
    for a, b in zip(got, calls()):
        assert torch.equal(a, b)


def test_binding_refuses():
    p = to_dev(problem(1, 1, 2, 8, 16, 16, "f32"))
    args = [p[n] for n in ("q", "k", "v", "g", "beta")]
    for i, bad in ((1, p["k"].bfloat16()), (2, p["v"].transpose(2, 3).contiguous().transpose(2, 3)), (3, p["g"][:, :, :4]),
                   (4, p["beta"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            kla.delta_forward(*(bad if j == i else x for j, x in enumerate(args)))
    with pytest.raises((TypeError, ValueError)):
        kla.delta_forward(*args, p["state0"].bfloat16())
    with pytest.raises(kla.KlaError):
        kla.delta_forward(*(torch.cat([x] * 3, 1) if i < 2 else x for i, x in enumerate(args)))  # 3 key heads, 2 value heads
