"""How many bits the gated delta rule's chunked kernels keep.

Everything that is not an input is held to 24 bits, so a bf16 call is the fp32
result rounded once."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from test_delta_gpu import DEV, problem, to_dev

pytestmark = pytest.mark.gpu


def close_values(*shape, seed):
    """1.71 and m 2^-20 more, 0 ≤ m < 256: 21 bits, set all over them."""
    r = torch.Generator().manual_seed(seed)
    return (1 + 2925 * 2.0 ** -12 + torch.randint(0, 256, shape, generator=r) * 2.0 ** -20).to(DEV)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (32, 128)])
def test_differences_of_states_are_exact(io, dk, dv):
    """Outputs and gradients that are differences of two close entries of a state.
    Each entry and their sum may be off by half a unit of 24 bits (2^-24 of a
    value below 2, three times: less than 2^-21, half of the states' steps); the
    difference is a value of at most eight bits, so its rounding to bf16 is
    exact. Operands of 16 bits are 2^-17 off."""
    B, H, T = 1, 2, 600
    zero = lambda *s: torch.zeros(*s, dtype=io, device=DEV)
    q, k, v = zero(B, H, T, dk), zero(B, H, T, dk), zero(B, H, T, dv)
    S, Z = close_values(B, H, dk, dv, seed=1), close_values(B, H, dk, dv, seed=2)
    gate, one = zero(B, H, T), zero(B, H, T) + 1
    q[..., 0], q[..., 1] = 1, -1
    o, last = kla.delta_forward(q, k, v, gate, one, S, scale=1.0)
    want = (S[:, :, 0] - S[:, :, 1])[:, :, None].expand(B, H, T, dv)
    assert torch.equal(last, S)
    assert float((o.float() - want).abs().max()) <= 2.0 ** -21
    q.zero_()
    v[..., 0], v[..., 1] = 1, -1
    g = kla.delta_backward(q, k, v, gate, one, S, go=v, gstateT=Z, scale=1.0)
    for n, x in (("gq", S), ("gk", Z)):
        want = (x[..., 0] - x[..., 1])[:, :, None].expand(B, H, T, dk)
        assert float((g[n].float() - want).abs().max()) <= 2.0 ** -21, n


@pytest.mark.parametrize("shape", [(2, 8, 8, 700, 64, 64), (2, 4, 8, 700, 128, 128)])
def test_bf16_is_fp32_rounded_once(shape):
    """The bf16 call against the fp32 call on the same values, rounded. Where the
    two differ by e before the rounding, a share 2 e / step of the values goes
    the other way, each by a step (2^-7 of the value at most): √(e · 2^-7) in the
    2-norm. Both are within 2^-21 of the exact values, so e ≤ 2^-20 and the bound
    is 8.6e-5 (operands of 16 bits give 1.2e-4 and more)."""
    p = problem(*shape, "bf16", seed=5, decay=0.1)
    r = torch.Generator().manual_seed(6)
    go = torch.randn(p["v"].shape, generator=r).bfloat16().to(DEV)
    gs = torch.randn(p["state0"].shape, generator=r).to(DEV)
    d = to_dev(p)
    names = ("q", "k", "v", "g", "beta")
    wide = {n: d[n].float() for n in names}
    o, last = kla.delta_forward(*(d[n] for n in names), d["state0"])
    o32, last32 = kla.delta_forward(*(wide[n] for n in names), d["state0"])
    a = kla.delta_backward(*(d[n] for n in names), d["state0"], go=go, gstateT=gs)
    b = kla.delta_backward(*(wide[n] for n in names), d["state0"], go=go.float(), gstateT=gs)
    for n, x, y in (("o", o, o32), *((n, a[n], b[n]) for n in ("gq", "gk", "gv"))):
        y = y.bfloat16().double()
        far = float((x.double() - y).norm() / y.norm())
        assert far <= (2.0 ** -20 * 2.0 ** -7) ** 0.5, (n, far)
    for x, y in ((last, last32), (a["gstate0"], b["gstate0"])):
        assert float((x - y).norm() / y.norm()) <= 2.0 ** -20


def by_tokens(q, k, v, g, beta, S, scale):
    """The definition in 64 bits, token by token, on the GPU."""
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    a, o = g.exp(), torch.empty_like(v)
    for t in range(q.shape[2]):
        S = S * a[:, :, t, None, None]
        missed = v[:, :, t] - (k[:, :, t].unsqueeze(-2) @ S).squeeze(-2)
        S = S + k[:, :, t].unsqueeze(-1) * (beta[:, :, t, None] * missed).unsqueeze(-2)
        o[:, :, t] = (q[:, :, t].unsqueeze(-2) @ S).squeeze(-2) * scale
    return o, S


def weak(B, H, T, dk, dv, g, beta):
    """Decays and writes so weak that the first tokens still matter at the end."""
    r = torch.Generator(device=DEV).manual_seed(7)
    randn = lambda *s: torch.randn(*s, generator=r, device=DEV)
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)
    return (unit(randn(B, H, T, dk)), unit(randn(B, H, T, dk)), randn(B, H, T, dv),
            torch.full((B, H, T), g, device=DEV), torch.full((B, H, T), beta, device=DEV), randn(B, H, dk, dv))


def rel(x, y):
    return float((x.double() - y).norm() / y.norm())


@pytest.mark.parametrize("B,H,T,dk,g", [(8, 128, 512, 16, -1e-5), (8, 128, 512, 16, -2e-6), (8, 128, 256, 32, -1e-5),
                                        (8, 128, 256, 32, -0.003), (1, 8, 40, 64, -1e-5), (8, 128, 200, 16, -0.4)])
def test_weak_decays_one_token_at_a_time(B, H, T, dk, g):
    """The same weak decay for every token. Each token rounds the state once, by
    2^-25 at most in the mean square, and T of them add in quadrature: √512 · 2^-25
    < 2^-20, the bound. The factors' own roundings would add up as they are, to
    2.4e-5."""
    args = weak(B, H, T, dk, dk, g, 0.002)
    assert kla.LIB.kla_delta_forward_workspace_size(B, H, H, T, dk, dk) == 0  # token by token
    o, S = kla.delta_forward(*args, scale=1.0)
    wo, wS = by_tokens(*args, 1.0)
    assert rel(o, wo) <= 2.0 ** -20 and rel(S, wS) <= 2.0 ** -20, (rel(o, wo), rel(S, wS))


def test_weak_decays_in_decode_tokens():
    """512 single tokens, held to the same bound."""
    args = weak(1, 8, 512, 64, 64, -1e-5, 0.002)
    wo, wS = by_tokens(*args, 1.0)
    S, o = args[-1].clone(), []
    for t in range(512):
        o.append(kla.delta_step(*(x[:, :, t].contiguous() for x in args[:5]), S, scale=1.0))
    assert rel(S, wS) <= 2.0 ** -20 and rel(torch.stack(o, 2), wo) <= 2.0 ** -20


@pytest.mark.parametrize("T,dk,g,beta", [(4096, 64, -1e-5, 0.01), (16384, 128, -2e-6, 0.001), (16384, 64, -1e-5, 0.002),
                                         (16384, 64, 0.0, 0.002), (8192, 64, -0.0001234, 0.02)])
def test_weak_decays_over_many_chunks(T, dk, g, beta):
    """The same weak decay for every token, over up to 256 chunks, forward and
    for the gradient of the first state. A chunk rounds the state a few times
    (the update's product and sum, four 2^-25 in the mean square): √256 · 2 ·
    2^-25 < 2^-20, the bound."""
    args = weak(1, 2, T, dk, 64, g, beta)
    o, S = kla.delta_forward(*args, scale=1.0)
    wo, wS = by_tokens(*args, 1.0)
    assert rel(o, wo) <= 2.0 ** -20 and rel(S, wS) <= 2.0 ** -20, (rel(o, wo), rel(S, wS))
    # the first state's gradient: Z ← a (Z − k β (kᵀZ)) from the end
    q, k, v, a, b = (x.double() for x in args[:5])
    Z = torch.randn(S.shape, generator=torch.Generator(device=DEV).manual_seed(8), device=DEV)
    got = kla.delta_backward(*args, gstateT=Z, scale=1.0)["gstate0"]
    Z, a = Z.double(), a.exp()
    for t in reversed(range(T)):
        u = b[:, :, t, None, None] * (k[:, :, t].unsqueeze(-2) @ Z)
        Z = a[:, :, t, None, None] * (Z - k[:, :, t].unsqueeze(-1) * u)
    assert rel(got, Z) <= 2.0 ** -20, rel(got, Z)
