"""A residual block as a model has it — layer norm with the residual sum, projections, causal convolution, gated linear
recurrence — trained through autograd and decoded one token at a time.

In fp32 against the same block in 64 bits on the CPU, written with torch: gradients pass through about 20 operations
and two projections of 48 inputs, so 2^-24 · (20 + 2 · 48) · 16 of the largest gradient bounds their error."""
import os
import re

import pytest
import torch
import torch.nn.functional as F

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, T, H, D, W = 2, 75, 3, 16, 4
C = H * D
TOL = 2.0 ** -24 * (20 + 2 * C) * 16


def parameters():
    r = torch.Generator().manual_seed(0)
    n = lambda *s, k=1.0: k * torch.randn(*s, generator=r)
    return {"norm_w": 1 + n(C, k=0.1), "norm_b": n(C, k=0.1), "w_x": n(C, C, k=C ** -0.5), "w_g": n(C, C, k=C ** -0.5),
            "w_i": n(C, C, k=C ** -0.5), "w_o": n(C, C, k=C ** -0.5), "taps": n(H, D, W, k=0.5),
            "rate": 0.05 + torch.rand(H, D, generator=r)}


def heads(t):
    return t.unflatten(-1, (H, D)).transpose(1, 2)


def block(p, x, residual, state=None, window=None):
    """Returns (what the block adds, total, the state and window behind the last token)."""
    n, total = kla.add_layer_norm(x, p["norm_w"], p["norm_b"], residual)
    c, window = kla.causal_conv(heads(n @ p["w_x"]).contiguous(), p["taps"], window=window)
    y, state = kla.gated_recurrence(c, heads(n @ p["w_g"]), heads(n @ p["w_i"]), p["rate"], state, decay="rate", scale="sqrt")
    return y.transpose(1, 2).flatten(2) @ p["w_o"], total, state, window


def token(p, x, residual, state, window):
    """The same for one token without gradients."""
    n, total = kla.layer_norm(x, p["norm_w"], p["norm_b"], residual)
    c, window = kla.conv(heads(n @ p["w_x"]).contiguous(), p["taps"], window=window, update_window=True)
    g, i = (heads(n @ p[w]).squeeze(2).contiguous() for w in ("w_g", "w_i"))
    y = kla.recurrence_step(c.squeeze(2), g, i, p["rate"], state, decay="rate", scale="sqrt")
    return y.flatten(1)[:, None] @ p["w_o"], total


def plain(p, x, residual):
    total = x + residual
    n = F.layer_norm(total, (C,), p["norm_w"], p["norm_b"])
    u = F.conv1d((n @ p["w_x"]).transpose(1, 2), p["taps"].reshape(C, 1, W), padding=W - 1, groups=C)[..., :T]
    c = F.silu(u).transpose(1, 2)
    a = torch.exp(-p["rate"].flatten() * torch.sigmoid(n @ p["w_g"]))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(n @ p["w_i"]) * c
    h, out = torch.zeros_like(b[:, 0]), []
    for t in range(T):
        h = a[:, t] * h + b[:, t]
        out.append(h)
    return torch.stack(out, 1) @ p["w_o"], total


def test_a_block_trains_and_decodes():
    p = parameters()
    r = torch.Generator().manual_seed(1)
    x, residual, weight = (torch.randn(B, T, C, generator=r) for _ in range(3))
    exact = {n: v.double().requires_grad_() for n, v in p.items()}
    here = {n: v.to(DEV).requires_grad_() for n, v in p.items()}
    out = {}
    for name, q, f in (("exact", exact, plain), ("here", here, block)):
        move = (lambda t: t.double()) if f is plain else (lambda t: t.to(DEV))
        x0, r0 = move(x).requires_grad_(), move(residual).requires_grad_()
        y, total, *_ = f(q, x0, r0)
        ((total + y) * move(weight)).sum().backward()
        out[name] = {"y": y, "total": total, "x": x0.grad, "residual": r0.grad, **{n: v.grad for n, v in q.items()}}
    for n, want in out["exact"].items():
        want, got = want.detach(), out["here"][n].detach().cpu().double()
        assert float((got - want).abs().max()) <= TOL * float(want.abs().max()), n
    # token by token from nothing
    q = {n: v.detach() for n, v in here.items()}
    state, window = torch.zeros(B, H, D, device=DEV), torch.zeros(B, H, W - 1, D, device=DEV)
    for t in range(T):
        y, total = token(q, x[:, t:t + 1].to(DEV), residual[:, t:t + 1].to(DEV), state, window)
        want = out["exact"]["y"][:, t:t + 1].detach()
        assert float((y.cpu().double() - want).abs().max()) <= TOL * float(out["exact"]["y"].detach().abs().max())
    # a long prompt, then tokens: the state goes over
    _, _, state, window = block(q, x[:, :T - 1].to(DEV), residual[:, :T - 1].to(DEV))
    state, window = state.clone(), window.clone()
    again, _ = token(q, x[:, T - 1:].to(DEV), residual[:, T - 1:].to(DEV), state, window)
    assert float((again - y).abs().max()) <= TOL * float(out["exact"]["y"].detach().abs().max())


def test_what_a_step_writes_autograd_knows():
    x, state = torch.rand(1, 2, 6, 16, device=DEV, requires_grad=True), torch.rand(1, 2, 16, device=DEV)
    y = kla.gated_recurrence(x, -torch.rand(1, 2, 6, 16, device=DEV), h0=state)[0]
    y.sum().backward(retain_graph=True)
    tok = torch.rand(1, 2, 16, device=DEV)
    kla.recurrence_step(tok, -tok, None, None, state)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.sum().backward()
    w = torch.rand(16, device=DEV, requires_grad=True)
    z = torch.rand(3, 16, device=DEV)
    out = kla.add_layer_norm(z, w)[0]
    kla.layer_norm(torch.rand(3, 16, device=DEV), y=z)
    with pytest.raises(RuntimeError, match="inplace operation"):
        out.sum().backward()


def test_captured_backward_while_an_eager_graph_of_the_leaves_lives():
    """A training step captured through autograd, on a side stream as torch asks, with fresh leaves."""
    x = torch.randn(2, 2, 100, 16, device=DEV)
    g = -torch.rand(2, 2, 100, 16, device=DEV)
    w = torch.ones(16, device=DEV)

    def step(x, w):
        y = kla.add_layer_norm(kla.gated_recurrence(x, g, scale="sqrt")[0], w)[0]
        return torch.autograd.grad(y.square().sum(), (x, w))

    want = step(x.clone().requires_grad_(), w.clone().requires_grad_())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        leaves = x.clone().requires_grad_(), w.clone().requires_grad_()
        for _ in range(2):
            step(*leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*leaves)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_readme_example_runs():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    block = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "recurrence_forward" in b]
    scope = {}
    exec(compile(block[0], "README.md", "exec"), scope)
    torch.cuda.synchronize()
    assert scope["y"].shape == (2, 8, 1000, 64) and bool(scope["y"].isfinite().all()) and bool(scope["y_t"].isfinite().all())
    assert scope["y"].transpose(1, 2).is_contiguous() and bool(scope["state"].isfinite().all())
