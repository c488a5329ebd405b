"""The autograd operations give first derivatives only, and say so. Run on the
CPU with stand-ins for the kernels' calls."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla


def like(names, args):
    return {n: torch.ones_like(x) for n, x in zip(names, args)}


@pytest.fixture(params=["scan", "causal_conv", "delta_rule", "qk_norm_rope"])
def call(request, monkeypatch):
    """A call of the operation on CPU tensors, its kernels replaced."""
    x, w, g = torch.ones(1, 1, 4, 16), torch.ones(16), torch.ones(1, 1, 4)
    S = torch.zeros(1, 1, 16, 16)
    names = {
        "scan": ("forward", "backward", (x,) * 6, lambda *a, **k: (a[0] * 2, S, S),
                 lambda *a, **k: like(("gq", "gk", "gv", "glam_v", "ga", "gpbar"), a)),
        "causal_conv": ("conv", "conv_backward", (x, torch.ones(1, 16, 4)), lambda *a, **k: (a[0] * 2, x),
                        lambda *a, **k: like(("gx", "gweight"), a)),
        "delta_rule": ("delta_forward", "delta_backward", (x, x, x, g, g), lambda *a, **k: (a[2] * 2, S),
                       lambda *a, **k: like(("gq", "gk", "gv", "gg", "gbeta"), a)),
        "qk_norm_rope": ("norm_rope", "norm_rope_backward", (x, x, w, w), lambda *a, **k: (a[0] * 2, a[1] * 2),
                         lambda *a, **k: like(("gq", "gk", "gq_weight", "gk_weight"), a)),
    }
    forward, backward, args, f, b = names[request.param]
    monkeypatch.setattr(kla, forward, f)
    monkeypatch.setattr(kla, backward, b)
    leaves = [a.clone().requires_grad_() for a in args]
    return lambda: (leaves, getattr(kla, request.param)(*leaves)[0])


def test_first_derivatives(call):
    leaves, y = call()
    assert all(torch.equal(g, torch.ones_like(x)) for x, g in zip(leaves, torch.autograd.grad(y.sum(), leaves)))


def test_second_derivatives_raise(call):
    leaves, y = call()
    grads = torch.autograd.grad(y.square().sum(), leaves, create_graph=True)
    again = sum((g * x).sum() for g, x in zip(grads, leaves))
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(again, leaves, retain_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        again.backward()


def test_gradients_under_create_graph_are_the_same(call):
    leaves, y = call()
    for create in (False, True):
        grads = torch.autograd.grad(y.sum(), leaves, retain_graph=True, create_graph=create)
        assert all(torch.equal(g, torch.ones_like(x)) for x, g in zip(leaves, grads))
