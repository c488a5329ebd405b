"""Gradients that autograd hands to the operations' backward passes may be contiguous and yet begin anywhere (a slice of
torch.cat's), while the kernels want them on 16 bytes: here with the kernels replaced, so that it runs without a GPU."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

B, H, T, D = 1, 2, 5, 16
X, S, G = torch.ones(B, H, T, D), torch.ones(B, H, D), torch.ones(B, H, T)
W, SS = torch.ones(H, D, 4), torch.ones(B, H, D, D)


def kernels(monkeypatch, name, outs, grads, watched):
    """Replaces the calls `name`; returns what the backward call was given."""
    seen = {}
    forward, backward = name
    monkeypatch.setattr(kla, forward, lambda *a, **k: outs())

    def back(*a, **k):
        seen.update({n: k[n] for n in watched})
        return {n: torch.ones_like(t) for n, t in grads.items()}
    monkeypatch.setattr(kla, backward, back)
    return seen


OPERATIONS = {
    "gated_recurrence": (("recurrence_forward", "recurrence_backward"), lambda: (X * 2, S * 2, S * 2), {"gx": X, "gg": X},
                         ("gy", "ghT"), (X, X)),
    "scan": (("forward", "backward"), lambda: (X * 2, SS * 2, SS * 2),
             {"gq": X, "gk": X, "gv": X, "glam_v": X, "ga": X, "gpbar": X}, ("gy", "glamT", "getaT"), (X,) * 6),
    "causal_conv": (("conv", "conv_backward"), lambda: (X * 2, torch.ones(B, H, 3, D)), {"gx": X, "gweight": W, "gbias": W[..., 0]},
                    ("gy", "gwindow_out"), (X, W)),
    "delta_rule": (("delta_forward", "delta_backward"), lambda: (X * 2, SS * 2),
                   {"gq": X, "gk": X, "gv": X, "gg": G, "gbeta": G}, ("go", "gstateT"), (X, X, X, G, G)),
    "qk_norm_rope": (("norm_rope", "norm_rope_backward"), lambda: (X * 2, X * 2), {"gq": X, "gk": X}, ("gyq", "gyk"), (X, X)),
}


@pytest.mark.parametrize("operation", OPERATIONS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_begin_on_16_bytes(monkeypatch, operation, dtype):
    names, outs, grads, watched, args = OPERATIONS[operation]
    cast = lambda t: t.to(dtype) if t.ndim == 4 and t.shape[-1] == D and t.shape[2] != D else t  # noqa: E731
    seen = kernels(monkeypatch, names, lambda: tuple(cast(t) for t in outs()), {n: cast(t) for n, t in grads.items()}, watched)
    leaves = [cast(t).clone().requires_grad_() for t in args]
    results = getattr(kla, operation)(*leaves)
    first = torch.ones(3, requires_grad=True)
    r = torch.Generator().manual_seed(0)
    weights = [torch.randn(t.numel(), generator=r).to(t.dtype) for t in results]
    loss = 0
    for t, w in zip(results, weights):  # each in a tensor of its own, behind three elements
        loss = loss + (torch.cat([first.to(t.dtype), t.flatten()]) * torch.cat([w.new_ones(3), w])).float().sum()
    loss.backward()
    assert set(seen) == set(watched)
    for (n, g), t, w in zip(((n, seen[n]) for n in watched), results, weights):
        assert g.data_ptr() % 16 == 0 and g.is_contiguous(), n
        assert torch.equal(g, w.view_as(t)), n


def test_gradients_that_begin_well_are_not_copied(monkeypatch):
    names, outs, grads, watched, args = OPERATIONS["gated_recurrence"]
    seen = kernels(monkeypatch, names, outs, grads, watched)
    gy, ghT = torch.randn_like(X), torch.randn_like(S)
    y, hT = kla.gated_recurrence(*(t.clone().requires_grad_() for t in args))
    torch.autograd.backward([y, hT], [gy, ghT])
    assert seen["gy"].data_ptr() == gy.data_ptr() and seen["ghT"].data_ptr() == ghT.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_recurrence_through_a_concatenation(dtype):
    r = torch.Generator(device="cuda").manual_seed(0)
    x, i, gy = (torch.randn(2, 3, 70, 16, generator=r, device="cuda").to(dtype) for _ in range(3))
    g = -torch.rand(2, 3, 70, 16, generator=r, device="cuda").to(dtype)
    ghT = torch.randn(2, 3, 16, generator=r, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x, g, i)]
    y, hT = kla.gated_recurrence(*leaves, scale="sqrt")
    three = torch.ones(3, device="cuda", requires_grad=True)
    behind = lambda t, w: (torch.cat([three.to(t.dtype), t.flatten()]) * torch.cat([w.new_ones(3), w.flatten()])).float().sum()  # noqa: E731
    (behind(y, gy) + behind(hT, ghT)).backward()
    want = kla.recurrence_backward(x, g, i, gy=gy, ghT=ghT, scale="sqrt", state_grad=False)
    assert all(torch.equal(t.grad, want[n]) for t, n in zip(leaves, ("gx", "gg", "gi")))
