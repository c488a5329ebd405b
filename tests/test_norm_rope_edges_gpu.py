"""The norm with rotation at its edges: rows that hold no numbers where the answer does not depend on them."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout,rot", [("half", 64), ("half", 6), ("interleaved", 32), ("half", 0)])
@pytest.mark.parametrize("weights", [False, True])
def test_without_a_norm_the_gradient_does_not_depend_on_the_row(io, layout, rot, weights):
    """gx = w ∘ Rᵀ gy, the same bits for any x: infinite, no number, or so large that its product with gy overflows."""
    r = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(2, 3, 37, 64, generator=r, device=DEV).to(io)
    gy = (2 * torch.randn(2, 3, 37, 64, generator=r, device=DEV)).to(io)
    w = 1 + 0.1 * torch.randn(64, generator=r, device=DEV) if weights else None
    f = kla.rope_frequencies(rot, device=DEV)[0] if rot else None
    how = {"norm": "none", "layout": layout}
    want = kla.norm_rope_backward(x, None, w, None, f, gyq=gy, **how)["gq"]
    assert bool(want.isfinite().all())
    bad = x.clone()
    bad[0, 0, 3, 5], bad[0, 1, 9, 63], bad[1, 2, 36, 0] = INF, -INF, NAN
    bad[1, 0, 7] = 3e38
    bad[1, 1, 8, 4:9] = INF
    assert torch.equal(kla.norm_rope_backward(bad, None, w, None, f, gyq=gy, **how)["gq"], want)


@pytest.mark.parametrize("B,T", [(1, 1), (1, 4), (2, 3)])
def test_positions_may_start_at_any_element(B, T):
    """A decode loop's positions[:, t:t + 1]: eight bytes further for each token."""
    q = torch.randn(B, 2, T, 32, device=DEV)
    w = 1 + 0.1 * torch.randn(32, device=DEV)
    f = kla.rope_frequencies(32, device=DEV)[0]
    many = torch.arange(7 * B * T + 1, device=DEV) * 1001
    for start in (1, 2, 3, 7):
        pos = many[start:start + B * T].view(B, T)
        want = kla.norm_rope(q, q, w, w, f, pos.clone())
        assert pos.data_ptr() % 16 == 8 * (start & 1)
        assert all(torch.equal(a, b) for a, b in zip(kla.norm_rope(q, q, w, w, f, pos), want))
        a, b = (kla.norm_rope_backward(q, q, w, w, f, p, gyq=q, gyk=q) for p in (pos, pos.clone()))
        assert all(torch.equal(a[n], b[n]) for n in a)
    x = q.requires_grad_()
    kla.qk_norm_rope(x, None, None, None, f, many[1:1 + B * T].view(B, T))[0].sum().backward()
    assert bool(x.grad.isfinite().all())
