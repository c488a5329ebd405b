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
