"""The gated delta rule at sizes of zero."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_key_heads_without_value_heads_have_zero_gradients(io):
    q = torch.full((2, 3, 5, 32), 7.0, dtype=io, device=DEV)
    v, g = torch.empty(2, 0, 5, 16, dtype=io, device=DEV), torch.empty(2, 0, 5, dtype=io, device=DEV)
    junk = [torch.full_like(q, 5.0) for _ in range(8)]  # what freed memory may hold
    torch.cuda.synchronize()
    del junk
    d = kla.delta_backward(q, q, v, g, g, go=v)
    assert float(d["gq"].abs().max()) == 0 and float(d["gk"].abs().max()) == 0
    o, S = kla.delta_forward(q, q, v, g, g)
    assert o.shape == v.shape and S.shape == (2, 0, 32, 16)
