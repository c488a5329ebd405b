"""The layer norm's gradients written over gy or over gtotal, as the C entry allows: the bits of a call with an output of
its own, also where there are more rows than the grid holds at once, so that rows ahead are on their way meanwhile."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# pieces of 16 bytes, pairs, single elements; a warp, some warps and a whole block a row
@pytest.mark.parametrize("D,io,rows", [(64, "bf16", 30000), (1024, "bf16", 6000), (4096, "bf16", 2000), (1024, "f32", 6000),
                                       (446, "bf16", 9000), (2050, "bf16", 2500), (517, "f32", 7000), (517, "bf16", 7000),
                                       (3001, "f32", 1500), (1024, "bf16", 1)])
@pytest.mark.parametrize("onto", ["gy", "gtotal"])
@pytest.mark.parametrize("sums", [True, False])
def test_gradients_in_place(D, io, rows, onto, sums):
    r = torch.Generator(device=DEV).manual_seed(D)
    x, gy, gt = (torch.randn(rows, D, generator=r, device=DEV).to(DT[io]) for _ in range(3))
    w = torch.rand(D, generator=r, device=DEV)
    want = kla.layer_norm_backward(x, w, gy=gy, gtotal=gt, param_grads=sums)
    gw, gb = (torch.empty(D, device=DEV) if sums else None for _ in range(2))
    space = torch.empty(kla.LIB.kla_layer_norm_backward_workspace_size(rows, D), dtype=torch.uint8, device=DEV) if sums else None
    out = gy if onto == "gy" else gt
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = kla.LIB.kla_layer_norm_backward(x.data_ptr(), w.data_ptr(), gy.data_ptr(), gt.data_ptr(), out.data_ptr(), p(gw), p(gb),
                                         rows, D, D, D, D, kla.F32 if io == "f32" else kla.BF16, 1e-5, p(space),
                                         0 if space is None else space.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == kla.OK
    assert torch.equal(out, want["gx"])
    if sums:
        assert torch.equal(gw, want["gweight"]) and torch.equal(gb, want["gbias"])
