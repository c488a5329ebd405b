"""The delta rule's chunked kernels as real batches run them: so many heads that
the chain takes blocks of 64 columns and that blocks follow one another on an SM
in the other kernels. Beside the bounds on single elements, results are held in
the 2-norm: 2^-20 of the 64-bit values for fp32 outputs and all states (operands
of 24 bits, a few roundings a chunk; the CPU model in test_delta_parts.py shows
that 16 bits anywhere do not pass), and twice that for gradients, which are made
of those and as many products again."""
import numpy as np
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from oracle import delta as O
from test_delta_gpu import DEV, DT, check_backward, check_forward, f64, near, problem, to_dev

pytestmark = pytest.mark.gpu

# B, key heads, heads, T, dk, dv: ragged ends, shared key heads, narrow heads in padded blocks
MANY = [(2, 40, 40, 420, 64, 64), (1, 20, 40, 300, 128, 128), (5, 8, 16, 130, 64, 128), (1, 80, 80, 200, 128, 64),
        (10, 8, 8, 131, 32, 16)]


def wide_blocks(B, H, dv, both):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return B * H * ((dv + 63) // 64 * 2) * (2 if both else 1) > sms


def rel(x, want):
    want = np.asarray(want)
    return float(np.linalg.norm(f64(x) - want) / np.linalg.norm(want))


def lasting(shape, io, seed):
    """Weak decays and strong writes: errors of states and updates stay."""
    p = problem(*shape, io, seed=seed, decay=0.002)
    p["beta"] = (2 * torch.sigmoid(torch.randn(p["beta"].shape, generator=torch.Generator().manual_seed(seed)))).to(DT[io])
    return p


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", MANY)
def test_forward(shape, io):
    assert wide_blocks(shape[0], shape[2], shape[5], False)
    p = problem(*shape, io, seed=sum(shape))
    p["g"][:, :, 70:72] = -float("inf")  # resets inside a chunk
    p["g"][:, :, 128] = -60.0            # and a strong decay where one starts
    check_forward(p, io)
    p["state0"] = None
    check_forward(p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", MANY)
def test_backward(shape, io):
    assert wide_blocks(shape[0], shape[2], shape[5], True)
    p = problem(*shape, io, seed=sum(shape))
    p["g"][:, :, 70:72] = -float("inf")
    p["g"][:, :, 128] = -60.0
    check_backward(p, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_backward_without_states(io):
    p = problem(2, 40, 40, 200, 64, 64, io, seed=2, state=False)
    check_backward(p, io, gs=False)


# the last has few heads and blocks of 32 columns
@pytest.mark.parametrize("shape", [*MANY[:2], (1, 4, 4, 640, 64, 64), (1, 2, 4, 640, 128, 128)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_outputs_and_states_in_the_2_norm(shape, io):
    p = lasting(shape, io, 3)
    d, n = to_dev(p), {x: f64(y) for x, y in p.items()}
    names = ("q", "k", "v", "g", "beta", "state0")
    o, S = kla.delta_forward(*(d[x] for x in names), scale=1.0)
    wo, wS, _ = O.forward(*(n[x] for x in names))
    assert rel(S, wS) <= 2.0 ** -20, rel(S, wS)
    if io == "f32":
        assert rel(o, wo) <= 2.0 ** -20, rel(o, wo)
    near(o, wo, io, shape[4], shape[3], "o")


@pytest.mark.parametrize("shape", [(2, 40, 40, 200, 64, 64), (1, 20, 40, 200, 128, 128), (1, 4, 4, 640, 64, 64)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_in_the_2_norm(shape, io):
    p = problem(*shape, io, seed=6, decay=0.1)
    d, n = to_dev(p), {x: f64(y) for x, y in p.items()}
    names = ("q", "k", "v", "g", "beta", "state0")
    r = torch.Generator().manual_seed(1)
    go, gs = torch.randn(p["v"].shape, generator=r).to(DT[io]), torch.randn(p["state0"].shape, generator=r)
    got = kla.delta_backward(*(d[x] for x in names), go=go.to(DEV), gstateT=gs.to(DEV), scale=1.0)
    want = O.backward(*(n[x] for x in names), f64(go), f64(gs))
    far = {x: rel(got[x], want[x]) for x in got if io == "f32" or x == "gstate0"}
    assert max(far.values()) <= 2.0 ** -19, far


@pytest.mark.parametrize("shape", [(2, 4, 8, 700, 64, 128), (2, 8, 8, 500, 16, 128), (2, 4, 8, 300, 64, 64),
                                   (2, 4, 4, 300, 128, 64), (2, 4, 4, 300, 128, 128)])
def test_gradients_of_wide_values_in_the_2_norm(shape):
    """fp32 gradients that add products over two slices of V's columns, and gk,
    which adds two products. Sums are cut to 24 bits with every instruction, by
    2^-24 at most and always downwards: as long as small products never meet
    large sums that is a few times, less than 2^-21 (24 times and more otherwise:
    9e-7 and 1.2e-6). The decay's gradient sums these again: twice that."""
    p = problem(*shape, "f32", seed=6, decay=0.1)
    d, n = to_dev(p), {x: f64(y) for x, y in p.items()}
    names = ("q", "k", "v", "g", "beta", "state0")
    r = torch.Generator().manual_seed(1)
    go, gs = torch.randn(p["v"].shape, generator=r), torch.randn(p["state0"].shape, generator=r)
    got = kla.delta_backward(*(d[x] for x in names), go=go.to(DEV), gstateT=gs.to(DEV), scale=1.0)
    want = O.backward(*(n[x] for x in names), f64(go), f64(gs))
    far = {x: rel(got[x], want[x]) for x in got}
    assert all(far[x] <= (2.0 ** -20 if x in ("gg", "gbeta") else 2.0 ** -21) for x in far), far
