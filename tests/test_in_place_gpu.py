"""What a call writes in place, autograd knows: a backward pass that had saved it
raises instead of going by the new values."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(*s):
    return torch.rand(*s, device=DEV)


def delta(T=6):
    return [rand(1, 2, T, 16), 0.2 * rand(1, 2, T, 16), rand(1, 2, T, 16), -rand(1, 2, T), rand(1, 2, T)]


def tokens(args):
    return [x[:, :, 0].contiguous() for x in args]


def by_delta_step():
    S = rand(1, 2, 16, 16)
    args = delta()
    args[0].requires_grad_()
    y = kla.delta_rule(*args, S)[0]
    return y, lambda: kla.delta_step(*tokens([x.detach() for x in args]), S)


def by_delta_forward():
    S = rand(1, 2, 16, 16)
    args = delta()
    args[0].requires_grad_()
    y = kla.delta_rule(*args, S)[0]
    return y, lambda: kla.delta_forward(*[x.detach() for x in args], S, stateT=S)


def by_step():
    lam, eta = 1 + rand(1, 2, 16, 16), rand(1, 2, 16, 16)
    args = [rand(1, 2, 6, 16) for _ in range(6)]
    args[0].requires_grad_()
    y = kla.scan(*args, lam, eta)[0]
    return y, lambda: kla.step(*tokens([x.detach() for x in args]), lam, eta)


def by_conv():
    x, w, window = rand(1, 2, 6, 16).requires_grad_(), rand(2, 16, 4), rand(1, 2, 3, 16)
    y = kla.causal_conv(x, w, None, window)[0]
    return y, lambda: kla.conv(x.detach(), w, None, window, update_window=True)


def by_norm_rope():
    q, other = rand(1, 2, 6, 16), rand(1, 2, 6, 16)
    y = kla.qk_norm_rope(q, None, rand(16).requires_grad_())[0]
    return y, lambda: kla.norm_rope(other, yq=q)


@pytest.mark.parametrize("make", [by_delta_step, by_delta_forward, by_step, by_conv, by_norm_rope])
def test_a_saved_tensor_that_a_call_overwrites_makes_the_backward_raise(make):
    y, write = make()
    y.sum().backward(retain_graph=True)
    write()
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.sum().backward()


def test_states_made_for_inference_are_stepped():
    with torch.inference_mode():
        S = rand(1, 2, 16, 16)
        before = S.clone()
        kla.delta_step(*tokens(delta()), S)
        assert not torch.equal(S, before)
