"""Refusals of the gated delta rule and of the norm with rotation: every bad
argument is turned down before any CUDA call. Only calls that fail validation
(or have nothing to do) get placeholder pointers."""
import ctypes

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

L = kla.LIB
A, SPACE = 0x100000, 0x10000000           # placeholders, far apart
NAMES = ("q", "k", "v", "g", "beta", "state0", "o", "stateT")
GRADS = ("q", "k", "v", "g", "beta", "state0", "go", "gstateT", "gq", "gk", "gv", "gg", "gbeta", "gstate0")
STEP = ("q", "k", "v", "g", "beta", "state", "o")


def pointers(names, **kw):
    return [ctypes.c_void_p(kw[n]) if n in kw else ctypes.c_void_p(A + SPACE * i) for i, n in enumerate(names)]


def forward(B=1, Hk=1, H=2, T=8, dk=16, dv=16, io=kla.F32, ws=A + 99 * SPACE, ws_bytes=1 << 30, **kw):
    return L.kla_delta_forward(*pointers(NAMES, **kw), B, Hk, H, T, dk, dv, io, 1.0, ctypes.c_void_p(ws), ws_bytes,
                               None)


def backward(B=1, Hk=1, H=2, T=8, dk=16, dv=16, io=kla.F32, ws=A + 99 * SPACE, ws_bytes=1 << 30, **kw):
    return L.kla_delta_backward(*pointers(GRADS, **kw), B, Hk, H, T, dk, dv, io, 1.0, ctypes.c_void_p(ws), ws_bytes,
                                None)


def step(B=1, Hk=1, H=2, dk=16, dv=16, io=kla.F32, **kw):
    return L.kla_delta_step(*pointers(STEP, **kw), B, Hk, H, dk, dv, io, 1.0, None)


@pytest.mark.parametrize("call", [forward, backward, step])
def test_delta_shapes_and_types(call):
    for bad in ({"dk": 24}, {"dv": 256}, {"dk": 0}):
        assert call(**bad) == kla.ERR_UNSUPPORTED_SHAPE
    for bad in ({"B": -1}, {"H": 3, "Hk": 2}, {"Hk": 0}, {"Hk": -1}, {"io": 5}):
        assert call(**bad) == kla.ERR_INVALID_ARG
    assert call(B=0) == kla.OK and call(H=0, Hk=0) == kla.OK


@pytest.mark.parametrize("call,names,free", [(forward, NAMES, {"state0", "stateT"}),
                                             (backward, GRADS, {"state0", "go", "gstateT", "gstate0"}),
                                             (step, STEP, set())])
def test_delta_pointers(call, names, free):
    for n in names:
        if n not in free:
            assert call(**{n: None}) == kla.ERR_INVALID_ARG, n
        off = 2 if n in ("g", "beta", "gg", "gbeta") else 4  # gates: whole elements only
        assert call(**{n: A + SPACE * names.index(n) + off}) == kla.ERR_MISALIGNED, n
    outs = {"o", "stateT", "state"} | {n for n in names if n.startswith("g") and n not in ("g", "go", "gstateT")}
    for n in outs & set(names):  # an output on an input, or on another output
        assert call(**{n: A + SPACE * names.index("k") + 16}) == kla.ERR_INVALID_ARG, n
    with_state = {"stateT": A + SPACE * NAMES.index("state0") + 16} if call is forward else {}
    assert not with_state or call(**with_state) == kla.ERR_INVALID_ARG  # a shifted in-place update


def test_delta_forward_workspace():
    need = L.kla_delta_forward_workspace_size(1, 1, 2, 600, 16, 16)
    assert need > 0 and forward(T=600, ws=None, ws_bytes=0) == kla.ERR_WORKSPACE
    assert forward(T=600, ws_bytes=need - 1) == kla.ERR_WORKSPACE
    assert forward(T=600, ws=A + 16) == kla.ERR_INVALID_ARG  # on q
    assert L.kla_delta_forward_workspace_size(1, 2, 3, 600, 16, 16) == ctypes.c_size_t(-1).value


def test_delta_backward_workspace():
    need = L.kla_delta_backward_workspace_size(1, 1, 2, 8, 16, 16)
    assert 0 < need < 1 << 30
    assert backward(ws=None, ws_bytes=0) == kla.ERR_WORKSPACE
    assert backward(ws_bytes=need - 1) == kla.ERR_WORKSPACE
    assert backward(ws=A + 16) == kla.ERR_INVALID_ARG  # on q
    assert L.kla_delta_backward_workspace_size(1, 2, 3, 8, 16, 16) == ctypes.c_size_t(-1).value
    assert L.kla_delta_backward_workspace_size(1, 1, 1, 0, 16, 16) == 0


def options(norm=1, layout=0, rot=16, eps=1e-6, scale=1.0, offset=0):
    return kla.NormRopeOptions(norm, layout, rot, eps, scale, offset)


NR = ("q", "k", "wq", "wk", "freq", "pos", "yq", "yk")
NRB = ("q", "k", "wq", "wk", "freq", "pos", "gyq", "gyk", "gq", "gk", "gwq", "gwk")


def triple(x):
    return None if x is None else (ctypes.c_longlong * 3)(*x)


def norm_rope(B=1, Hq=2, Hk=1, T=4, D=16, io=kla.F32, opt=None, sq=None, sk=None, **kw):
    return L.kla_norm_rope(*pointers(NR, **kw), B, Hq, Hk, T, D, triple(sq), triple(sk), io,
                           ctypes.byref(opt or options()), None)


def norm_rope_backward(B=1, Hq=2, Hk=1, T=4, D=16, io=kla.F32, opt=None, sq=None, sk=None, gsq=None,
                       ws=A + 99 * SPACE, ws_bytes=1 << 30, **kw):
    return L.kla_norm_rope_backward(*pointers(NRB, **kw), B, Hq, Hk, T, D, triple(sq), triple(sk), triple(gsq), None,
                                    io, ctypes.byref(opt or options()), ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("call", [norm_rope, norm_rope_backward])
def test_norm_rope_shapes_options_and_strides(call):
    for bad in ({"D": 24}, {"D": 256}):
        assert call(**bad) == kla.ERR_UNSUPPORTED_SHAPE
    for o in (options(norm=3), options(layout=2), options(rot=15), options(rot=18), options(rot=-2),
              options(eps=-1.0), options(eps=float("nan"))):
        assert call(opt=o) == kla.ERR_INVALID_ARG
    for bad in ({"B": -1}, {"Hq": -1}, {"io": 2}, {"sq": (64, -16, 16)}):
        assert call(**bad) == kla.ERR_INVALID_ARG
    assert call(sq=(130, 64, 16), B=2) == kla.ERR_MISALIGNED
    assert call(sq=(256, 64, 20), io=kla.BF16) == kla.ERR_MISALIGNED


@pytest.mark.parametrize("call,names", [(norm_rope, NR), (norm_rope_backward, NRB)])
def test_norm_rope_pointers(call, names):
    need = {"q", "k", "freq"} | ({"yq", "yk"} if call is norm_rope else {"gq", "gk"})
    for n in names:
        if n in need:
            assert call(**{n: None}) == kla.ERR_INVALID_ARG, n
        assert call(**{n: A + SPACE * names.index(n) + 8}) == kla.ERR_MISALIGNED, n
    for n in names[6:] if call is norm_rope else names[8:]:
        assert call(**{n: A + SPACE + 16}) == kla.ERR_INVALID_ARG, n  # on k
    if call is norm_rope:  # strides reach further than contiguous rows would
        assert call(sq=(0, 1 << 26, 16), yk=A + (1 << 28) + 64) == kla.ERR_INVALID_ARG


def test_norm_rope_backward_workspace_and_gradient_strides():
    assert norm_rope_backward(ws=None, ws_bytes=0) == kla.ERR_WORKSPACE
    assert norm_rope_backward(gsq=(64, 32, 18)) == kla.ERR_MISALIGNED


def test_binding_refuses_host_tensors_and_unknown_choices():
    x = torch.zeros(1, 1, 4, 16)
    s = torch.zeros(1, 1, 4)
    for f in (lambda: kla.delta_forward(x, x, x, s, s), lambda: kla.norm_rope(x), lambda: kla.norm_rope_backward(x)):
        with pytest.raises(ValueError):
            f()


def test_rope_frequencies():
    plain, one = kla.rope_frequencies(8, 10000.0)
    assert one == 1.0 and torch.allclose(plain, torch.tensor([1.0, 0.1, 0.01, 0.001]))
    assert torch.allclose(kla.rope_frequencies(8, scaling="linear", factor=4)[0], plain / 4)
    ntk = kla.rope_frequencies(8, scaling="ntk", factor=4)[0]
    assert ntk[0] == plain[0] and torch.isclose(ntk[-1], plain[-1] / 4)
    bands, up = kla.rope_frequencies(64, scaling="bands", factor=8, original_length=4096)
    full = kla.rope_frequencies(64)[0]
    turns = 4096 * full / 6.283185307
    assert torch.equal(bands[turns > 40], full[turns > 40]) and torch.allclose(bands[turns < 0.8], full[turns < 0.8] / 8)
    assert bool((bands[:-1] > bands[1:]).all()) and up > 1.2
    for bad in ({"rot_dim": 7}, {"rot_dim": 8, "scaling": "x"}, {"rot_dim": 8, "scaling": "linear", "factor": 0.5},
                {"rot_dim": 8, "scaling": "bands", "factor": 2}):
        with pytest.raises(ValueError):
            kla.rope_frequencies(**bad)


@pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")
def test_valid_calls_without_a_device_report_a_cuda_error():
    assert forward() == kla.ERR_CUDA and step() == kla.ERR_CUDA and backward() == kla.ERR_CUDA
    assert norm_rope() == kla.ERR_CUDA and norm_rope_backward() == kla.ERR_CUDA
