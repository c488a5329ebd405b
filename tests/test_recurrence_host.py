"""Refusals of the gated linear recurrence and of the layer norm: every bad
argument is turned down before any CUDA call. Only calls that fail validation
(or have nothing to do) get placeholder pointers."""
import ctypes

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

L = kla.LIB
A, SPACE = 0x100000, 0x10000000  # placeholders, far apart
FWD = ("x", "g", "i", "rate", "h0", "y", "hT", "kept")
STEP = ("x", "g", "i", "rate", "state", "y")
BWD = ("x", "g", "i", "rate", "h0", "kept", "gy", "ghT", "gx", "gg", "gi", "grate", "gh0")
LN = ("x", "weight", "bias", "residual", "y", "total")
LNB = ("x", "weight", "gy", "gtotal", "gx", "gweight", "gbias")
FAR = A + 99 * SPACE


def at(names, n):
    return A + SPACE * names.index(n)


def pointers(names, **kw):
    return [ctypes.c_void_p(kw[n]) if n in kw else ctypes.c_void_p(at(names, n)) for n in names]


def triple(x):
    return None if x is None else (ctypes.c_longlong * 3)(*x)


def opt(decay=2, scale=1):
    return ctypes.byref(kla.RecurrenceOptions(decay, scale))


def forward(B=1, H=2, T=8, D=16, io=kla.F32, o=None, sx=None, sy=None, **kw):
    return L.kla_recurrence_forward(*pointers(FWD, **kw), B, H, T, D, triple(sx), None, None, triple(sy), io, o or opt(), None)


def step(B=1, H=2, D=16, io=kla.F32, o=None, **kw):
    kw.pop("T", None)
    return L.kla_recurrence_step(*pointers(STEP, **kw), B, H, D, io, o or opt(), None)


def backward(B=1, H=2, T=8, D=16, io=kla.F32, o=None, sx=None, sgx=None, ws=FAR, ws_bytes=1 << 30, **kw):
    return L.kla_recurrence_backward(*pointers(BWD, **kw), B, H, T, D, triple(sx), None, None, None, triple(sgx), None, None,
                                     io, o or opt(), ctypes.c_void_p(ws), ws_bytes, None)


def norm(rows=4, D=16, xs=16, rs=16, io=kla.F32, eps=1e-5, **kw):
    return L.kla_layer_norm(*pointers(LN, **kw), rows, D, xs, rs, io, eps, None)


def norm_backward(rows=4, D=16, xs=16, ys=16, ts=16, io=kla.F32, eps=1e-5, ws=FAR, ws_bytes=1 << 30, **kw):
    return L.kla_layer_norm_backward(*pointers(LNB, **kw), rows, D, xs, ys, ts, io, eps, ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("call", [forward, step, backward])
def test_recurrence_shapes_types_and_options(call):
    for bad in ({"D": 12}, {"D": 4}, {"D": 0}, {"B": 1 << 16, "H": 1 << 15}, {"B": 1 << 16, "H": 1 << 10, "D": 64}):
        assert call(**bad) == kla.ERR_UNSUPPORTED_SHAPE, bad
    for bad in ({"B": -1}, {"H": -1}, {"io": 2}, {"o": opt(3)}, {"o": opt(-1)}, {"o": opt(0, 3)}, {"o": opt(0, -1)}):
        assert call(**bad) == kla.ERR_INVALID_ARG, bad
    assert call(B=0, rate=None, **({"grate": None} if call is backward else {})) == kla.OK


def test_recurrence_lengths():
    assert forward(T=-1) == kla.ERR_INVALID_ARG and backward(T=-1) == kla.ERR_INVALID_ARG
    assert forward(T=1 << 30, B=1 << 10, D=128) == kla.ERR_UNSUPPORTED_SHAPE
    assert L.kla_recurrence_checkpoints_size(2, 3, 65, 16) == 2 * 2 * 3 * 16 * 4
    assert L.kla_recurrence_checkpoints_size(2, 3, 64, 12) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("call,names,free,outs", [
    (forward, FWD, {"i", "h0", "hT", "kept"}, {"y", "hT", "kept"}), (step, STEP, {"i"}, {"y", "state"}),
    (backward, BWD, {"i", "h0", "kept", "gy", "ghT", "grate", "gh0"}, {"gx", "gg", "gi", "grate", "gh0"})])
def test_recurrence_pointers(call, names, free, outs):
    for n in names:
        if n not in free:
            assert call(**{n: None}) == kla.ERR_INVALID_ARG, n
        assert call(**{n: at(names, n) + 8}) == kla.ERR_MISALIGNED, n
    for n in outs:  # an output on an input, or on another output
        assert call(**{n: at(names, "g") + 16}) == kla.ERR_INVALID_ARG, n
    if call is forward:
        assert call(hT=at(names, "h0") + 16) == kla.ERR_INVALID_ARG  # a shifted in-place update
        assert call(sx=(0, 1 << 26, 16), y=A + (1 << 28) + 64) == kla.ERR_INVALID_ARG  # strides reach further
    if call is backward:
        assert call(gg=at(names, "gx")) == kla.ERR_INVALID_ARG and call(gi=at(names, "gg")) == kla.ERR_INVALID_ARG
        assert call(gh0=at(names, "grate")) == kla.ERR_INVALID_ARG


def test_recurrence_strides():
    for call in (forward, backward):
        assert call(sx=(256, -16, 16)) == kla.ERR_INVALID_ARG
        assert call(sx=(256, 130, 16)) == kla.ERR_MISALIGNED
        assert call(sx=(256, 128, 20), io=kla.BF16) == kla.ERR_MISALIGNED
    assert forward(sy=(256, 128, 8)) == kla.ERR_INVALID_ARG      # rows of an output on each other
    assert backward(sgx=(256, 0, 16)) == kla.ERR_INVALID_ARG
    assert backward(T=1, H=1, sgx=(3, 5, 7), gy=at(BWD, "gy") + 4) == kla.ERR_MISALIGNED  # (unused strides are not read)


def test_recurrence_workspace():
    need = L.kla_recurrence_backward_workspace_size(1, 2, 200, 16, 0)
    less = L.kla_recurrence_backward_workspace_size(1, 2, 200, 16, 1)
    assert need == less + 4 * 2 * 16 * 4 and less == 4 * 2 * 16 * 4
    assert backward(T=200, kept=None, ws=None, ws_bytes=0) == kla.ERR_WORKSPACE
    assert backward(T=200, kept=None, ws_bytes=need - 1) == kla.ERR_WORKSPACE
    assert backward(T=200, ws_bytes=less - 1) == kla.ERR_WORKSPACE
    assert backward(T=200, ws=A + 16) == kla.ERR_INVALID_ARG  # on x


def test_layer_norm_refusals():
    for call in (norm, norm_backward):
        for bad in ({"D": 0}, {"D": 8193}, {"rows": 1 << 31}):
            assert call(**bad) == kla.ERR_UNSUPPORTED_SHAPE, bad
        for bad in ({"rows": -1}, {"io": 2}, {"eps": -1.0}, {"eps": float("nan")}, {"xs": -16}):
            assert call(**bad) == kla.ERR_INVALID_ARG, bad
    for n in ("x", "y", "total"):
        assert norm(**{n: None}) == kla.ERR_INVALID_ARG
    for n in LN:
        assert norm(**{n: at(LN, n) + 2}) == kla.ERR_MISALIGNED
    for n in ("weight", "bias"):
        assert norm(**{n: at(LN, n) + 8}) == kla.ERR_MISALIGNED
    for n in ("y", "total"):
        assert norm(**{n: A + 16}) == kla.ERR_INVALID_ARG                 # a shifted in-place call
        assert norm(**{n: at(LN, "weight")}) == kla.ERR_INVALID_ARG
        assert norm(xs=32, **{n: A}) == kla.ERR_INVALID_ARG               # in place on rows with gaps
    assert norm(y=at(LN, "total")) == kla.ERR_INVALID_ARG
    for n in ("x", "gx"):
        assert norm_backward(**{n: None}) == kla.ERR_INVALID_ARG
    for n in LNB:
        assert norm_backward(**{n: at(LNB, n) + 2}) == kla.ERR_MISALIGNED
    for n in ("gx", "gweight", "gbias"):
        assert norm_backward(**{n: A + 16}) == kla.ERR_INVALID_ARG
    assert norm_backward(gx=A) == kla.ERR_INVALID_ARG                     # gx may be gy or gtotal, not x
    assert norm_backward(gweight=at(LNB, "gx")) == kla.ERR_INVALID_ARG
    assert norm_backward(ws=None, ws_bytes=0) == kla.ERR_WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")
def test_valid_calls_without_a_device_report_a_cuda_error():
    assert forward() == kla.ERR_CUDA and step() == kla.ERR_CUDA and backward() == kla.ERR_CUDA
    assert norm() == kla.ERR_CUDA and norm_backward() == kla.ERR_CUDA
    assert norm(y=A) == kla.ERR_CUDA and norm(total=A, y=at(LN, "residual")) == kla.ERR_CUDA  # in place: nothing to refuse
    assert forward(hT=at(FWD, "h0")) == kla.ERR_CUDA


def test_binding_refuses_host_tensors_and_unknown_choices():
    x = torch.zeros(1, 1, 4, 16)
    for f in (lambda: kla.recurrence_forward(x, x), lambda: kla.recurrence_backward(x, x), lambda: kla.layer_norm(x),
              lambda: kla.recurrence_step(x[0], x[0], None, None, x[0]), lambda: kla.layer_norm_backward(x, gy=x),
              lambda: kla.recurrence_forward(x, x, decay="power")):
        with pytest.raises(ValueError):
            f()


@pytest.fixture(params=["gated_recurrence", "add_layer_norm"])
def call(request, monkeypatch):
    """A call of the operation on CPU tensors, its kernels replaced."""
    x, w, s = torch.ones(1, 1, 4, 16), torch.ones(16), torch.zeros(1, 1, 16)
    if request.param == "gated_recurrence":
        monkeypatch.setattr(kla, "recurrence_forward", lambda *a, **k: (a[0] * 2, s, s))
        monkeypatch.setattr(kla, "recurrence_backward", lambda *a, **k: {"gx": torch.ones_like(x), "gg": torch.ones_like(x)})
        args = (x, x)
    else:
        monkeypatch.setattr(kla, "layer_norm", lambda *a, **k: (a[0] * 2, a[0] + a[3]))
        monkeypatch.setattr(kla, "layer_norm_backward", lambda *a, **k: {"gx": torch.ones_like(x), "gweight": torch.ones_like(w),
                                                                         "gbias": torch.ones_like(w)})
        args = (x, w, w, x)
    leaves = [a.clone().requires_grad_() for a in args]
    return lambda: (leaves, getattr(kla, request.param)(*leaves)[0])


def test_first_derivatives_only(call):
    leaves, y = call()
    for create in (False, True):
        grads = torch.autograd.grad(y.sum(), leaves, retain_graph=True, create_graph=create)
        assert all(torch.equal(g, torch.ones_like(x)) for x, g in zip(leaves, grads))
    with pytest.raises(RuntimeError, match="second derivatives"):
        sum((g * x).sum() for g, x in zip(grads, leaves)).backward()
