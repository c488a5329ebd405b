"""NaN and infinities in the recurrence's inputs: a NaN reaches what its channel's formulas let it reach, and nothing
else changes in a bit."""
import itertools

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, H, T, D, AT = 2, 2, 201, 64, 77
HITS = [(0, 0, 0), (0, 1, 5), (1, 1, 63)]  # channels with a NaN at token AT
KINDS = list(itertools.product(["log", "sigmoid", "rate"], ["none", "sqrt", "complement"]))


def make(decay, dtype):
    r = torch.Generator().manual_seed(5)
    x, g, i, gy = (torch.randn(B, H, T, D, generator=r).to(dtype).to(DEV) for _ in range(4))
    rate = torch.rand(H, D, generator=r).to(DEV) + 0.1 if decay == "rate" else None
    return {"x": x, "g": -g.abs() - 0.01 if decay == "log" else g, "i": i, "rate": rate}, gy


def run(a, gy, how):
    h0 = torch.full((B, H, D), 0.5, device=DEV)
    y, hT, kept = kla.recurrence_forward(**a, h0=h0, **how, checkpoints=True)
    d = kla.recurrence_backward(**a, h0=h0, **how, gy=gy, ghT=torch.ones_like(hT), checkpoints=kept)
    return {"y": y, "hT": hT, **d}


def same(got, want, nan, what):
    assert torch.equal(got.isnan(), nan), what
    assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want)), what


@pytest.mark.parametrize("decay,scale", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", ["x", "g", "i"])
def test_nan_reaches_its_channel(decay, scale, dtype, which):
    how = {"decay": decay, "scale": scale}
    a, gy = make(decay, dtype)
    want = run(a, gy, how)
    assert not any(t.isnan().any() for t in want.values())
    a[which] = a[which].clone()
    for b, h, d in HITS:
        a[which][b, h, AT, d] = float("nan")
    got = run(a, gy, how)
    hit = torch.zeros(B, H, D, dtype=torch.bool, device=DEV)
    for place in HITS:
        hit[place] = True
    t = torch.arange(T, device=DEV)[:, None]
    mask = lambda tokens: hit[:, :, None] & tokens  # noqa: E731
    scaled = scale != "none"
    # h is NaN from the token on; G before it where its decay is; dL/dlog a = G (a h_before + s' σ(i) x)
    nan = {"y": mask(t >= AT), "hT": hit, "gh0": hit & (which == "g"), "grate": hit.any(0)}
    if which == "g":
        nan.update(gx=mask((t < AT) | ((t == AT) & scaled)), gg=mask(t >= 0), gi=mask((t < AT) | ((t == AT) & scaled)))
    else:
        nan.update(gx=mask((t == AT) & (which == "i")), gg=mask((t > AT) | ((t == AT) & scaled)), gi=mask(t == AT))
    for n in got:
        same(got[n], want[n], nan[n], n)


@pytest.mark.parametrize("decay,scale", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", ["x", "g", "i"])
def test_nan_in_a_step(decay, scale, dtype, which):
    how = {"decay": decay, "scale": scale}
    a, _ = make(decay, dtype)
    rate = a.pop("rate")
    a = {n: v[:, :, 0].contiguous() for n, v in a.items()}
    state = torch.randn(B, H, D, device=DEV)
    clean = state.clone()
    y = kla.recurrence_step(**a, rate=rate, state=clean, **how)
    hit = torch.zeros(B, H, D, dtype=torch.bool, device=DEV)
    for place in HITS:
        hit[place] = True
    a[which][hit] = float("nan")
    same(kla.recurrence_step(**a, rate=rate, state=state, **how), y, hit, "y")
    same(state, clean, hit, "state")


@pytest.mark.parametrize("scale", ["none", "sqrt", "complement"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_and_nan_rates(scale, dtype):
    """An infinite rate remembers nothing: a = 0 and s = 1, so that y = x, also behind the last token of a tile that
    is not full; a NaN rate leaves its channel NaN in every batch row."""
    how = {"decay": "rate", "scale": scale}
    a, gy = make("rate", dtype)
    a["i"] = None
    want = run(a, gy, how)
    a["rate"] = a["rate"].clone()
    assert (a["rate"] > 0.375).sum(1).min() > 1  # (a block whose rates are all smaller takes another path)
    a["rate"][0, 3], a["rate"][1, 7] = float("inf"), float("nan")
    got = run(a, gy, how)
    # two approximate square roots, 2^-22 each, and half a step of the type
    close = {"rtol": 2.0 ** -21 + (2.0 ** -8 if dtype == torch.bfloat16 else 0), "atol": 0}
    x, gx = a["x"][:, 0, :, 3].float(), gy[:, 0, :, 3].float()
    gx[:, -1] += 1
    torch.testing.assert_close(got["y"][:, 0, :, 3].float(), x, **close)
    torch.testing.assert_close(got["hT"][:, 0, 3], x[:, -1], **close)
    torch.testing.assert_close(got["gx"][:, 0, :, 3].float(), gx, **close)
    assert not got["gg"][:, 0, :, 3].any() and not got["gh0"][:, 0, 3].any()
    # the tokens that fill the last tiles, 64 for each of 16 blocks at most, add 2^-126 G h each, where |G h| < 100
    assert got["grate"][0, 3].abs() <= B * 1024 * 100 * 2.0 ** -126
    for n in ("y", "gg"):
        assert got[n][:, 1, :, 7].isnan().all(), n
    for n in ("hT", "gh0"):
        assert got[n][:, 1, 7].isnan().all(), n
    assert got["grate"][1, 7].isnan()
    rest = torch.ones(H, D, dtype=torch.bool, device=DEV)
    rest[0, 3] = rest[1, 7] = False
    for n, v in got.items():
        keep = rest if n == "grate" else rest[:, None] if v.ndim == 4 else rest
        assert torch.equal(torch.where(keep, v, 0), torch.where(keep, want[n], 0)), n

    state = torch.randn(B, H, D, device=DEV)
    step = {n: a[n][:, :, 0].contiguous() for n in ("x", "g")}
    y = kla.recurrence_step(**step, i=None, rate=a["rate"], state=state, **how)
    torch.testing.assert_close(y[:, 0, 3].float(), step["x"][:, 0, 3].float(), **close)
    assert y[:, 1, 7].isnan().all()
