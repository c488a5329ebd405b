"""The norm with rotation as real prompts run it: a block goes through several
heads of its tokens, two rows at a time with the next two on their way, and in
the gradients through several groups of tokens. Heads of q and k differ in
number, are odd, and leave a last part of a group; tokens are not a multiple of
a block's. Against the definition in 64 bits, on the GPU; tolerances as in
test_norm_rope_gpu.py."""
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
THREADS = 256


def geometry(B, Hq, Hk, T, D, io, bwd):
    """Heads that a block takes and groups of work per block, as the launch chooses them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_block = THREADS * (16 // io.itemsize) // D
    groups = -(-B * T // per_block)
    want, heads = sms * 2, max(Hq, Hk)
    s = min(max(-(-want // groups), 1), heads)
    per = -(-heads // s)
    n = groups * -(-heads // per)
    return per, n / (min(n, want) if bwd else n)


def definition(x, w, gy, pos, freq, norm, layout, eps, rot_scale):
    """y, gx and gw, with each pair of entries as a complex number."""
    x, w, gy = x.double(), w.double(), gy.double()
    half, D = len(freq), x.shape[-1]
    turn = rot_scale * torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None, :, None] * freq.double())

    def rotate(z, turn):
        z = z.clone()
        if layout == "half":
            c = torch.complex(z[..., :half], z[..., half:2 * half]) * turn
            z[..., :half], z[..., half:2 * half] = c.real, c.imag
        else:
            c = torch.view_as_complex(z[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
            z[..., :2 * half] = torch.view_as_real(c).flatten(-2)
        return z

    n = {"none": None, "rms": 1 / D, "l2": 1}[norm]
    size = torch.ones_like(x[..., :1]) if n is None else (x.square().sum(-1, keepdim=True) * n + eps).sqrt()
    g = rotate(gy, turn.conj())
    gw = (g * x / size).sum((0, 1, 2))
    gx = g * w / size
    if n is not None:
        gx = gx - x * (g * w * x).sum(-1, keepdim=True) / size ** 3 * n
    return rotate(x / size * w, turn), gx, gw


def near(got, want, io, D, what, terms=0):
    got = got.double()
    top = want.abs().amax(-1, keepdim=True) if terms == 0 else want.abs().max()
    tol = (16 * (D + terms) ** 0.5 + 8 * torch.pi) * 2.0 ** -24 * (1.5 * top + 1e-6 * want.abs().max())
    err = (got - want).abs()
    if io == torch.bfloat16:
        err = err - 2.0 ** -8 * want.abs()
    assert bool((err <= tol + 1e-30).all()), f"{what}: {float((err - tol).max()):.3g} over"


CASES = [  # B, Hq, Hk, T, D, type, norm, layout, rotated
    (2, 7, 3, 4099, 64, torch.bfloat16, "rms", "half", 64), (2, 7, 3, 4099, 64, torch.bfloat16, "l2", "interleaved", 32),
    (2, 5, 2, 2051, 128, torch.float32, "rms", "half", 128), (1, 3, 5, 8191, 16, torch.float32, "l2", "half", 6),
    (3, 1, 9, 3001, 32, torch.bfloat16, "rms", "interleaved", 32), (2, 16, 1, 4099, 128, torch.bfloat16, "none", "half", 24),
    (1, 2, 2, 20011, 64, torch.float32, "rms", "half", 64)]


@pytest.mark.parametrize("heads_last", [True, False])
@pytest.mark.parametrize("B,Hq,Hk,T,D,io,norm,layout,rot", CASES)
def test_many_tokens_and_heads(B, Hq, Hk, T, D, io, norm, layout, rot, heads_last):
    per, _ = geometry(B, Hq, Hk, T, D, io, False)
    per_back, jobs = geometry(B, Hq, Hk, T, D, io, True)
    assert per > 1 and per_back > 1 and jobs > 1  # a block takes several heads, and backward several groups
    r = torch.Generator(device=DEV).manual_seed(T + D)
    randn = lambda *s: torch.randn(*s, generator=r, device=DEV)

    def rows(h):
        return randn(B, T, h, D).to(io).transpose(1, 2) if heads_last else randn(B, h, T, D).to(io)

    q, k, gyq, gyk = rows(Hq), rows(Hk), randn(B, Hq, T, D).to(io), randn(B, Hk, T, D).to(io)
    wq, wk = 1 + 0.3 * randn(D), 1 + 0.3 * randn(D)
    freq = kla.rope_frequencies(rot, device=DEV)[0]
    pos = (torch.randint(0, 1 << 20, (B, 1), generator=r, device=DEV) + torch.arange(T, device=DEV)).contiguous()
    kw = {"norm": norm, "layout": layout, "eps": 1e-6, "rot_scale": 1.25}
    yq, yk = kla.norm_rope(q, k, wq, wk, freq, pos, **kw)
    g = kla.norm_rope_backward(q, k, wq, wk, freq, pos, gyq=gyq, gyk=gyk, **kw)
    for n, x, w, y, gy in (("q", q, wq, yq, gyq), ("k", k, wk, yk, gyk)):
        wy, wx, ww = definition(x, w, gy, pos, freq, norm, layout, 1e-6, 1.25)
        near(y, wy, io, D, "y" + n)
        near(g["g" + n], wx, io, D, "g" + n)
        near(g[f"g{n}_weight"], ww, torch.float32, D, f"g{n}_weight", terms=B * T * x.shape[1])
