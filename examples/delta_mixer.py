"""A small model of gated delta rule layers: layer norm with the residual sum,
causal convolution, norm of queries and keys with the position rotation, the delta rule, and an output projection.
It learns to recall which value followed a key earlier in the sequence, then
answers one token at a time from the carried state, and both ways agree.

    python examples/delta_mixer.py
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bayesian_filtering_linear_gb300 import kla  # noqa: E402


class DeltaMixer(torch.nn.Module):
    """Hk key heads serve H value heads; widths per head are dk and dv."""

    def __init__(self, width, Hk=2, H=4, dk=32, dv=32, taps=4):
        super().__init__()
        self.Hk, self.H, self.dk, self.dv, self.taps = Hk, H, dk, dv, taps
        self.qkv = torch.nn.Linear(width, 2 * Hk * dk + H * dv, bias=False)
        self.gates = torch.nn.Linear(width, 2 * H)
        self.out = torch.nn.Linear(H * dv, width, bias=False)
        self.taps_q, self.taps_k, self.taps_v = (torch.nn.Parameter(0.5 * torch.randn(h, d, taps))
                                                 for h, d in ((Hk, dk), (Hk, dk), (H, dv)))
        self.q_weight, self.k_weight = (torch.nn.Parameter(torch.ones(dk)) for _ in range(2))
        self.rate = torch.nn.Parameter(torch.linspace(-6.0, 0.0, H))
        freq, self.rot_scale = kla.rope_frequencies(dk // 2)
        self.register_buffer("freq", freq)

    def forward(self, x, carried=None):
        """x [B,T,width]; `carried`: what the previous tokens left (None at the start). Returns (y, carried)."""
        B, T, _ = x.shape
        parts = self.qkv(x).split([self.Hk * self.dk, self.Hk * self.dk, self.H * self.dv], -1)
        g, b = self.gates(x).transpose(1, 2).chunk(2, 1)
        g, b = (-self.rate.exp()[:, None] * F.softplus(g)).contiguous(), b.sigmoid().contiguous()
        at, windows, state = carried or (0, (None,) * 3, None)
        mixed = []  # a few tokens back by the causal convolution, one stream each
        for part, taps, window in zip(parts, (self.taps_q, self.taps_k, self.taps_v), windows):
            part = part.unflatten(-1, taps.shape[:2]).transpose(1, 2).contiguous()
            mixed.append(kla.causal_conv(part, taps, window=window))
        (q, k, v), windows = zip(*mixed)
        q, k = kla.qk_norm_rope(q, k, self.q_weight, self.k_weight, self.freq, norm="l2", rot_scale=self.rot_scale,
                                offset=at)
        if carried is not None and T == 1 and not torch.is_grad_enabled():
            o = kla.delta_step(*(t.squeeze(2) for t in (q, k, v, g, b)), state).unsqueeze(2)
        else:
            o, state = kla.delta_rule(q, k, v, g, b, state)
        return self.out(o.transpose(1, 2).flatten(2)), (at + T, windows, state)


class Recall(torch.nn.Module):
    def __init__(self, symbols, width=64, layers=2):
        super().__init__()
        self.embed = torch.nn.Embedding(symbols, width)
        self.norms = torch.nn.ModuleList(torch.nn.LayerNorm(width) for _ in range(layers + 1))
        self.mixers = torch.nn.ModuleList(DeltaMixer(width) for _ in range(layers))
        self.head = torch.nn.Linear(width, symbols)

    def norm(self, i, x, y):
        """The norm of x + y (y: what the last layer adds, None before the first), and that sum."""
        n, total = kla.add_layer_norm(x, self.norms[i].weight, self.norms[i].bias, y, eps=self.norms[i].eps)
        return n, x if total is None else total

    def forward(self, tokens, carried=None):
        x, y, left = self.embed(tokens), None, []
        for i, mixer in enumerate(self.mixers):
            n, x = self.norm(i, x, y)
            y, c = mixer(n, None if carried is None else carried[i])
            left.append(c)
        return self.head(self.norm(-1, x, y)[0]), left


def batch(B, pairs, symbols, generator, device):
    """key value key value ... then the keys again, each to be answered with its value."""
    half = symbols // 2
    keys = torch.stack([torch.randperm(half, generator=generator)[:pairs] for _ in range(B)])
    values = half + torch.randint(0, half, (B, pairs), generator=generator)
    order = torch.stack([torch.randperm(pairs, generator=generator) for _ in range(B)])
    told = torch.stack([keys, values], -1).flatten(1)
    return torch.cat([told, keys.gather(1, order)], 1).to(device), values.gather(1, order).to(device)


def main(steps=400, B=64, pairs=12, symbols=64, device="cuda", say=print):
    torch.manual_seed(0)
    r = torch.Generator().manual_seed(1)
    model = Recall(symbols).to(device)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    for step in range(steps):
        tokens, answers = batch(B, pairs, symbols, r, device)
        logits, _ = model(tokens)
        loss = F.cross_entropy(logits[:, 2 * pairs:].flatten(0, 1), answers.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 100 == 0 or step == steps - 1:
            say(f"step {step}: loss {float(loss.detach()):.3f}")
    with torch.no_grad():
        tokens, answers = batch(B, pairs, symbols, r, device)
        whole, _ = model(tokens)
        right = float((whole[:, 2 * pairs:].argmax(-1) == answers).float().mean())
        carried, answers_by_token = None, []
        for t in range(tokens.shape[1]):  # one token at a time from the carried state
            logits, carried = model(tokens[:, t:t + 1], carried)
            answers_by_token.append(logits)
        apart = float((torch.cat(answers_by_token, 1) - whole).abs().max() / whole.abs().max())
    say(f"answers right: {right:.3f}; one token at a time differs by {apart:.2e} of the largest logit")
    return float(loss.detach()), right, apart


if __name__ == "__main__":
    main()
