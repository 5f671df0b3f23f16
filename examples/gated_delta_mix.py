"""A time-mix layer whose state is a matrix per head: token shift, projections, the gated delta
rule, then each head's norm with a gate -- trained for a few steps on a recall task, then run as a
language model would be served: a ragged batch of prompts in one call, and token by token from the
states that call left.

    python examples/gated_delta_mix.py

The library's calls are the recurrence, the norm and the shift, forward and backward; the
projections and the optimizer are torch's.
"""

from __future__ import annotations

import functools
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_recurrence_rnn_amd as L  # noqa: E402


def first_derivative(backward):
    """Refuses a backward that is to be differentiated itself (create_graph): the calls in it leave no
    graph, so every second derivative through them would silently be zero."""

    @functools.wraps(backward)
    def checked(ctx, *grads):
        if torch.is_grad_enabled():
            raise RuntimeError("this function has no second derivative")
        return backward(ctx, *grads)

    return checked


class GatedDelta(torch.autograd.Function):
    """(o, state_out) of the gated delta rule; the backward starts from the forward's checkpoint."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, lengths):
        o, s, ckpt = L.gated_delta_forward_ckpt(q, k, v, g, beta, state=state, lengths=lengths)
        ctx.save_for_backward(q, k, v, g, beta, state, lengths, ckpt)
        return o, s

    @staticmethod
    @first_derivative
    def backward(ctx, go, gs):
        q, k, v, g, beta, state, lengths, ckpt = ctx.saved_tensors
        gs = None if gs is None else gs.contiguous()
        return L.gated_delta_backward(q, k, v, g, beta, go.contiguous(), state=state, gstate=gs, lengths=lengths,
                                      ckpt=ckpt) + (None,)


class HeadNorm(torch.autograd.Function):
    """Each head of o normalised, times silu(gate)."""

    @staticmethod
    def forward(ctx, o, heads, weight, bias, gate):
        ctx.heads = heads
        ctx.save_for_backward(o, weight, bias, gate)
        return L.group_norm_act(o, heads, weight, bias, gate=gate)

    @staticmethod
    @first_derivative
    def backward(ctx, gy):
        o, weight, bias, gate = ctx.saved_tensors
        gx, gw, gb, gg = L.group_norm_act_backward(o, ctx.heads, weight, bias, gy.contiguous(), gate=gate)
        return gx, None, gw, gb, gg


class TokenShift(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, mu, x_prev):
        ctx.save_for_backward(x, mu, x_prev)
        return L.token_shift(x, mu, x_prev)

    @staticmethod
    @first_derivative
    def backward(ctx, g):
        x, mu, x_prev = ctx.saved_tensors
        return L.token_shift_backward(x, mu, g.contiguous(), x_prev)[:2] + (None,)


class GatedDeltaMix(torch.nn.Module):
    """C channels in ``heads`` heads; ``dtype`` is the recurrence's and the norm's type."""

    def __init__(self, C, heads, dtype=torch.bfloat16):
        super().__init__()
        self.C, self.H, self.D, self.dtype = C, heads, C // heads, dtype
        # Mixes of a token with the one before it, for q, for k, for v and the gates: at first q and
        # v see the token, k the one before, so that what a token says is stored under its
        # predecessor; q and k start from one projection.
        self.mu = torch.nn.Parameter(torch.tensor([1.0, 0.0, 1.0])[:, None].repeat(1, C))
        self.q, self.k, self.v = (torch.nn.Linear(C, C, bias=False) for _ in range(3))
        self.k.load_state_dict(self.q.state_dict())
        self.gates = torch.nn.Linear(C, C + 2 * heads)
        self.rate = torch.nn.Parameter(torch.linspace(-5.0, -1.0, heads))  # log decay rates
        self.weight, self.bias = torch.nn.Parameter(torch.ones(C)), torch.nn.Parameter(torch.zeros(C))
        self.out = torch.nn.Linear(C, C, bias=False)

    def inputs(self, x, x_prev):
        """q, k, v, g, beta of the recurrence and the norm's gate, from x (B,T,C)."""
        B, T, C = x.shape
        mixed = TokenShift.apply(x, self.mu, x_prev)
        q, k, v = (f(m).view(B, T, self.H, self.D) for f, m in zip((self.q, self.k, self.v), mixed))
        z, a, b = self.gates(mixed[2]).split([C, self.H, self.H], dim=-1)
        unit = [F.normalize(F.silu(t), dim=-1) for t in (q, k)]
        g = -torch.exp(self.rate) * F.softplus(a)
        return [t.to(self.dtype).contiguous() for t in (*unit, v, g, torch.sigmoid(b), z)]

    def forward(self, x, x_prev=None, state=None, lengths=None):
        """(y, state_out) for x (B,T,C) float32."""
        *rec, z = self.inputs(x, x_prev)
        o, s = GatedDelta.apply(*rec, state, lengths)
        y = HeadNorm.apply(o.view(x.shape), self.H, self.weight, self.bias, z)
        return self.out(y.float()), s

    @torch.no_grad()
    def step(self, x, x_prev, state):
        """One token: x (B,C), the token before it, and the state, updated in place."""
        *rec, z = self.inputs(x[:, None], x_prev)
        o = L.gated_delta_decode_step(*(t[:, 0].contiguous() for t in rec), state)
        y = L.group_norm_act(o.view(x.shape), self.H, self.weight, self.bias, gate=z[:, 0].contiguous())
        return self.out(y.float())


def recall_batch(gen, B, pairs, vocab):
    """Rows of ``pairs`` (key, value) tokens, then one of the keys; the target is its value."""
    dev = gen.device
    keys = torch.rand(B, vocab, generator=gen, device=dev).argsort(dim=1)[:, :pairs]
    vals = torch.randint(vocab, (B, pairs), generator=gen, device=dev)
    pick = torch.randint(pairs, (B, 1), generator=gen, device=dev)
    seq = torch.stack([keys, vals + vocab], dim=2).view(B, 2 * pairs)
    return torch.cat([seq, keys.gather(1, pick)], 1), vals.gather(1, pick)[:, 0]


class RecallModel(torch.nn.Module):
    def __init__(self, vocab, C=128, heads=4, dtype=torch.bfloat16):
        super().__init__()
        self.embed = torch.nn.Embedding(2 * vocab, C)
        self.mix = GatedDeltaMix(C, heads, dtype)
        self.head = torch.nn.Linear(C, vocab)

    def forward(self, tokens):
        x = F.rms_norm(self.embed(tokens), (self.mix.C,))
        return self.head(self.mix(x)[0][:, -1])


def train(steps=150, B=64, pairs=20, vocab=32, dtype=torch.bfloat16, seed=0):
    """Losses of ``steps`` training steps on the recall task, and the model."""
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    model = RecallModel(vocab, dtype=dtype).to(dev)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        tokens, target = recall_batch(gen, B, pairs, vocab)
        loss = F.cross_entropy(model(tokens), target)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses, model


@torch.no_grad()
def serve(mix, lengths=(70, 1, 33), more=5, seed=1):
    """Prompts of unlike lengths in one call, then ``more`` tokens one by one; returns the largest
    difference (relative to the outputs' RMS) from running each whole row at once."""
    dev = mix.q.weight.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, T = len(lengths), max(lengths)
    x = torch.randn(B, T + more, mix.C, generator=gen, device=dev)
    lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
    _, state = mix(x[:, :T].contiguous(), lengths=lens)
    rows = torch.arange(B, device=dev)
    worst = 0.0
    whole = [mix(x[b:b + 1, :n + more].contiguous())[0][0] for b, n in enumerate(lengths)]
    for i in range(more):
        at = lens.long() + i
        prev = x[rows, at - 1] * (at > 0)[:, None]  # an empty prompt's first token has none before it
        y = mix.step(x[rows, at].contiguous(), prev, state)
        for b, n in enumerate(lengths):
            ref = whole[b][n + i]
            worst = max(worst, ((y[b] - ref).abs().max() / ref.square().mean().sqrt()).item())
    return worst


def main():
    losses, model = train()
    print("recall loss (%.2f by guessing): first 10 steps %.3f, last 10 steps %.3f" 
          % (math.log(32), sum(losses[:10]) / 10, sum(losses[-10:]) / 10))
    print("decoding against whole rows: largest difference %.2e of the RMS" % serve(model.mix))


if __name__ == "__main__":
    main()
