"""A stack of selective state space layers: the residual's addition with the root-mean-square norm, a
short causal convolution, the selective scan with its gate, and projections -- trained for a few steps on
a copying task, then run as a language model would be served: a ragged batch of prompts in one call, and
token by token from the states that call left.

    python examples/selective_mix.py

The library's calls are the norm, the convolution and the scan, forward and backward; the
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


class NormAdd(torch.autograd.Function):
    """(y, s): s = x + residual and its norm y."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, s = L.rms_norm_add(x, weight, residual=residual)
        ctx.save_for_backward(s, weight)
        return y, s

    @staticmethod
    @first_derivative
    def backward(ctx, gy, gs):
        s, weight = ctx.saved_tensors
        gx, gr, gw = L.rms_norm_add_backward(s, weight, gy.contiguous(), gsum=gs.contiguous())
        return gx, gr, gw


class ShortConv(torch.autograd.Function):
    """(y, state_out) of the convolution from no earlier inputs."""

    @staticmethod
    def forward(ctx, x, weight, bias, lengths):
        y, s = L.short_conv_act(x, weight, bias=bias, lengths=lengths)
        ctx.save_for_backward(x, weight, bias, lengths)
        ctx.mark_non_differentiable(s)
        return y, s

    @staticmethod
    @first_derivative
    def backward(ctx, gy, _):
        x, weight, bias, lengths = ctx.saved_tensors
        return L.short_conv_act_backward(x, weight, gy.contiguous(), bias=bias, lengths=lengths)[:3] + (None,)


class Scan(torch.autograd.Function):
    """(y, state_out) of the scan from a zero state; the backward starts from the forward's checkpoint."""

    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, z, dt_bias, lengths):
        y, s, ckpt = L.scan_selective_ckpt(u, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, lengths=lengths)
        ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, lengths, ckpt)
        ctx.mark_non_differentiable(s)
        return y, s

    @staticmethod
    @first_derivative
    def backward(ctx, gy, _):
        u, dt, A, B, C, D, z, dt_bias, lengths, ckpt = ctx.saved_tensors
        return L.scan_selective_backward(u, dt, A, B, C, gy.contiguous(), D=D, z=z, dt_bias=dt_bias, lengths=lengths,
                                         ckpt=ckpt)[:8] + (None,)


class SelectiveMix(torch.nn.Module):
    """C channels, widened ``expand`` times inside; N states a channel; ``dtype`` is the type of the
    library's operators, the residual stream is float32."""

    def __init__(self, C, expand=2, N=16, taps=4, rank=None, dtype=torch.bfloat16):
        super().__init__()
        E, rank = expand * C, rank or max(1, C // 16)
        self.C, self.E, self.N, self.K, self.rank, self.dtype = C, E, N, taps, rank, dtype
        self.norm = torch.nn.Parameter(torch.ones(C))
        self.into, self.gate = torch.nn.Linear(C, E, bias=False), torch.nn.Linear(C, E, bias=False)
        self.conv = torch.nn.Parameter((2 * torch.rand(E, taps) - 1) * taps ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(E))
        self.maps = torch.nn.Linear(E, rank + 2 * N, bias=False)  # the step's low-rank part, B and C
        self.step_out = torch.nn.Linear(rank, E, bias=False)
        step = torch.exp(torch.empty(E).uniform_(math.log(1e-3), math.log(1e-1)))
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.logA = torch.nn.Parameter(torch.log(torch.arange(1, N + 1, dtype=torch.float32)).repeat(E, 1))
        self.D = torch.nn.Parameter(torch.ones(E))
        self.out = torch.nn.Linear(E, C, bias=False)

    def _inputs(self, u):
        """dt, A, B, C of the scan from the convolution's output u (..., E)."""
        low, B, C = self.maps(u.float()).split([self.rank, self.N, self.N], dim=-1)
        dt = self.step_out(low)
        B, C = (t.to(self.dtype).unsqueeze(-2).contiguous() for t in (B, C))
        return dt.to(self.dtype).contiguous(), -torch.exp(self.logA), B, C

    def forward(self, x, residual, lengths=None):
        """(y, residual, states) for x (B,T,C) in the operators' type and the residual (B,T,C) float32;
        states are the convolution's and the scan's."""
        n, residual = NormAdd.apply(x, residual, self.norm)
        n = n.float()
        u, tail = ShortConv.apply(self.into(n).to(self.dtype), self.conv, self.conv_bias, lengths)
        dt, A, B, C = self._inputs(u)
        y, state = Scan.apply(u, dt, A, B, C, self.D, self.gate(n).to(self.dtype), self.dt_bias, lengths)
        return self.out(y.float()).to(self.dtype), residual, (tail, state)

    @torch.no_grad()
    def step(self, x, residual, states):
        """One token: x, residual (B,C); the states are updated in place."""
        n, residual = L.rms_norm_add(x, self.norm, residual=residual)
        n = n.float()
        u = L.short_conv_decode_step(self.into(n).to(self.dtype), self.conv, states[0], bias=self.conv_bias)
        dt, A, B, C = self._inputs(u)
        y = L.scan_selective_decode_step(u, dt, A, B, C, states[1], D=self.D, z=self.gate(n).to(self.dtype),
                                         dt_bias=self.dt_bias)
        return self.out(y.float()).to(self.dtype), residual


class CopyModel(torch.nn.Module):
    def __init__(self, vocab, C=64, layers=2, dtype=torch.bfloat16):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, C)
        self.layers = torch.nn.ModuleList(SelectiveMix(C, dtype=dtype) for _ in range(layers))
        self.norm = torch.nn.Parameter(torch.ones(C))
        self.head = torch.nn.Linear(C, vocab)

    def forward(self, tokens, lengths=None):
        """(logits, states of the layers) for tokens (B,T)."""
        residual = self.embed(tokens)
        x, states = torch.zeros_like(residual).to(self.layers[0].dtype), []
        for layer in self.layers:
            x, residual, s = layer(x, residual, lengths)
            states.append(s)
        return self.head(NormAdd.apply(x, residual, self.norm)[0].float()), states

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits behind one more token (B,) of each row."""
        residual = self.embed(tokens)
        x = torch.zeros_like(residual).to(self.layers[0].dtype)
        for layer, s in zip(self.layers, states):
            x, residual = layer.step(x, residual, s)
        return self.head(L.rms_norm_add(x, self.norm, residual=residual)[0].float())


def copy_batch(gen, B, items, blanks, vocab):
    """``items`` tokens among blanks (token 0), then as many markers (token 1): the items, in order."""
    dev = gen.device
    what = torch.randint(2, vocab, (B, items), generator=gen, device=dev)
    where = torch.rand(B, items + blanks, generator=gen, device=dev).argsort(dim=1)[:, :items].sort(dim=1)[0]
    seq = torch.zeros(B, items + blanks, dtype=torch.long, device=dev).scatter_(1, where, what)
    return torch.cat([seq, torch.ones(B, items, dtype=torch.long, device=dev)], 1), what


def train(steps=300, B=64, items=4, blanks=28, vocab=10, dtype=torch.bfloat16, seed=0):
    """Losses of ``steps`` training steps on the copying task, and the model."""
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    model = CopyModel(vocab, dtype=dtype).to(dev)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        tokens, target = copy_batch(gen, B, items, blanks, vocab)
        logits = model(tokens)[0][:, -items:]
        loss = F.cross_entropy(logits.flatten(0, 1), target.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses, model


@torch.no_grad()
def serve(model, lengths=(70, 1, 0, 33), more=5, seed=1):
    """Prompts of unlike lengths in one call, then ``more`` tokens one by one; returns the largest
    difference (relative to the logits' RMS) from running each whole row at once."""
    dev = model.head.weight.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, T = len(lengths), max(lengths)
    tokens = torch.randint(model.embed.num_embeddings, (B, T + more), generator=gen, device=dev)
    lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
    _, states = model(tokens[:, :T], lens)
    whole = [model(tokens[b:b + 1, :n + more])[0][0] for b, n in enumerate(lengths)]
    rows = torch.arange(B, device=dev)
    worst = 0.0
    for i in range(more):
        logits = model.step(tokens[rows, lens.long() + i], states)
        for b, n in enumerate(lengths):
            ref = whole[b][n + i]
            worst = max(worst, ((logits[b] - ref).abs().max() / ref.square().mean().sqrt()).item())
    return worst


def main():
    losses, model = train()
    print("copying loss (%.2f by guessing): first 10 steps %.3f, last 10 steps %.3f"
          % (math.log(8), sum(losses[:10]) / 10, sum(losses[-10:]) / 10))
    print("decoding against whole rows: largest difference %.2e of the RMS" % serve(model))


if __name__ == "__main__":
    main()
