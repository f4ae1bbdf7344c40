"""A state space layer made of the package's operators: a few steps of training
on packed documents, then prompts and single tokens from carried states.

    python3 examples/ssm_layer.py [--dim 1024] [--states 16] [--groups 1]
                                  [--tokens 4096] [--steps 10] [--answer 16]

The layer: a projection to the scan's gate, its inputs (x, B, C) and its step
sizes; the causal convolution with SiLU over (x, B, C); the selective scan; the
group norm with its gate; a projection back.  The projections are PyTorch's.
A prompt of several documents and the tokens that follow it one at a time go
through the same weights, with the last inputs of the convolution and the
states of the scan carried in two caches; the example checks that they answer
as the whole sequences at once do.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
from torch import nn
from torch.nn import functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import varlen_depthwise_causal_amd as vdc  # noqa: E402
from varlen_depthwise_causal_amd import autograd as vga  # noqa: E402


class SsmLayer(nn.Module):
    """width channels in the model, 2 * width in the scan (a multiple of 8)."""

    def __init__(self, width, states=16, groups=1, norm_groups=8, device=None):
        super().__init__()
        inner = 2 * width
        self.sizes = (inner, inner + 2 * groups * states, inner)  # gate | x, B, C | step sizes
        self.inner, self.states, self.groups, self.norm_groups = inner, states, groups, norm_groups
        bf16 = {"dtype": torch.bfloat16, "device": device}
        self.proj_in = nn.Linear(width, sum(self.sizes), bias=False, **bf16)
        self.proj_out = nn.Linear(inner, width, bias=False, **bf16)
        channels = self.sizes[1]
        self.conv_weight = nn.Parameter(torch.empty(channels, 4, device=device).uniform_(-0.5, 0.5))
        self.conv_bias = nn.Parameter(torch.zeros(channels, device=device))
        # decay rates 1 ... states of each channel, step sizes from 0.001 to 0.1
        self.A_log = nn.Parameter(torch.arange(1.0, states + 1, device=device).log().repeat(inner, 1))
        self.D = nn.Parameter(torch.ones(inner, device=device))
        step = torch.exp(torch.empty(inner, device=device).uniform_(math.log(1e-3), math.log(0.1)))
        self.dt_bias = nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.norm_weight = nn.Parameter(torch.ones(inner, device=device))

    def _split(self, u):
        return self.proj_in(u).split(self.sizes, dim=-1)

    def _scan_inputs(self, xbc):
        n = self.groups * self.states
        x, B, C = xbc.split((self.inner, n, n), dim=-1)
        shape = (self.groups, self.states)
        return x, B.unflatten(-1, shape), C.unflatten(-1, shape)

    def forward(self, u, cu_seqlens):
        """Packed documents u [S, width], each from a zero state; differentiable."""
        z, xbc, dt = self._split(u)
        xbc = vga.causal_conv1d_silu(xbc.contiguous(), self.conv_weight, cu_seqlens, self.conv_bias)
        x, B, C = self._scan_inputs(xbc)
        y = vga.selective_scan(x, dt, -self.A_log.exp(), B, C, cu_seqlens, D=self.D, dt_bias=self.dt_bias)
        return self.proj_out(vga.group_norm_silu(y, self.norm_weight, self.norm_groups, z=z))

    def caches(self, slots):
        """The carried states of that many sequences."""
        device = self.D.device
        return (torch.zeros(slots, 3, self.sizes[1], dtype=torch.bfloat16, device=device),
                torch.zeros(slots, self.inner, self.states, device=device))

    @torch.no_grad()
    def prefill(self, u, cu_seqlens, caches, slots, resume=None):
        """Packed prompts; document i leaves its states in slot slots[i], and
        goes on from them where resume[i]."""
        z, xbc, dt = self._split(u)
        conv, state = caches
        xbc = vdc.conv1d_prefill(xbc.contiguous(), self.conv_weight, cu_seqlens, conv, bias=self.conv_bias,
                                 state_index=slots, resume=resume)
        x, B, C = self._scan_inputs(xbc)
        y = vdc.selective_scan_fwd(x, dt, -self.A_log.exp(), B, C, cu_seqlens, D=self.D, dt_bias=self.dt_bias,
                                   state=state, state_index=slots, resume=resume)
        return self.proj_out(vdc.group_norm_silu_fwd(y, self.norm_weight, self.norm_groups, z=z))

    @torch.no_grad()
    def step(self, u, caches, slots):
        """One token of each sequence, u [rows, width]; row i has slot slots[i]."""
        z, xbc, dt = self._split(u)
        conv, state = caches
        xbc = vdc.conv1d_update(xbc, conv, self.conv_weight, bias=self.conv_bias, state_index=slots)
        x, B, C = self._scan_inputs(xbc)
        y = vdc.selective_update(x, dt, -self.A_log.exp(), B, C, state, D=self.D, dt_bias=self.dt_bias,
                                 state_index=slots)
        return self.proj_out(vdc.group_norm_silu_fwd(y, self.norm_weight, self.norm_groups, z=z))


def _edges(lengths, device):
    return torch.tensor([0] + lengths, device=device).cumsum(0).to(torch.int32)


def train(layer, width, lengths, steps, device):
    """Plain gradient descent towards targets that depend on earlier tokens;
    returns the losses."""
    cu = _edges(lengths, device)
    u = torch.randn(sum(lengths), width, device=device).bfloat16()
    target = torch.zeros_like(u, dtype=torch.float32)
    for lo, hi in zip(cu.tolist(), cu.tolist()[1:]):
        past = u[lo:hi].float().cumsum(0)
        target[lo:hi] = past / torch.arange(1, hi - lo + 1, device=device)[:, None].sqrt()
    optimizer = torch.optim.AdamW(layer.parameters(), lr=2e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        optimizer.zero_grad(set_to_none=True)
        loss = F.mse_loss(layer(u, cu).float(), target)
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    return losses


def answer(layer, width, lengths, tokens, device):
    """Prompts in two parts, then single tokens; returns those outputs and the
    outputs of the whole sequences at once, each [sequences, tokens, width]."""
    n = len(lengths)
    seqs = [torch.randn(k + tokens, width, device=device).bfloat16() for k in lengths]
    with torch.no_grad():
        whole = layer(torch.cat(seqs), _edges([k + tokens for k in lengths], device))
    parts = whole.split([k + tokens for k in lengths])
    want = torch.stack([p[-tokens:] for p in parts])

    caches = layer.caches(n + 2)
    slots = torch.arange(n + 1, 1, -1, device=device, dtype=torch.int32)  # any slots will do
    first = [k // 2 for k in lengths]
    layer.prefill(torch.cat([s[:k] for s, k in zip(seqs, first)]), _edges(first, device), caches, slots)
    layer.prefill(torch.cat([s[f:k] for s, f, k in zip(seqs, first, lengths)]),
                  _edges([k - f for f, k in zip(first, lengths)], device), caches, slots,
                  resume=torch.ones(n, dtype=torch.bool, device=device))
    got = [layer.step(torch.stack([s[k + i] for s, k in zip(seqs, lengths)]), caches, slots)
           for i in range(tokens)]
    return torch.stack(got, 1), want


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--dim", type=int, default=1024, help="channels of the model, half of the scan's")
    p.add_argument("--states", type=int, default=16)
    p.add_argument("--groups", type=int, default=1)
    p.add_argument("--tokens", type=int, default=4096, help="tokens of a training step, in four documents")
    p.add_argument("--steps", type=int, default=10)
    p.add_argument("--answer", type=int, default=16, help="single tokens after each prompt")
    a = p.parse_args()
    torch.manual_seed(0)
    layer = SsmLayer(a.dim, a.states, a.groups, device="cuda:0")
    cut = a.tokens // 8
    losses = train(layer, a.dim, [cut, 4 * cut, 2 * cut, a.tokens - 7 * cut], a.steps, "cuda:0")
    print("loss %s" % " ".join("%.4f" % v for v in losses))
    got, want = answer(layer, a.dim, [300, 17, 90, 1], a.answer, "cuda:0")
    off = (got.float() - want.float()).norm() / want.float().norm()
    print("single tokens against whole sequences: relative difference %.1e" % off.item())


if __name__ == "__main__":
    main()
