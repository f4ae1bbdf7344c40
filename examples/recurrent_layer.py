"""A stack of recurrent layers made of the package's operators: a few steps of
training on packed documents, then prompts and single tokens from carried
states, and sequences that are put aside in 8 bits and taken back.

    python3 examples/recurrent_layer.py [--dim 1024] [--layers 2] [--tokens 4096]
                                        [--steps 10] [--answer 16]

A layer: the layer norm on the residual stream; a projection to a gate and the
recurrence's inputs; the causal convolution with SiLU over the inputs; a
projection of them to the recurrence's two gates; the gated linear recurrence; a
projection back.  The projections are PyTorch's.  Prompts of several documents
and the tokens that follow them one at a time go through the same weights, with
the last inputs of the convolution and the states of the recurrence carried in
two caches a layer; the example checks that they answer as the whole sequences
at once do.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch import nn
from torch.nn import functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import varlen_depthwise_causal_amd as vdc  # noqa: E402
from varlen_depthwise_causal_amd import autograd as vga  # noqa: E402

BLOCK = 64  # values of a state that share a scale when it is put aside


class RecurrentLayer(nn.Module):
    """width channels in the model, inner = 3 / 2 of it in the recurrence (a multiple of 8)."""

    def __init__(self, width, device=None):
        super().__init__()
        self.inner = inner = width * 3 // 2 // 8 * 8
        bf16 = {"dtype": torch.bfloat16, "device": device}
        self.norm_weight = nn.Parameter(torch.ones(width, device=device))
        self.norm_bias = nn.Parameter(torch.zeros(width, device=device))
        self.proj_in = nn.Linear(width, 2 * inner, bias=False, **bf16)
        self.proj_gates = nn.Linear(inner, 2 * inner, **bf16)
        self.proj_out = nn.Linear(inner, width, bias=False, **bf16)
        self.conv_weight = nn.Parameter(torch.empty(inner, 4, device=device).uniform_(-0.5, 0.5))
        self.conv_bias = nn.Parameter(torch.zeros(inner, device=device))
        # decays of 0.9 to 0.999 a token at an open gate
        soft = -torch.empty(inner, device=device).uniform_(0.9, 0.999).log() / 8
        self.decay = nn.Parameter(soft + torch.log(-torch.expm1(-soft)))

    def mix(self, y, cu_seqlens):
        """Packed documents, each from a zero state; differentiable."""
        x, z = self.proj_in(y).split(self.inner, dim=-1)
        x = vga.causal_conv1d_silu(x.contiguous(), self.conv_weight, cu_seqlens, self.conv_bias)
        r, i = self.proj_gates(x).split(self.inner, dim=-1)
        return self.proj_out(vga.gated_recurrence(x, r, i, self.decay, cu_seqlens, z))

    def caches(self, slots):
        """The carried states of that many sequences."""
        device = self.decay.device
        return (torch.zeros(slots, 3, self.inner, dtype=torch.bfloat16, device=device),
                torch.zeros(slots, self.inner, device=device))

    def prefill(self, y, cu_seqlens, caches, slots, resume):
        x, z = self.proj_in(y).split(self.inner, dim=-1)
        conv, state = caches
        x = vdc.conv1d_prefill(x.contiguous(), self.conv_weight, cu_seqlens, conv, bias=self.conv_bias,
                               state_index=slots, resume=resume)
        r, i = self.proj_gates(x).split(self.inner, dim=-1)
        return self.proj_out(vdc.gated_recurrence_fwd(x, r, i, self.decay, cu_seqlens, z=z, state=state,
                                                      state_index=slots, resume=resume))

    def step(self, y, caches, slots):
        x, z = self.proj_in(y).split(self.inner, dim=-1)
        conv, state = caches
        x = vdc.conv1d_update(x, conv, self.conv_weight, bias=self.conv_bias, state_index=slots)
        r, i = self.proj_gates(x).split(self.inner, dim=-1)
        return self.proj_out(vdc.gated_recurrence_update(x, r, i, self.decay, state, z=z, state_index=slots))


class RecurrentModel(nn.Module):
    def __init__(self, width, layers=2, device=None):
        super().__init__()
        self.layers = nn.ModuleList(RecurrentLayer(width, device) for _ in range(layers))
        self.norm_weight = nn.Parameter(torch.ones(width, device=device))
        self.norm_bias = nn.Parameter(torch.zeros(width, device=device))

    def forward(self, u, cu_seqlens):
        """Packed documents u [S, width], each from a zero state; differentiable."""
        stream, branch = None, u
        for layer in self.layers:
            if stream is None:
                y, stream = vga.layer_norm(u, layer.norm_weight, layer.norm_bias), u
            else:
                y, stream = vga.layer_norm(branch, layer.norm_weight, layer.norm_bias, stream)
            branch = layer.mix(y, cu_seqlens)
        return vga.layer_norm(branch, self.norm_weight, self.norm_bias, stream)[0]

    def caches(self, slots):
        return [layer.caches(slots) for layer in self.layers]

    @torch.no_grad()
    def _serve(self, u, run):
        stream, branch = None, u
        for n, layer in enumerate(self.layers):
            y, stream = vdc.layer_norm_fwd(branch, layer.norm_weight, bias=layer.norm_bias, residual=stream)
            branch = run(layer, n, y)
        return vdc.layer_norm_fwd(branch, self.norm_weight, bias=self.norm_bias, residual=stream)[0]

    def prefill(self, u, cu_seqlens, caches, slots, resume=None):
        """Packed prompts; document i leaves its states in slot slots[i], and
        goes on from them where resume[i]."""
        return self._serve(u, lambda layer, n, y: layer.prefill(y, cu_seqlens, caches[n], slots, resume))

    def step(self, u, caches, slots):
        """One token of each sequence, u [rows, width]; row i has slot slots[i]."""
        return self._serve(u, lambda layer, n, y: layer.step(y, caches[n], slots))


class Pool:
    """Places for states put aside, a byte a value and a scale for 64 of them."""

    def __init__(self, caches, places, code=torch.int8):
        self.held = []
        for layer in caches:
            for cache in layer:
                E = cache[0].numel()
                codes = torch.zeros(places, E, dtype=torch.int8, device=cache.device).view(code)
                scales = torch.zeros(places, (E + BLOCK - 1) // BLOCK, device=cache.device)
                self.held.append((codes, scales))

    def put(self, caches, slots, places):
        """The sequences of these slots leave for these places."""
        for cache, (codes, scales) in zip((c for layer in caches for c in layer), self.held):
            vdc.state_quantize(cache, codes, scales, state_index=slots, pool_index=places)

    def take(self, caches, slots, places):
        """The sequences of these places come back, to any slots."""
        for cache, (codes, scales) in zip((c for layer in caches for c in layer), self.held):
            vdc.state_dequantize(codes, scales, cache, pool_index=places, state_index=slots)


def _edges(lengths, device):
    return torch.tensor([0] + lengths, device=device).cumsum(0).to(torch.int32)


def train(model, width, lengths, steps, device):
    """Plain gradient descent towards targets that depend on earlier tokens;
    returns the losses."""
    cu = _edges(lengths, device)
    u = torch.randn(sum(lengths), width, device=device).bfloat16()
    target = torch.zeros_like(u, dtype=torch.float32)
    for lo, hi in zip(cu.tolist(), cu.tolist()[1:]):
        past = u[lo:hi].float().cumsum(0)
        target[lo:hi] = past / torch.arange(1, hi - lo + 1, device=device)[:, None].sqrt()
    optimizer = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        optimizer.zero_grad(set_to_none=True)
        loss = F.mse_loss(model(u, cu).float(), target)
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    return losses


def answer(model, width, lengths, tokens, device, park=None):
    """Prompts in two parts, then single tokens; returns those outputs and the
    outputs of the whole sequences at once, each [sequences, tokens, width].
    park: the code (torch.int8 or torch.float8_e4m3fn) in which all sequences are
    put aside between the prompts and the tokens, to come back in other slots."""
    n = len(lengths)
    seqs = [torch.randn(k + tokens, width, device=device).bfloat16() for k in lengths]
    with torch.no_grad():
        whole = model(torch.cat(seqs), _edges([k + tokens for k in lengths], device))
    parts = whole.split([k + tokens for k in lengths])
    want = torch.stack([p[-tokens:] for p in parts])

    caches = model.caches(n + 2)
    slots = torch.arange(n + 1, 1, -1, device=device, dtype=torch.int32)  # any slots will do
    first = [k // 2 for k in lengths]
    model.prefill(torch.cat([s[:k] for s, k in zip(seqs, first)]), _edges(first, device), caches, slots)
    model.prefill(torch.cat([s[f:k] for s, f, k in zip(seqs, first, lengths)]),
                  _edges([k - f for f, k in zip(first, lengths)], device), caches, slots,
                  resume=torch.ones(n, dtype=torch.bool, device=device))
    if park is not None:
        pool = Pool(caches, n, park)
        places = torch.arange(n, device=device, dtype=torch.int32)
        pool.put(caches, slots, places)
        slots = slots - 2
        pool.take(caches, slots, places)
    got = [model.step(torch.stack([s[k + i] for s, k in zip(seqs, lengths)]), caches, slots)
           for i in range(tokens)]
    return torch.stack(got, 1), want


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--dim", type=int, default=1024, help="channels of the model")
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--tokens", type=int, default=4096, help="tokens of a training step, in four documents")
    p.add_argument("--steps", type=int, default=10)
    p.add_argument("--answer", type=int, default=16, help="single tokens after each prompt")
    a = p.parse_args()
    torch.manual_seed(0)
    model = RecurrentModel(a.dim, a.layers, device="cuda:0")
    cut = a.tokens // 8
    losses = train(model, a.dim, [cut, 4 * cut, 2 * cut, a.tokens - 7 * cut], a.steps, "cuda:0")
    print("loss %s" % " ".join("%.4f" % v for v in losses))
    for park in (None, torch.int8, torch.float8_e4m3fn):
        got, want = answer(model, a.dim, [300, 17, 90, 1], a.answer, "cuda:0", park)
        off = (got.float() - want.float()).norm() / want.float().norm()
        print("single tokens%s against whole sequences: relative difference %.1e"
              % ("" if park is None else " from states put aside as %s" % park, off.item()))


if __name__ == "__main__":
    main()
