"""A recurrent layer around the packed convolution: the gated linear recurrence
(prompts, training, single tokens), the layer norm on a residual stream, and
carried states that are put aside in 8 bits and taken back.

Like the package's other calls these only check and marshal arguments (C ABI
in include/vdc.h); every step of the computation runs in libvdc.so's HIP
kernels on the current stream, and there is no fallback.  Activation inputs
are BF16 with dense rows (a slice of wider rows is fine), outputs are dense.

The checks are in C++ (csrc/vdc_torch.cpp, built beside the library): in Python
they take longer than the kernels of a single token.
"""
from __future__ import annotations

import os
import threading

import torch  # noqa: F401  (the binding needs its libraries)

from ._build import BINDING
from ._lib import VDC_BWD, VDC_FWD, load

__all__ = ["gated_recurrence_fwd", "gated_recurrence_bwd", "gated_recurrence_keep_rows",
           "gated_recurrence_workspace_bytes", "gated_recurrence_update", "layer_norm_fwd", "layer_norm_bwd",
           "layer_norm_workspace_bytes", "state_quantize", "state_dequantize"]

_lock = threading.Lock()


class _Binding:
    """The compiled calls, loaded when the first of them is made."""

    def __getattr__(self, name):
        with _lock:
            if not os.path.exists(BINDING):
                raise ImportError("%s is not built; run varlen_depthwise_causal_amd._build.build() or "
                                  "__graft_entry__.build()" % BINDING)
            from . import _vdc_torch
            for n in dir(_vdc_torch):
                if not n.startswith("_"):
                    setattr(self, n, getattr(_vdc_torch, n))
        return object.__getattribute__(self, name)


_call = _Binding()


# ---------------------------------------------- gated linear recurrence --

def gated_recurrence_keep_rows(S: int) -> int:
    """Rows of the states that gated_recurrence_fwd keeps for its backward."""
    return int(load().gated_recurrence_keep_rows(S))


def gated_recurrence_workspace_bytes(direction: str, S: int, C: int) -> int:
    """Workspace bytes of gated_recurrence_fwd ("fwd") / gated_recurrence_bwd ("bwd")."""
    return int(load().gated_recurrence_workspace_bytes({"fwd": VDC_FWD, "bwd": VDC_BWD}[direction], S, C))


def gated_recurrence_fwd(x, r, i, decay, cu_seqlens, *, z=None, scale=8.0, state=None, state_index=None, resume=None,
                         keep=None, out=None, workspace=None):
    """The gated linear recurrence over packed documents; returns y, BF16 [S, C].

    With u = 2 scale softplus(decay) sigmoid(r):

        h[t] = exp(-u / 2) h[t-1] + sqrt(1 - exp(-u)) sigmoid(i) x,   y = h silu(z), or h

    x, r, i, z: BF16 [S, C]; decay: [C], FP32 or BF16.  A token with r at -inf
    or the lowest finite number (a masked token) leaves the state as it is.
    state: FP32 [slots, C], where every document leaves its last state;
    state_index and resume as in conv1d_prefill.
    keep: True, or an FP32 [gated_recurrence_keep_rows(S), C] tensor, for
    training (without a state): returns (y, keep) with the states that
    gated_recurrence_bwd starts from."""
    return _call.recurrence_fwd(x, r, i, decay, z, scale, cu_seqlens, state, state_index, resume, keep, out, workspace)


def gated_recurrence_bwd(x, r, i, decay, cu_seqlens, dy, keep, *, z=None, scale=8.0, workspace=None):
    """Gradients of gated_recurrence_fwd without a state, from its inputs and
    what it kept of them: (dx, dr, di, ddecay, dz), dz None without a gate.
    ddecay has decay's dtype, the others BF16."""
    return _call.recurrence_bwd(x, r, i, decay, z, scale, cu_seqlens, dy, keep, workspace)


def gated_recurrence_update(x, r, i, decay, state, *, z=None, scale=8.0, state_index=None, out=None):
    """One token of each sequence through the recurrence: x, r, i, z BF16
    [rows, C]; state FP32 [slots, C], read and replaced.  A row without a slot
    is padding and gives zeros.  Returns y."""
    return _call.recurrence_update(x, r, i, decay, z, scale, state, state_index, out)


# ------------------------------------------------------------ layer norm --

def layer_norm_fwd(x, weight, *, bias=None, residual=None, eps=1e-5, out=None, stream_out=None):
    """Layer norm of each token's channels on a residual stream: with s =
    bf16(x + residual), or x without one, y = weight * xhat(s) + bias.
    x, residual: BF16 [S, C], C at most 16384; weight, bias: FP32 or BF16 [C].
    Returns (y, s); s is x itself without a residual."""
    return _call.norm_fwd(x, weight, bias, residual, eps, out, stream_out)


def layer_norm_workspace_bytes(S: int, C: int) -> int:
    """Workspace bytes of layer_norm_bwd."""
    return int(load().layer_norm_workspace_bytes(S, C))


def layer_norm_bwd(s, weight, dy, *, bias=None, dstream=None, eps=1e-5, workspace=None):
    """Gradients of layer_norm_fwd from what it normalised: (dx, dweight,
    dbias), dbias None without a bias.  dstream, BF16 [S, C]: the gradient that
    reaches the sum past the norm; dx has it added and is the gradient of x and
    of the residual alike."""
    return _call.norm_bwd(s, weight, dy, bias, dstream, eps, workspace)


# ------------------------------------------------------ states put aside --

def state_quantize(state, codes, scales, *, state_index=None, pool_index=None):
    """Carried states put aside: states leave a cache for a pool of 8-bit codes
    with a scale for every 64 values.

    state: FP32 or BF16 [slots, ...], a cache of any of the package's operators;
    codes: int8 or float8_e4m3fn [pool, E], E values of a state; scales: FP32
    [pool, ceil(E / 64)].  State state_index[j] goes to place pool_index[j] (int32;
    j itself without one; as many as the index has, or as the cache has slots); one
    whose slot or place does not exist is left out.  No place may be named twice."""
    _call.quantize(state, codes, scales, state_index, pool_index)


def state_dequantize(codes, scales, state, *, pool_index=None, state_index=None):
    """States put aside by state_quantize taken back into a cache, in place:
    code * scale.  Arguments as there; no slot may be named twice."""
    _call.dequantize(state, codes, scales, state_index, pool_index)
