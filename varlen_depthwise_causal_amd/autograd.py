"""Autograd wrapper of the packed varlen width-4 depthwise causal conv1d +
SiLU (documentation page CakeCausalConv1dFunction, class description).

Only (x, weight, cu_seqlens, bias) are saved: the backward recomputes the
preactivation from x inside the backward kernel, so no activation other than
the inputs is kept alive between the passes.  The kernels read the output
gradient as dense row-major BF16, so a gradient of any other dtype or
strides is converted (a copy) before the call.  The weight and bias
gradients are returned in the dtypes of the parameters they belong to.
Every step runs in libvdc.so's kernels through conv1d_fwd / conv1d_bwd.

selective_scan and group_norm_silu wrap the other operators of a state space
layer in the same way: the inputs alone are saved, their backward passes
compute the rest again.  So do gated_recurrence, which keeps one state in 64
tokens beside them, and layer_norm, which saves what it normalised.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (
    conv1d_bwd,
    conv1d_fwd,
    gated_recurrence_bwd,
    gated_recurrence_fwd,
    group_norm_silu_bwd,
    group_norm_silu_fwd,
    layer_norm_bwd,
    layer_norm_fwd,
    selective_scan_bwd,
    selective_scan_fwd,
)

__all__ = ["CausalConv1dFunction", "causal_conv1d_silu", "SelectiveScanFunction", "selective_scan",
           "GroupNormSiluFunction", "group_norm_silu", "GatedRecurrenceFunction", "gated_recurrence",
           "LayerNormFunction", "layer_norm"]


def _dense(grad):
    """The gradient as dense rows of BF16, which the kernels read."""
    return grad.to(torch.bfloat16).contiguous()


def _needed(ctx, grads):
    """The gradients of the inputs that need one, in the inputs' order."""
    return tuple(g if n else None for g, n in zip(grads, ctx.needs_input_grad))


class CausalConv1dFunction(torch.autograd.Function):
    """y = bf16(silu(depthwise causal conv(x) + bias)) per document, with the
    backward of conv1d_bwd under the chosen SiLU' policy."""

    @staticmethod
    def forward(ctx, x, weight, cu_seqlens, bias=None, silu_grad_preactivation="bf16"):
        if silu_grad_preactivation not in ("bf16", "fp32"):
            raise ValueError("silu_grad_preactivation must be 'bf16' or 'fp32'")
        y = conv1d_fwd(x, weight, cu_seqlens, bias=bias)
        ctx.save_for_backward(x, weight, cu_seqlens, bias)
        ctx.policy = silu_grad_preactivation
        return y

    @staticmethod
    def backward(ctx, grad_y):
        x, weight, cu_seqlens, bias = ctx.saved_tensors
        dy = grad_y
        if dy.dtype != torch.bfloat16 or not dy.is_contiguous():
            dy = dy.to(torch.bfloat16).contiguous()
        grads = conv1d_bwd(x, weight, cu_seqlens, dy, bias=bias,
                           silu_grad_preactivation=ctx.policy)
        dx, dweight = grads[0], grads[1]
        dbias = grads[2] if bias is not None else None
        need = ctx.needs_input_grad
        return (dx if need[0] else None, dweight if need[1] else None, None,
                dbias if (bias is not None and need[3]) else None, None)


def causal_conv1d_silu(x, weight, cu_seqlens, bias=None, silu_grad_preactivation="bf16"):
    """Differentiable forward: returns y (x's shape, BF16)."""
    return CausalConv1dFunction.apply(x, weight, cu_seqlens, bias, silu_grad_preactivation)


class SelectiveScanFunction(torch.autograd.Function):
    """selective_scan_fwd without a carried state, with the backward of
    selective_scan_bwd.  dA, dD and ddt_bias come in the parameters' dtypes."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, dt_softplus=True):
        y = selective_scan_fwd(x, dt, A, B, C, cu_seqlens, D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus)
        ctx.save_for_backward(x, dt, A, B, C, cu_seqlens, D, z, dt_bias)
        ctx.dt_softplus = dt_softplus
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, dt, A, B, C, cu_seqlens, D, z, dt_bias = ctx.saved_tensors
        dx, ddt, dA, dB, dC, dD, dz, dbias = selective_scan_bwd(
            x, dt, A, B, C, cu_seqlens, _dense(grad_y), D=D, z=z, dt_bias=dt_bias, dt_softplus=ctx.dt_softplus)
        return _needed(ctx, (dx, ddt, dA, dB, dC, None, dD, dz, dbias, None))


def selective_scan(x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, dt_softplus=True):
    """Differentiable selective scan over packed documents, each from a zero
    state: returns y, BF16 [S, C].  Arguments as in selective_scan_fwd."""
    return SelectiveScanFunction.apply(x, dt, A, B, C, cu_seqlens, D, z, dt_bias, dt_softplus)


class GroupNormSiluFunction(torch.autograd.Function):
    """group_norm_silu_fwd with the backward of group_norm_silu_bwd."""

    @staticmethod
    def forward(ctx, x, weight, groups, bias=None, z=None, eps=1e-5):
        y = group_norm_silu_fwd(x, weight, groups, bias=bias, z=z, eps=eps)
        ctx.save_for_backward(x, weight, bias, z)
        ctx.groups, ctx.eps = groups, eps
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, weight, bias, z = ctx.saved_tensors
        dx, dweight, dbias, dz = group_norm_silu_bwd(x, weight, ctx.groups, _dense(grad_y), bias=bias, z=z,
                                                     eps=ctx.eps)
        return _needed(ctx, (dx, dweight, None, dbias, dz, None))


def group_norm_silu(x, weight, groups, bias=None, z=None, eps=1e-5):
    """Differentiable gated group norm: returns y, BF16 [S, C].  Arguments as
    in group_norm_silu_fwd."""
    return GroupNormSiluFunction.apply(x, weight, groups, bias, z, eps)


class GatedRecurrenceFunction(torch.autograd.Function):
    """gated_recurrence_fwd without a carried state, with the backward of
    gated_recurrence_bwd.  ddecay comes in the parameter's dtype."""

    @staticmethod
    def forward(ctx, x, r, i, decay, cu_seqlens, z=None, scale=8.0):
        y, keep = gated_recurrence_fwd(x, r, i, decay, cu_seqlens, z=z, scale=scale, keep=True)
        ctx.save_for_backward(x, r, i, decay, cu_seqlens, z, keep)
        ctx.scale = scale
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, r, i, decay, cu_seqlens, z, keep = ctx.saved_tensors
        dx, dr, di, ddecay, dz = gated_recurrence_bwd(x, r, i, decay, cu_seqlens, _dense(grad_y), keep, z=z,
                                                      scale=ctx.scale)
        return _needed(ctx, (dx, dr, di, ddecay, None, dz, None))


def gated_recurrence(x, r, i, decay, cu_seqlens, z=None, scale=8.0):
    """Differentiable gated linear recurrence over packed documents, each from
    a zero state: returns y, BF16 [S, C].  Arguments as in gated_recurrence_fwd."""
    return GatedRecurrenceFunction.apply(x, r, i, decay, cu_seqlens, z, scale)


class LayerNormFunction(torch.autograd.Function):
    """layer_norm_fwd with the backward of layer_norm_bwd.  x and the residual
    have one gradient, in which the stream's own joins the norm's."""

    @staticmethod
    def forward(ctx, x, weight, bias=None, residual=None, eps=1e-5):
        y, stream = layer_norm_fwd(x, weight, bias=bias, residual=residual, eps=eps)
        ctx.save_for_backward(stream, weight, bias)
        ctx.eps, ctx.sum = eps, residual is not None
        ctx.set_materialize_grads(False)
        return (y, stream) if ctx.sum else y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_stream=None):
        stream, weight, bias = ctx.saved_tensors
        if grad_y is None:  # only the stream goes on
            return _needed(ctx, (grad_stream, None, None, grad_stream, None))
        dstream = None if grad_stream is None else _dense(grad_stream)
        dx, dweight, dbias = layer_norm_bwd(stream, weight, _dense(grad_y), bias=bias, dstream=dstream, eps=ctx.eps)
        return _needed(ctx, (dx, dweight, dbias, dx if ctx.sum else None, None))


def layer_norm(x, weight, bias=None, residual=None, eps=1e-5):
    """Differentiable layer norm: returns y, BF16 [S, C], or (y, stream) where
    a residual is added first.  Arguments as in layer_norm_fwd."""
    return LayerNormFunction.apply(x, weight, bias, residual, eps)
