"""A recurrent layer around the packed convolution: the gated linear recurrence
(prompts, training, single tokens), the layer norm on a residual stream, and
carried states that are put aside in 8 bits and taken back.

Like the package's other calls these only check and marshal arguments (C ABI
in include/vdc.h); every step of the computation runs in libvdc.so's HIP
kernels on the current stream, and there is no fallback.  Activation inputs
are BF16 with dense rows (a slice of wider rows is fine), outputs are dense.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from ._lib import VDC_BWD, VDC_E4M3, VDC_FWD, VDC_INT8, VdcError, VdcRecurrence, load
from .ssm import _CODES, _at, _cache, _cu, _dense, _out, _param, _ptr, _rows, _stream, _workspace

__all__ = ["gated_recurrence_fwd", "gated_recurrence_bwd", "gated_recurrence_keep_rows",
           "gated_recurrence_workspace_bytes", "gated_recurrence_update", "layer_norm_fwd", "layer_norm_bwd",
           "layer_norm_workspace_bytes", "state_quantize", "state_dequantize"]

_F32, _BF16 = torch.float32, torch.bfloat16


# As in module ssm the checks first ask whether a tensor is the usual one; most
# of what a single token costs is the host's.

def _act(t, what, shape, C, device):
    """Row stride of a BF16 [S, C] activation whose rows are dense."""
    if t.dtype is _BF16 and t.shape == shape and t.device == device:
        stride, one = t.stride()
        if one == 1 and C <= stride <= 1 << 25:
            return stride
    return _rows(t, what, shape, C, device)


def _x_act(x):
    """Sizes, device and row stride of the activation that gives them."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, C], got %s" % (list(x.shape),))
    shape, device = x.shape, x.device
    S, C = shape
    stride = _act(x, "x", shape, C, device)
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    return shape, S, C, device, stride


def _recur_cache(state, C, state_index, resume, sequences, device):
    """Number of slots of an FP32 [slots, C] cache."""
    if (state.dtype is _F32 and state.dim() == 2 and state.shape[1] == C and state.is_contiguous()
            and state.device == device and state_index is not None and _list(state_index, torch.int32, sequences, device)
            and (resume is None or _list(resume, torch.bool, sequences, device))):
        return state.shape[0]
    return _cache(state, "state", (C,), _F32, state_index, resume, sequences, device)


def _list(t, dtype, n, device):
    return t.dtype is dtype and t.shape == (n,) and t.is_contiguous() and t.device == device


@functools.lru_cache(maxsize=1024)
def _bytes(name, *sizes):
    return int(getattr(load(), name)(*sizes))


# The library launches on the device that is current, so a call for tensors on
# another one is made with that one current.
_device_at = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, device, *args):
    fn = getattr(load(), name)
    if _device_at() == device.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc:
        raise VdcError(rc, name)


# ---------------------------------------------- gated linear recurrence --

# struct vdc_recurrence of include/vdc.h, field by field; bytes, made by one call.
_RECUR = struct.Struct("@2q4P4qPifPqPqPP")
assert _RECUR.size == ctypes.sizeof(VdcRecurrence)


def _recur_args(x, r, i, decay, z, scale, cu_seqlens, state, state_index, resume):
    shape, S, C, dev, xs = _x_act(x)
    rs, is_ = _act(r, "r", shape, C, dev), _act(i, "i", shape, C, dev)
    zs = C if z is None else _act(z, "z", shape, C, dev)
    code = _param(decay, "decay", (C,), dev)
    sequences, docs, slots = S, 0, 0
    if cu_seqlens is not None:
        sequences = docs = _cu(cu_seqlens, dev)
    if state is not None:
        slots = _recur_cache(state, C, state_index, resume, sequences, dev)
    elif state_index is not None or resume is not None:
        raise ValueError("state_index and resume need a state")
    a = _RECUR.pack(S, C, x.data_ptr(), r.data_ptr(), i.data_ptr(), _at(z), xs, rs, is_, zs, decay.data_ptr(), code,
                    scale, _at(cu_seqlens), docs, _at(state), slots, _at(state_index), _at(resume))
    return a, S, C, dev, xs


def gated_recurrence_keep_rows(S: int) -> int:
    """Rows of the states that gated_recurrence_fwd keeps for its backward."""
    return _bytes("gated_recurrence_keep_rows", S)


def gated_recurrence_workspace_bytes(direction: str, S: int, C: int) -> int:
    """Workspace bytes of gated_recurrence_fwd ("fwd") / gated_recurrence_bwd ("bwd")."""
    return _bytes("gated_recurrence_workspace_bytes", {"fwd": VDC_FWD, "bwd": VDC_BWD}[direction], S, C)


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
    a, S, C, dev, xs = _recur_args(x, r, i, decay, z, scale, cu_seqlens, state, state_index, resume)
    out = _out(out, x, xs, x.shape, "out", dev)
    want = keep is not None and keep is not False
    if want:
        if state is not None:
            raise ValueError("keep is for the training forward, without a state")
        shape = (gated_recurrence_keep_rows(S), C)
        if keep is True:
            keep = torch.empty(shape, dtype=_F32, device=dev)
        else:
            _dense(keep, "keep", _F32, shape, dev)
    need = _bytes("gated_recurrence_workspace_bytes", VDC_FWD, S, C)
    ws, ws_n = None, 0
    if need or workspace is not None:
        workspace, ws_n = _workspace(need, workspace, dev)
        ws = workspace.data_ptr()
    _call("gated_recurrence_fwd", dev, a, out.data_ptr(), keep.data_ptr() if want else None, ws, ws_n, _stream(dev))
    return (out, keep) if want else out


def gated_recurrence_bwd(x, r, i, decay, cu_seqlens, dy, keep, *, z=None, scale=8.0, workspace=None):
    """Gradients of gated_recurrence_fwd without a state, from its inputs and
    what it kept of them: (dx, dr, di, ddecay, dz), dz None without a gate.
    ddecay has decay's dtype, the others BF16."""
    a, S, C, dev, xs = _recur_args(x, r, i, decay, z, scale, cu_seqlens, None, None, None)
    dy_stride = _act(dy, "dy", x.shape, C, dev)
    _dense(keep, "keep", _F32, (gated_recurrence_keep_rows(S), C), dev)
    dx = _out(None, x, xs, x.shape, "dx", dev)
    dr, di = torch.empty_like(dx), torch.empty_like(dx)
    dz = None if z is None else torch.empty_like(dx)
    ddecay = torch.empty_like(decay)
    workspace, ws_n = _workspace(_bytes("gated_recurrence_workspace_bytes", VDC_BWD, S, C), workspace, dev)
    _call("gated_recurrence_bwd", dev, a, dy.data_ptr(), dy_stride, keep.data_ptr(), dx.data_ptr(), dr.data_ptr(),
          di.data_ptr(), ddecay.data_ptr(), _ptr(dz), workspace.data_ptr(), ws_n, _stream(dev))
    return dx, dr, di, ddecay, dz


def gated_recurrence_update(x, r, i, decay, state, *, z=None, scale=8.0, state_index=None, out=None):
    """One token of each sequence through the recurrence: x, r, i, z BF16
    [rows, C]; state FP32 [slots, C], read and replaced.  A row without a slot
    is padding and gives zeros.  Returns y."""
    if state is None:
        raise ValueError("gated_recurrence_update needs a state")
    a, _, _, dev, xs = _recur_args(x, r, i, decay, z, scale, None, state, state_index, None)
    out = _out(out, x, xs, x.shape, "out", dev)
    _call("gated_recurrence_update", dev, a, out.data_ptr(), _stream(dev))
    return out


# ------------------------------------------------------------ layer norm --

def layer_norm_fwd(x, weight, *, bias=None, residual=None, eps=1e-5, out=None, stream_out=None):
    """Layer norm of each token's channels on a residual stream: with s =
    bf16(x + residual), or x without one, y = weight * xhat(s) + bias.
    x, residual: BF16 [S, C], C at most 16384; weight, bias: FP32 or BF16 [C].
    Returns (y, s); s is x itself without a residual."""
    shape, S, C, dev, xs = _x_act(x)
    w_code = _param(weight, "weight", (C,), dev)
    b_code = 0 if bias is None else _param(bias, "bias", (C,), dev)
    out = _out(out, x, xs, shape, "out", dev)
    rs = C
    if residual is not None:
        rs = _act(residual, "residual", shape, C, dev)
        stream_out = _out(stream_out, x, xs, shape, "stream_out", dev)
    elif stream_out is not None:
        raise ValueError("stream_out needs a residual")
    _call("layer_norm_fwd", dev, x.data_ptr(), xs, _ptr(residual), rs, weight.data_ptr(), w_code, _ptr(bias), b_code,
          S, C, eps, out.data_ptr(), _ptr(stream_out), _stream(dev))
    return out, x if residual is None else stream_out


def layer_norm_workspace_bytes(S: int, C: int) -> int:
    """Workspace bytes of layer_norm_bwd."""
    return _bytes("layer_norm_workspace_bytes", S, C)


def layer_norm_bwd(s, weight, dy, *, bias=None, dstream=None, eps=1e-5, workspace=None):
    """Gradients of layer_norm_fwd from what it normalised: (dx, dweight,
    dbias), dbias None without a bias.  dstream, BF16 [S, C]: the gradient that
    reaches the sum past the norm; dx has it added and is the gradient of x and
    of the residual alike."""
    shape, S, C, dev, ss = _x_act(s)
    dys = _act(dy, "dy", shape, C, dev)
    w_code = _param(weight, "weight", (C,), dev)
    b_code = 0 if bias is None else _param(bias, "bias", (C,), dev)
    dss = C if dstream is None else _act(dstream, "dstream", shape, C, dev)
    dx = _out(None, s, ss, shape, "dx", dev)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    workspace, ws_n = _workspace(_bytes("layer_norm_workspace_bytes", S, C), workspace, dev)
    _call("layer_norm_bwd", dev, s.data_ptr(), ss, weight.data_ptr(), w_code, dy.data_ptr(), dys, _ptr(dstream), dss,
          S, C, eps, dx.data_ptr(), dw.data_ptr(), _ptr(db), b_code, workspace.data_ptr(), ws_n, _stream(dev))
    return dx, dw, db


# ------------------------------------------------------ states put aside --

_POOL_CODES = {torch.int8: VDC_INT8, torch.float8_e4m3fn: VDC_E4M3}
_POOL_BLOCK = 64


def _pool_args(state, codes, scales, state_index, pool_index):
    dtype = _CODES.get(state.dtype)
    if dtype is None:
        raise TypeError("state must be float32 or bfloat16, got %s" % state.dtype)
    dev = state.device
    if not state.is_cuda:
        raise ValueError("state must be a device tensor")
    if state.dim() < 2 or not state.is_contiguous():
        raise ValueError("state must be a contiguous [slots, ...] cache")
    slots = state.shape[0]
    E = 1
    for n in state.shape[1:]:
        E *= n
    code = _POOL_CODES.get(codes.dtype)
    if code is None:
        raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)
    if codes.dim() != 2 or codes.shape[1] != E:
        raise ValueError("codes must be [pool, %d], got %s" % (E, list(codes.shape)))
    pool = codes.shape[0]
    _dense(codes, "codes", codes.dtype, (pool, E), dev)
    _dense(scales, "scales", _F32, (pool, (E + _POOL_BLOCK - 1) // _POOL_BLOCK), dev)
    given = [t for t in (state_index, pool_index) if t is not None]
    rows = given[0].numel() if given else slots
    for t, what in ((state_index, "state_index"), (pool_index, "pool_index")):
        if t is not None:
            _dense(t, what, torch.int32, (rows,), dev)
    if (state_index is None and rows > slots) or (pool_index is None and rows > pool):
        raise ValueError("%d states do not fit %d slots and %d places" % (rows, slots, pool))
    return dtype, slots, E, code, pool, rows, dev


def state_quantize(state, codes, scales, *, state_index=None, pool_index=None):
    """Carried states put aside: states leave a cache for a pool of 8-bit codes
    with a scale for every 64 values.

    state: FP32 or BF16 [slots, ...], a cache of any of the package's operators;
    codes: int8 or float8_e4m3fn [pool, E], E values of a state; scales: FP32
    [pool, ceil(E / 64)].  State state_index[j] goes to place pool_index[j] (int32;
    j itself without one; as many as the index has, or as the cache has slots); one
    whose slot or place does not exist is left out.  No place may be named twice."""
    dtype, slots, E, code, pool, rows, dev = _pool_args(state, codes, scales, state_index, pool_index)
    _call("state_quantize", dev, state.data_ptr(), dtype, slots, E, _ptr(state_index), codes.data_ptr(), code,
          scales.data_ptr(), pool, _ptr(pool_index), rows, _stream(dev))


def state_dequantize(codes, scales, state, *, pool_index=None, state_index=None):
    """States put aside by state_quantize taken back into a cache, in place:
    code * scale.  Arguments as there; no slot may be named twice."""
    dtype, slots, E, code, pool, rows, dev = _pool_args(state, codes, scales, state_index, pool_index)
    _call("state_dequantize", dev, codes.data_ptr(), code, scales.data_ptr(), pool, _ptr(pool_index),
          state.data_ptr(), dtype, slots, E, _ptr(state_index), rows, _stream(dev))
