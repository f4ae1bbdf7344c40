"""The state space layer around the packed convolution: the convolution with a
carried state (prompts and single tokens), the selective scan (prompts,
training, single tokens) and the gated group norm.

Like the package's other calls these only check and marshal arguments (C ABI
in include/vdc.h); every step of the computation runs in libvdc.so's HIP
kernels on the current stream, and there is no fallback.  Activation inputs
are BF16 with dense rows (a slice of wider rows is fine), outputs are dense.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from ._lib import VDC_BF16, VDC_BWD, VDC_F32, VDC_FWD, VdcError, VdcScan, load

__all__ = ["conv1d_prefill", "conv1d_update", "selective_scan_fwd", "selective_scan_bwd",
           "selective_scan_workspace_bytes", "selective_update", "group_norm_silu_fwd",
           "group_norm_silu_bwd", "group_norm_silu_workspace_bytes"]

_CODES = {torch.float32: VDC_F32, torch.bfloat16: VDC_BF16}
_BF16 = torch.bfloat16


# The checks below are most of what a call costs the host, and for single tokens
# most of what it costs at all, so each first asks, in one expression, whether a
# tensor is the usual one, and looks for what is wrong with it only if not.  The
# device is x's, which _x_rows has found to be a GPU.

def _rows(t, what, shape, dense, device):
    """Row stride of a BF16 activation of this shape, whose rows of `dense`
    elements are dense themselves."""
    if t.dtype is _BF16 and t.shape == shape and t.device == device and t.is_contiguous():
        return dense
    if t.dtype != _BF16:
        raise TypeError("%s must be bfloat16" % what)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, list(shape), list(t.shape)))
    if t.device != device:
        raise ValueError("%s must be a device tensor on %s" % (what, device))
    strides, inner = t.stride(), 1
    for n, s in zip(reversed(shape[1:]), reversed(strides[1:])):
        if n != 1 and s != inner:
            raise ValueError("%s must have dense rows, got strides %s" % (what, strides))
        inner *= n
    # One row has no stride of its own, and neither has a row of a tensor
    # without elements.
    if shape[0] <= 1 or dense == 0:
        return dense
    if strides[0] < dense:
        raise ValueError("the rows of %s overlap (strides %s)" % (what, strides))
    return strides[0]


def _x_rows(x, C, device):
    stride = _rows(x, "x", x.shape, C, device)
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    return stride


def _param(t, what, shape, device):
    """dtype code of an FP32 or BF16 parameter of this shape."""
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (what, t.dtype))
    if not (t.shape == shape and t.device == device and t.is_contiguous()):
        _dense(t, what, t.dtype, shape, device)
    return code


def _dense(t, what, dtype, shape, device):
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, list(shape), list(t.shape)))
    if t.device != device:
        raise ValueError("%s must be a device tensor on %s" % (what, device))
    raise ValueError("%s must be contiguous" % what)


def _activation(x):
    if x.dim() != 2:
        raise ValueError("x must be [rows, C], got %s" % (list(x.shape),))
    rows, C = x.shape
    return rows, C, x.device


def _out(out, like, stride, shape, what, device):
    """The caller's output, or a new one, shaped like an input whose row stride
    is known."""
    if out is None:
        if stride == shape[-1] and like.is_contiguous():
            return torch.empty_like(like)  # the quickest of torch's ways
        return torch.empty(shape, dtype=_BF16, device=device)
    _dense(out, what, _BF16, shape, device)
    return out


def _cu(cu_seqlens, device):
    if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a non-empty 1-D int32 tensor")
    _dense(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, device)
    return cu_seqlens.numel() - 1


def _cache(state, what, tail, dtype, state_index, resume, sequences, device):
    """Number of slots of a state cache, with the checks of what chooses them."""
    if state.dim() != 1 + len(tail):
        raise ValueError("%s must be [slots, %s]" % (what, ", ".join(map(str, tail))))
    slots = state.shape[0]
    _dense(state, what, dtype, (slots,) + tail, device)
    if state_index is not None:
        _dense(state_index, "state_index", torch.int32, (sequences,), device)
    elif sequences > slots:
        raise ValueError("%s has %d slots for %d sequences" % (what, slots, sequences))
    if resume is not None:
        if resume.dtype not in (torch.bool, torch.uint8):
            raise TypeError("resume must be bool or uint8, got %s" % resume.dtype)
        _dense(resume, "resume", resume.dtype, (sequences,), device)
    return slots


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, which would
# cost as much as half of the smallest kernels.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(need, workspace, device):
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous device tensor on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


# ------------------------------------------- convolution, carried state --

def conv1d_prefill(x, weight, cu_seqlens, state, *, bias=None, state_index=None, resume=None, out=None):
    """conv1d_fwd over packed prompts that may go on from a carried state.

    state: BF16 [slots, 3, C], each sequence's last three inputs (row 0 the
    oldest), updated in place; document i has slot state_index[i] (int32; its
    own number without one, none where the index is outside the cache).
    resume: bool or uint8 [num_docs], documents whose slot is the history
    before their first token (default: none).  Returns y."""
    if x.dim() == 3 and x.shape[0] == 1:
        x = x[0]
        shape = (1,) + tuple(x.shape)
    else:
        shape = x.shape
    S, C, dev = _activation(x)
    if _x_rows(x, C, dev) != C:
        raise ValueError("x must be contiguous")
    w_code = _param(weight, "weight", (C, 4), dev)
    b_code = 0 if bias is None else _param(bias, "bias", (C,), dev)
    docs = _cu(cu_seqlens, dev)
    slots = _cache(state, "state", (3, C), _BF16, state_index, resume, docs, dev)
    if out is None:
        out = torch.empty_like(x) if len(shape) == 2 else torch.empty(shape, dtype=_BF16, device=dev)
    else:
        _dense(out, "out", _BF16, shape, dev)
    rc = load().conv1d_prefill(_ptr(x), _ptr(weight), w_code, _ptr(bias), b_code, _ptr(cu_seqlens),
                               docs, S, C, _ptr(state), slots, _ptr(state_index), _ptr(resume),
                               _ptr(out), _stream(dev))
    if rc:
        raise VdcError(rc, "conv1d_prefill")
    return out


def conv1d_update(x, state, weight, *, bias=None, state_index=None, out=None):
    """One token of each sequence through the convolution: x BF16 [rows, C];
    state as in conv1d_prefill, read and moved up by the token.  A row without
    a slot is padding and gives zeros.  Returns y [rows, C]."""
    rows, C, dev = _activation(x)
    stride = _x_rows(x, C, dev)
    w_code = _param(weight, "weight", (C, 4), dev)
    b_code = 0 if bias is None else _param(bias, "bias", (C,), dev)
    slots = _cache(state, "state", (3, C), _BF16, state_index, None, rows, dev)
    out = _out(out, x, stride, x.shape, "out", dev)
    rc = load().conv1d_update(_ptr(x), stride, _ptr(weight), w_code, _ptr(bias), b_code, rows, C,
                              _ptr(state), slots, _ptr(state_index), _ptr(out), _stream(dev))
    if rc:
        raise VdcError(rc, "conv1d_update")
    return out


# -------------------------------------------------------- selective scan --

# struct vdc_scan of include/vdc.h, field by field; bytes, made by one call,
# where a ctypes structure takes one for each field.
_SCAN = struct.Struct("@4q5P5q3P4iPqPqPP")
assert _SCAN.size == ctypes.sizeof(VdcScan)


def _at(t):
    return 0 if t is None else t.data_ptr()


def _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu_seqlens, state, state_index, resume):
    S, width, dev = _activation(x)
    if A.dim() != 2 or B.dim() not in (2, 3):
        raise ValueError("A must be [C, N] and B, C [rows, groups, N] or [rows, N]")
    N = A.shape[1]
    if B.dim() == 2:
        B, C = B.unsqueeze(1), C.unsqueeze(1)
    groups = B.shape[1]
    shape, bc_shape, per_row = x.shape, (S, groups, N), groups * N
    zs, d_code, bias_code = width, 0, 0
    xs, dts = _x_rows(x, width, dev), _rows(dt, "dt", shape, width, dev)
    if z is not None:
        zs = _rows(z, "z", shape, width, dev)
    Bs, Cs = _rows(B, "B", bc_shape, per_row, dev), _rows(C, "C", bc_shape, per_row, dev)
    a_code = _param(A, "A", (width, N), dev)
    if D is not None:
        d_code = _param(D, "D", (width,), dev)
    if dt_bias is not None:
        bias_code = _param(dt_bias, "dt_bias", (width,), dev)
    sequences, docs, slots = S, 0, 0
    if cu_seqlens is not None:
        sequences = docs = _cu(cu_seqlens, dev)
    if state is not None:
        slots = _cache(state, "state", (width, N), torch.float32, state_index, resume, sequences, dev)
    elif state_index is not None or resume is not None:
        raise ValueError("state_index and resume need a state")
    a = _SCAN.pack(S, width, N, groups, x.data_ptr(), dt.data_ptr(), _at(z), B.data_ptr(), C.data_ptr(),
                   xs, dts, zs, Bs, Cs, A.data_ptr(), _at(D), _at(dt_bias), a_code, d_code, bias_code,
                   1 if dt_softplus else 0, _at(cu_seqlens), docs, _at(state), slots, _at(state_index),
                   _at(resume))
    return a, S, width, N, groups, dev, xs


def selective_scan_workspace_bytes(direction: str, S: int, C: int, N: int, groups: int = 1) -> int:
    """Workspace bytes of selective_scan_fwd ("fwd") / selective_scan_bwd ("bwd")."""
    d = {"fwd": VDC_FWD, "bwd": VDC_BWD}[direction]
    return int(load().selective_scan_workspace_bytes(d, S, C, N, groups))


def selective_scan_fwd(x, dt, A, B, C, cu_seqlens, *, D=None, z=None, dt_bias=None, dt_softplus=True,
                       state=None, state_index=None, resume=None, out=None, workspace=None):
    """The selective scan over packed documents; returns y, BF16 [S, C].

    x, dt, z: BF16 [S, C]; B, C: BF16 [S, groups, N] or [S, N]; A: [C, N], D and
    dt_bias: [C], each FP32 or BF16.  The step size is softplus(dt + dt_bias),
    0 at -inf (a masked token), or their sum without dt_softplus; y is gated by
    silu(z) where z is given.
    state: FP32 [slots, C, N], where every document leaves its last state;
    state_index and resume as in conv1d_prefill."""
    a, S, width, N, groups, dev, xs = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu_seqlens,
                                                 state, state_index, resume)
    out = _out(out, x, xs, x.shape, "out", dev)
    lib = load()
    need = lib.selective_scan_workspace_bytes(VDC_FWD, S, width, N, groups)
    ws, ws_n = None, 0
    if need or workspace is not None:
        workspace, ws_n = _workspace(need, workspace, dev)
        ws = workspace.data_ptr()
    rc = lib.selective_scan_fwd(a, out.data_ptr(), ws, ws_n, _stream(dev))
    if rc:
        raise VdcError(rc, "selective_scan_fwd")
    return out


def selective_scan_bwd(x, dt, A, B, C, cu_seqlens, dy, *, D=None, z=None, dt_bias=None,
                       dt_softplus=True, workspace=None):
    """Gradients of selective_scan_fwd without a state, from its inputs alone:
    (dx, ddt, dA, dB, dC, dD, dz, ddt_bias), None for what was not given.
    dA, dD and ddt_bias have the parameters' dtypes, the others BF16."""
    a, S, width, N, groups, dev, xs = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu_seqlens,
                                                 None, None, None)
    dy_stride = _rows(dy, "dy", x.shape, width, dev)
    dx = _out(None, x, xs, x.shape, "dx", dev)
    ddt = torch.empty_like(dx)
    dz = None if z is None else torch.empty_like(dx)
    dB = torch.empty(B.shape, dtype=_BF16, device=dev)
    dC = torch.empty(B.shape, dtype=_BF16, device=dev)
    dA = torch.empty_like(A)
    dD = None if D is None else torch.empty_like(D)
    dbias = None if dt_bias is None else torch.empty_like(dt_bias)
    lib = load()
    need = lib.selective_scan_workspace_bytes(VDC_BWD, S, width, N, groups)
    workspace, ws_n = _workspace(need, workspace, dev)
    rc = lib.selective_scan_bwd(a, dy.data_ptr(), dy_stride, dx.data_ptr(), ddt.data_ptr(),
                                _ptr(dz), dB.data_ptr(), dC.data_ptr(), dA.data_ptr(), _ptr(dD),
                                _ptr(dbias), workspace.data_ptr(), ws_n, _stream(dev))
    if rc:
        raise VdcError(rc, "selective_scan_bwd")
    return dx, ddt, dA, dB, dC, dD, dz, dbias


def selective_update(x, dt, A, B, C, state, *, D=None, z=None, dt_bias=None, dt_softplus=True,
                     state_index=None, out=None):
    """One token of each sequence through the scan: x, dt, z BF16 [rows, C], B
    and C [rows, groups, N] or [rows, N]; state FP32 [slots, C, N], read and
    replaced.  A row without a slot is padding and gives zeros.  Returns y."""
    if state is None:
        raise ValueError("selective_update needs a state")
    a, _, _, _, _, dev, xs = _scan_args(x, dt, A, B, C, D, z, dt_bias, dt_softplus, None, state, state_index,
                                        None)
    out = _out(out, x, xs, x.shape, "out", dev)
    rc = load().selective_update(a, out.data_ptr(), _stream(dev))
    if rc:
        raise VdcError(rc, "selective_update")
    return out


# ------------------------------------------------------------ group norm --

def _norm_args(x, weight, groups, bias, z):
    S, C, dev = _activation(x)
    groups = int(groups)
    if groups < 1 or C % groups:
        raise ValueError("groups must divide C = %d, got %d" % (C, groups))
    xs = _x_rows(x, C, dev)
    w_code = _param(weight, "weight", (C,), dev)
    b_code = 0 if bias is None else _param(bias, "bias", (C,), dev)
    zs = C if z is None else _rows(z, "z", x.shape, C, dev)
    return S, C, dev, groups, xs, w_code, b_code, zs


def group_norm_silu_fwd(x, weight, groups, *, bias=None, z=None, eps=1e-5, out=None):
    """Group norm of each token's channels with a SiLU, channels last: with v =
    weight * xhat + bias, y = silu(v), or v * silu(z) where a gate z is given.
    x, z: BF16 [S, C]; weight, bias: FP32 or BF16 [C].  Returns y."""
    S, C, dev, groups, xs, w_code, b_code, zs = _norm_args(x, weight, groups, bias, z)
    out = _out(out, x, xs, x.shape, "out", dev)
    rc = load().group_norm_silu_fwd(x.data_ptr(), xs, weight.data_ptr(), w_code, _ptr(bias), b_code,
                                    _ptr(z), zs, S, C, groups, eps, out.data_ptr(), _stream(dev))
    if rc:
        raise VdcError(rc, "group_norm_silu_fwd")
    return out


def group_norm_silu_workspace_bytes(S: int, C: int, groups: int) -> int:
    """Workspace bytes of group_norm_silu_bwd."""
    return int(load().group_norm_silu_workspace_bytes(S, C, groups))


def group_norm_silu_bwd(x, weight, groups, dy, *, bias=None, z=None, eps=1e-5, workspace=None):
    """Gradients of group_norm_silu_fwd from its inputs: (dx, dweight, dbias,
    dz), None for what was not given, dweight and dbias of the parameters'
    dtypes."""
    S, C, dev, groups, xs, w_code, b_code, zs = _norm_args(x, weight, groups, bias, z)
    dys = _rows(dy, "dy", x.shape, C, dev)
    dx = _out(None, x, xs, x.shape, "dx", dev)
    dz = None if z is None else torch.empty_like(dx)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    lib = load()
    workspace, ws_n = _workspace(lib.group_norm_silu_workspace_bytes(S, C, groups), workspace, dev)
    rc = lib.group_norm_silu_bwd(x.data_ptr(), xs, weight.data_ptr(), w_code, _ptr(bias), b_code,
                                 _ptr(z), zs, dy.data_ptr(), dys, S, C, groups, eps, dx.data_ptr(),
                                 dw.data_ptr(), _ptr(db), _ptr(dz), workspace.data_ptr(), ws_n,
                                 _stream(dev))
    if rc:
        raise VdcError(rc, "group_norm_silu_bwd")
    return dx, dw, db, dz
