"""What needs no GPU: the refusals of the recurrent layer's entry points (every
call fails before anything is enqueued; its pointers are fake device addresses
that are never dereferenced), the binding's checks, and the 64-bit definitions
the GPU tests compare with, held to torch's gradients, to differences and to a
search over all codes."""
import ctypes
import os

import pytest
import torch

import layer_ref as L
from layer_cases import norm_inputs, recur_inputs

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = range(5)
F32, BF16 = 0, 1
FWD, BWD = 0, 1


def at(i):
    """A fake device address, far from the others."""
    return 0x7E0000000000 + i * 0x10000000000 // 16


@pytest.fixture(scope="module")
def lib():
    from varlen_depthwise_causal_amd import _build, _lib
    if not os.path.exists(_build.LIBRARY):
        _build.build()
    return _lib.load()


# ---------------------------------------------- gated linear recurrence --

def recur(**change):
    from varlen_depthwise_causal_amd._lib import VdcRecurrence
    k = dict(S=100, C=64, x=at(0), r=at(1), i=at(2), z=at(3), x_stride=64, r_stride=128, i_stride=128, z_stride=64,
             decay=at(4), decay_dtype=F32, scale=8.0, cu_seqlens=at(5), num_docs=3, state=at(6), slots=3)
    k.update(change)
    return VdcRecurrence(**{n: v for n, v in k.items() if v is not None})


RECUR_BAD = [({"C": 0}, EINVAL), ({"C": 2 ** 20 + 1}, EINVAL), ({"S": -1}, EINVAL), ({"S": 2 ** 31 - 4095}, EINVAL),
             ({"x_stride": 63}, EINVAL), ({"r_stride": 63}, EINVAL), ({"i_stride": 2 ** 25 + 1}, EINVAL),
             ({"z_stride": 0}, EINVAL), ({"x": None}, EINVAL), ({"r": None}, EINVAL), ({"i": None}, EINVAL),
             ({"decay": None}, EINVAL), ({"scale": -1.0}, EINVAL), ({"scale": float("nan")}, EINVAL),
             ({"scale": float("inf")}, EINVAL), ({"decay_dtype": 2}, EDTYPE), ({"x": at(0) + 1}, EALIGN),
             ({"r": at(1) + 1}, EALIGN), ({"i": at(2) + 1}, EALIGN), ({"z": at(3) + 1}, EALIGN),
             ({"decay": at(4) + 2}, EALIGN)]
PROMPT_BAD = [({"num_docs": 0}, EINVAL), ({"num_docs": -1}, EINVAL), ({"num_docs": 2 ** 31 - 4095}, EINVAL),
              ({"cu_seqlens": None}, EINVAL),
              ({"cu_seqlens": at(5) + 2}, EALIGN)]
STATE_BAD = [({"slots": 2}, EINVAL), ({"slots": -1}, EINVAL), ({"state": at(6) + 2}, EALIGN),
             ({"state": at(0)}, EINVAL), ({"state": at(4)}, EINVAL), ({"state_index": at(6)}, EINVAL),
             ({"state_index": at(7) + 1}, EALIGN)]


def fwd(lib, y=at(20), keep=None, ws=at(21), wsn=1 << 40, **change):
    return lib.gated_recurrence_fwd(ctypes.byref(recur(**change)), y, keep, ws, wsn, None)


def bwd(lib, dy=at(10), dys=64, keep=at(11), dx=at(12), dr=at(13), di=at(14), dd=at(15), dz=at(16), ws=at(21),
        wsn=1 << 40, **change):
    change.setdefault("state", None)
    return lib.gated_recurrence_bwd(ctypes.byref(recur(**change)), dy, dys, keep, dx, dr, di, dd, dz, ws, wsn, None)


@pytest.mark.parametrize("bad,code", RECUR_BAD + PROMPT_BAD + STATE_BAD + [
    ({"y": None}, EINVAL), ({"y": at(20) + 1}, EALIGN), ({"y": at(0)}, EINVAL), ({"y": at(6)}, EINVAL),
    ({"keep": at(22)}, EINVAL), ({"keep": at(22) + 2, "state": None}, EALIGN), ({"keep": at(20), "state": None}, EINVAL),
    ({"keep": at(1), "state": None}, EINVAL), ({"y": at(5)}, EINVAL), ({"state": at(5)}, EINVAL)])
def test_gated_recurrence_fwd_refuses(lib, bad, code):
    assert fwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", RECUR_BAD + PROMPT_BAD + [
    ({"state": at(6)}, EINVAL), ({"dy": None}, EINVAL), ({"dys": 63}, EINVAL), ({"keep": None}, EINVAL),
    ({"dx": None}, EINVAL), ({"dr": None}, EINVAL), ({"di": None}, EINVAL), ({"dd": None}, EINVAL),
    ({"dz": None}, EINVAL), ({"z": None}, EINVAL), ({"dd": at(15) + 2}, EALIGN), ({"dx": at(12) + 1}, EALIGN),
    ({"keep": at(11) + 2}, EALIGN), ({"dx": at(13)}, EINVAL), ({"dx": at(10)}, EINVAL), ({"di": at(11)}, EINVAL),
    ({"dd": at(4)}, EINVAL), ({"ws": at(10)}, EINVAL), ({"ws": at(16)}, EINVAL), ({"wsn": 8}, EWORKSPACE),
    ({"ws": None}, EWORKSPACE), ({"ws": at(21) + 4}, EALIGN)])
def test_gated_recurrence_bwd_refuses(lib, bad, code):
    assert bwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", RECUR_BAD + STATE_BAD + [({"state": None}, EINVAL), ({"S": 4}, EINVAL),
                                                             ({"y": None}, EINVAL), ({"y": at(3)}, EINVAL)])
def test_gated_recurrence_update_refuses(lib, bad, code):
    k = {"S": 3, **bad}
    y = k.pop("y", at(20))
    assert lib.gated_recurrence_update(ctypes.byref(recur(**k)), y, None) == code


def test_gated_recurrence_sizes(lib):
    assert [lib.gated_recurrence_keep_rows(S) for S in (-1, 0, 1, 64, 65, 2 ** 31)] == [0, 0, 1, 1, 2, 0]
    for S, C in ((-1, 8), (8, 0), (8, 2 ** 20 + 1), (0, 8), (2 ** 30, 2 ** 20)):
        assert lib.gated_recurrence_workspace_bytes(BWD, S, C) == 0
        assert lib.gated_recurrence_workspace_bytes(FWD, S, C) == 0
    assert lib.gated_recurrence_workspace_bytes(7, 8, 8) == 0
    assert lib.gated_recurrence_workspace_bytes(BWD, 8, 8) > 0
    # 2^23 tiles of 64 tokens and 64 channels or more
    wide = dict(C=2 ** 20, x_stride=2 ** 20, r_stride=2 ** 20, i_stride=2 ** 20, z_stride=2 ** 20, state=None)
    assert fwd(lib, S=65536, **wide) == EINVAL and bwd(lib, S=65536, dys=2 ** 20, **wide) == EINVAL


# ------------------------------------------------------------ layer norm --

def norm_fwd(lib, x=at(0), xs=64, res=at(1), rs=64, w=at(2), wd=F32, b=at(3), bd=F32, S=10, C=64, eps=1e-5, y=at(4),
             st=at(5)):
    return lib.layer_norm_fwd(x, xs, res, rs, w, wd, b, bd, S, C, eps, y, st, None)


def norm_bwd(lib, x=at(0), xs=64, w=at(2), wd=F32, dy=at(6), dys=64, ds=at(7), dss=64, S=10, C=64, eps=1e-5,
             dx=at(8), dw=at(9), db=at(10), bd=F32, ws=at(11), wsn=1 << 30):
    return lib.layer_norm_bwd(x, xs, w, wd, dy, dys, ds, dss, S, C, eps, dx, dw, db, bd, ws, wsn, None)


NORM_BAD = [({"C": 0}, EINVAL), ({"C": 16385}, EINVAL), ({"S": -1}, EINVAL), ({"xs": 63}, EINVAL), ({"x": None}, EINVAL),
            ({"w": None}, EINVAL), ({"eps": -1.0}, EINVAL), ({"eps": float("nan")}, EINVAL), ({"wd": 5}, EDTYPE),
            ({"bd": 5}, EDTYPE), ({"x": at(0) + 1}, EALIGN), ({"w": at(2) + 2}, EALIGN), ({"S": 2 ** 31}, EINVAL)]


@pytest.mark.parametrize("bad,code", NORM_BAD + [
    ({"rs": 63}, EINVAL), ({"res": None}, EINVAL), ({"st": None}, EINVAL), ({"y": None}, EINVAL), ({"y": at(0)}, EINVAL),
    ({"y": at(5)}, EINVAL), ({"st": at(1)}, EINVAL), ({"st": at(0)}, EINVAL), ({"y": at(4) + 1}, EALIGN),
    ({"b": at(3) + 2}, EALIGN), ({"res": at(1) + 1}, EALIGN), ({"y": at(3)}, EINVAL)])
def test_layer_norm_fwd_refuses(lib, bad, code):
    assert norm_fwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", NORM_BAD + [
    ({"dys": 63}, EINVAL), ({"dss": 63}, EINVAL), ({"dy": None}, EINVAL), ({"dx": None}, EINVAL), ({"dw": None}, EINVAL),
    ({"dx": at(6)}, EINVAL), ({"dx": at(7)}, EINVAL), ({"dw": at(2)}, EINVAL), ({"dw": at(10)}, EINVAL),
    ({"db": at(10) + 2}, EALIGN), ({"dy": at(6) + 1}, EALIGN), ({"ds": at(7) + 1}, EALIGN), ({"wsn": 8}, EWORKSPACE),
    ({"ws": None}, EWORKSPACE), ({"ws": at(11) + 8}, EALIGN), ({"ws": at(6)}, EINVAL)])
def test_layer_norm_bwd_refuses(lib, bad, code):
    assert norm_bwd(lib, **bad) == code


# ------------------------------------------------------ states put aside --

def quantize(lib, state=at(0), dtype=F32, slots=8, E=200, si=at(1), codes=at(2), code=0, scales=at(3), pool=9,
             pi=at(4), rows=5):
    return lib.state_quantize(state, dtype, slots, E, si, codes, code, scales, pool, pi, rows, None)


def dequantize(lib, state=at(0), dtype=F32, slots=8, E=200, si=at(1), codes=at(2), code=0, scales=at(3), pool=9,
               pi=at(4), rows=5):
    return lib.state_dequantize(codes, code, scales, pool, pi, state, dtype, slots, E, si, rows, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("bad,want", [
    ({"slots": -1}, EINVAL), ({"pool": -1}, EINVAL), ({"rows": -1}, EINVAL), ({"E": 0}, EINVAL),
    ({"E": 2 ** 28 + 1}, EINVAL), ({"rows": 2 ** 24}, EINVAL), ({"dtype": 2}, EDTYPE), ({"code": 2}, EDTYPE),
    ({"si": None, "slots": 4}, EINVAL), ({"pi": None, "pool": 4}, EINVAL), ({"state": None}, EINVAL),
    ({"codes": None}, EINVAL), ({"scales": None}, EINVAL), ({"state": at(0) + 2}, EALIGN), ({"scales": at(3) + 2}, EALIGN),
    ({"si": at(1) + 2}, EALIGN), ({"pi": at(4) + 1}, EALIGN), ({"codes": at(0)}, EINVAL), ({"codes": at(3)}, EINVAL),
    ({"scales": at(0) + 64}, EINVAL), ({"si": at(2)}, EINVAL), ({"pi": at(0)}, EINVAL)])
def test_states_put_aside_refuses(lib, call, bad, want):
    assert call(lib, **bad) == want


def test_nothing_to_do(lib):
    n = lib.conv1d_launch_count()
    assert fwd(lib, S=0, num_docs=1, state=None) == OK and fwd(lib, S=0, num_docs=0) == OK
    assert lib.gated_recurrence_update(ctypes.byref(recur(S=0)), at(20), None) == OK
    assert norm_fwd(lib, S=0) == OK
    for call in (quantize, dequantize):
        assert call(lib, rows=0) == OK and call(lib, slots=0) == OK and call(lib, pool=0) == OK
    assert lib.conv1d_launch_count() == n


# ---------------------------------------------------- the binding's checks --

def test_the_binding_refuses_what_is_no_device_tensor():
    import varlen_depthwise_causal_amd as vdc
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w, cu = torch.zeros(8), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        vdc.gated_recurrence_fwd(x, x, x, w, cu)
    with pytest.raises(ValueError, match="device"):
        vdc.layer_norm_fwd(x, w)
    with pytest.raises(TypeError, match="bfloat16"):
        vdc.layer_norm_fwd(x.float(), w)
    with pytest.raises(ValueError, match="state"):
        vdc.gated_recurrence_update(x, x, x, w, None)
    state, codes, scales = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="device"):
        vdc.state_quantize(state, codes, scales)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        vdc.state_quantize(state.double(), codes, scales)


def test_the_binding_is_required(monkeypatch):
    """No fallback where the compiled calls are missing."""
    from varlen_depthwise_causal_amd import layer
    with pytest.raises(AttributeError):
        layer._call.no_such_call
    monkeypatch.setattr(layer, "BINDING", "/nowhere/_vdc_torch.so")
    with pytest.raises(ImportError, match="not built"):
        layer._Binding().norm_fwd


def test_the_binding_refuses_arguments_of_other_types():
    import varlen_depthwise_causal_amd as vdc
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: vdc.layer_norm_fwd(None, x), lambda: vdc.layer_norm_fwd(x, 3),
                 lambda: vdc.gated_recurrence_fwd(x, x, x, [1.0], None),
                 lambda: vdc.state_quantize("cache", x, x), lambda: vdc.layer_norm_fwd(x, torch.zeros(8), eps="small")):
        with pytest.raises((TypeError, ValueError)):
            call()


# ------------------------------------------------------- the definitions --

def test_recurrence_against_torch_gradients():
    k, docs, cu = recur_inputs(1, [5, 0, 9, 1], 6, device="cpu")
    v = {n: t.double().requires_grad_() for n, t in k.items()}
    u = 16 * torch.nn.functional.softplus(v["decay"]) * torch.sigmoid(v["r"])
    a, m, ys = torch.exp(-u / 2), (-torch.expm1(-u)).sqrt(), []
    for lo, hi in docs:
        h = torch.zeros(6, dtype=torch.float64)
        for t in range(lo, hi):
            h = a[t] * h + m[t] * torch.sigmoid(v["i"][t]) * v["x"][t]
            ys.append(h)
    y = torch.stack(ys) * torch.nn.functional.silu(v["z"])
    dy = torch.randn(15, 6, generator=torch.Generator().manual_seed(2)).double()
    y.backward(dy)
    ref = L.Recurrence(k["x"], k["r"], k["i"], k["decay"], docs, k["z"])
    assert torch.allclose(ref.y, y, rtol=1e-12, atol=1e-14)
    for n, (g, bound) in ref.grads(dy).items():
        assert torch.allclose(g, v[n[1:]].grad, rtol=1e-11, atol=1e-13), n
        assert bool((bound >= 0).all()) and float((bound / g.abs().clamp(min=1e-3)).max()) < 1e-2


def test_recurrence_against_differences():
    k, docs, _ = recur_inputs(3, [7, 4], 5, device="cpu")
    k = {n: t.double() for n, t in k.items()}
    dy = torch.randn(11, 5, generator=torch.Generator().manual_seed(4)).double()
    grads = L.Recurrence(k["x"], k["r"], k["i"], k["decay"], docs, k["z"]).grads(dy)
    for n in k:
        for j in (0, k[n].numel() // 2, k[n].numel() - 1):
            f = []
            for e in (1e-5, -1e-5):
                q = dict(k)
                q[n] = k[n].clone()
                q[n].view(-1)[j] += e
                f.append(float((L.Recurrence(q["x"], q["r"], q["i"], q["decay"], docs, q["z"]).y * dy).sum()))
            got = float(grads["d" + n][0].reshape(-1)[j])
            assert abs((f[0] - f[1]) / 2e-5 - got) <= 1e-7 * max(1.0, abs(got)), n


def test_layer_norm_against_torch_gradients():
    k = norm_inputs(5, 7, 33, device="cpu")
    s = (k["x"].float() + k["residual"].float()).bfloat16()
    v = {n: t.double().requires_grad_() for n, t in (("s", s), ("w", k["weight"]), ("b", k["bias"]))}
    y = torch.nn.functional.layer_norm(v["s"], (33,), v["w"], v["b"], 1e-5)
    torch.autograd.backward([y, v["s"]], [k["dy"].double(), k["dstream"].double()])
    ref = L.LayerNorm(s, k["weight"], k["bias"])
    assert torch.allclose(ref.y, y, rtol=1e-12, atol=1e-13)
    for n, (g, _) in ref.grads(k["dy"], k["dstream"]).items():
        assert torch.allclose(g, v[{"dx": "s", "dweight": "w", "dbias": "b"}[n]].grad, rtol=1e-10, atol=1e-12), n


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_codes_against_a_search(code):
    g = torch.Generator().manual_seed(6)
    v = torch.randn(200, generator=g).double()
    v[3], v[64:128] = 0.0, 0.0
    q, scale = L.put_aside(v, code)
    mags = L.codes_of(code)
    every = torch.cat([-mags.flip(0), mags])
    for j in range(200):
        s = float(scale[j // 64].double())
        if s == 0:
            assert float(q[j]) == 0
            continue
        assert abs(float(q[j]) - float(v[j]) / s) <= float((every - v[j] / s).abs().min()) + 1e-15
    assert torch.equal(L.take_back(q, scale, torch.float32), q.float() * scale.repeat_interleave(64)[:200])
