"""What needs no GPU: the refusals of the state space layer's entry points
(every call fails before anything is enqueued; its pointers are fake device
addresses that are never dereferenced), and the 64-bit definitions the GPU
tests compare with, held to torch's gradients and to differences."""
import ctypes
import os

import pytest
import torch

import ssm_ref as R
from ssm_cases import Maker, scan_inputs

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = range(5)
F32, BF16 = 0, 1
FWD, BWD = 0, 1
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


def at(i):
    """A fake device address, far from the others."""
    return 0x7E0000000000 + i * 0x10000000000 // 16


@pytest.fixture(scope="module")
def lib():
    from varlen_depthwise_causal_amd import _build, _lib
    if not os.path.exists(_build.LIBRARY):
        _build.build()
    return _lib.load()


def prefill(lib, x=at(0), w=at(1), wd=F32, b=at(2), bd=F32, cu=at(3), D=4, S=100, C=64, st=at(4), slots=4,
            ix=None, resume=None, y=at(5)):
    return lib.conv1d_prefill(x, w, wd, b, bd, cu, D, S, C, st, slots, ix, resume, y, None)


@pytest.mark.parametrize("bad,code", [
    ({"C": 63}, EINVAL), ({"C": 0}, EINVAL), ({"S": -1}, EINVAL), ({"D": -1}, EINVAL), ({"D": 0}, EINVAL),
    ({"slots": 3}, EINVAL), ({"slots": -1}, EINVAL), ({"st": None}, EINVAL), ({"x": None}, EINVAL),
    ({"w": None}, EINVAL), ({"cu": None}, EINVAL), ({"y": None}, EINVAL), ({"wd": 2}, EDTYPE),
    ({"bd": 7}, EDTYPE), ({"st": at(4) + 8}, EALIGN), ({"x": at(0) + 2}, EALIGN), ({"ix": at(6) + 2}, EALIGN),
    ({"st": at(0)}, EINVAL), ({"y": at(4)}, EINVAL), ({"y": at(0)}, EINVAL)])
def test_conv1d_prefill_refuses(lib, bad, code):
    assert prefill(lib, **bad) == code


def test_nothing_to_do(lib):
    n = lib.conv1d_launch_count()
    assert prefill(lib, S=0, D=0) == OK
    assert update(lib, rows=0) == OK
    assert fwd(lib, S=0, num_docs=1, state=None) == OK
    assert lib.selective_update(ctypes.byref(scan(S=0)), at(20), None) == OK
    assert norm_fwd(lib, S=0) == OK
    assert lib.conv1d_launch_count() == n


def update(lib, x=at(0), xs=64, w=at(1), wd=F32, b=at(2), bd=F32, rows=3, C=64, st=at(4), slots=4, ix=None,
           y=at(5)):
    return lib.conv1d_update(x, xs, w, wd, b, bd, rows, C, st, slots, ix, y, None)


@pytest.mark.parametrize("bad,code", [
    ({"C": 60}, EINVAL), ({"rows": -1}, EINVAL), ({"rows": 5}, EINVAL), ({"xs": 56}, EINVAL),
    ({"xs": 68}, EINVAL), ({"x": None}, EINVAL), ({"y": None}, EINVAL), ({"wd": -1}, EDTYPE),
    ({"x": at(0) + 8}, EALIGN), ({"y": at(4)}, EINVAL), ({"st": at(1)}, EINVAL), ({"st": at(4) + 2}, EALIGN)])
def test_conv1d_update_refuses(lib, bad, code):
    assert update(lib, **bad) == code


def scan(**change):
    from varlen_depthwise_causal_amd._lib import VdcScan
    k = dict(S=100, C=64, N=16, groups=2, x=at(0), dt=at(1), z=at(2), B=at(3), Cm=at(4), x_stride=64, dt_stride=64,
             z_stride=128, B_stride=96, C_stride=96, A=at(5), D=at(6), dt_bias=at(7), A_dtype=F32, D_dtype=F32,
             dt_bias_dtype=F32, dt_softplus=1, cu_seqlens=at(8), num_docs=3, state=at(9), slots=3)
    k.update(change)
    return VdcScan(**{n: v for n, v in k.items() if v is not None})


SCAN_BAD = [({"C": 0}, EINVAL), ({"C": 2 ** 20 + 1}, EINVAL), ({"N": 0}, EINVAL), ({"N": 65}, EINVAL),
            ({"groups": 3}, EINVAL), ({"groups": 0}, EINVAL), ({"S": -1}, EINVAL), ({"x_stride": 63}, EINVAL),
            ({"z_stride": 10}, EINVAL), ({"B_stride": 31}, EINVAL), ({"C_stride": 2 ** 31 + 1}, EINVAL),
            ({"x": None}, EINVAL), ({"dt": None}, EINVAL), ({"B": None}, EINVAL), ({"A": None}, EINVAL),
            ({"A_dtype": 3}, EDTYPE), ({"D_dtype": -1}, EDTYPE), ({"dt_bias_dtype": 2}, EDTYPE),
            ({"x": at(0) + 1}, EALIGN), ({"A": at(5) + 2}, EALIGN), ({"z": at(2) + 1}, EALIGN)]
PROMPT_BAD = [({"num_docs": 0}, EINVAL), ({"num_docs": -1}, EINVAL), ({"cu_seqlens": None}, EINVAL)]
STATE_BAD = [({"slots": 2}, EINVAL), ({"slots": -1}, EINVAL), ({"state": at(9) + 2}, EALIGN),
             ({"state": at(0)}, EINVAL), ({"state": at(5)}, EINVAL), ({"state_index": at(9)}, EINVAL)]


def fwd(lib, y=at(20), ws=at(21), wsn=1 << 40, **change):
    return lib.selective_scan_fwd(ctypes.byref(scan(**change)), y, ws, wsn, None)


def bwd(lib, dy=at(10), dys=64, dx=at(11), ddt=at(12), dz=at(13), dB=at(14), dC=at(15), dA=at(16), dD=at(17),
        db=at(18), ws=at(21), wsn=1 << 40, **change):
    change.setdefault("state", None)
    return lib.selective_scan_bwd(ctypes.byref(scan(**change)), dy, dys, dx, ddt, dz, dB, dC, dA, dD, db, ws, wsn,
                                  None)


@pytest.mark.parametrize("bad,code", SCAN_BAD + PROMPT_BAD + STATE_BAD + [
    ({"y": None}, EINVAL), ({"y": at(20) + 1}, EALIGN), ({"y": at(0)}, EINVAL), ({"y": at(9)}, EINVAL),
    ({"S": 5000, "wsn": 8}, EWORKSPACE), ({"S": 5000, "ws": None}, EWORKSPACE),
    ({"S": 5000, "ws": at(21) + 4}, EALIGN), ({"S": 5000, "ws": at(9)}, EINVAL)])
def test_selective_scan_fwd_refuses(lib, bad, code):
    assert fwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", SCAN_BAD + PROMPT_BAD + [
    ({"state": at(9)}, EINVAL), ({"dy": None}, EINVAL), ({"dys": 63}, EINVAL), ({"dx": None}, EINVAL),
    ({"ddt": None}, EINVAL), ({"dB": None}, EINVAL), ({"dC": None}, EINVAL), ({"dA": None}, EINVAL),
    ({"dz": None}, EINVAL), ({"z": None}, EINVAL), ({"dD": None}, EINVAL), ({"D": None}, EINVAL),
    ({"db": None}, EINVAL), ({"dt_bias": None}, EINVAL), ({"dA": at(16) + 2}, EALIGN), ({"dx": at(11) + 1}, EALIGN),
    ({"dx": at(12)}, EINVAL), ({"dx": at(10)}, EINVAL), ({"dA": at(5)}, EINVAL), ({"ws": at(10)}, EINVAL),
    ({"wsn": 8}, EWORKSPACE), ({"ws": None}, EWORKSPACE)])
def test_selective_scan_bwd_refuses(lib, bad, code):
    assert bwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", [b for b in SCAN_BAD if "z_stride" not in b[0]] + STATE_BAD + [
    ({"state": None}, EINVAL), ({"S": 4}, EINVAL)])
def test_selective_update_refuses(lib, bad, code):
    k = {"S": 3, **bad}
    assert lib.selective_update(ctypes.byref(scan(**k)), at(20), None) == code


def norm_fwd(lib, x=at(0), xs=64, w=at(1), wd=F32, b=at(2), bd=F32, z=at(3), zs=64, S=10, C=64, G=4, eps=1e-5,
             y=at(4)):
    return lib.group_norm_silu_fwd(x, xs, w, wd, b, bd, z, zs, S, C, G, eps, y, None)


def norm_bwd(lib, x=at(0), xs=64, w=at(1), wd=F32, b=at(2), bd=F32, z=at(3), zs=64, dy=at(5), dys=64, S=10, C=64,
             G=4, eps=1e-5, dx=at(6), dw=at(7), db=at(8), dz=at(9), ws=at(10), wsn=1 << 30):
    return lib.group_norm_silu_bwd(x, xs, w, wd, b, bd, z, zs, dy, dys, S, C, G, eps, dx, dw, db, dz, ws, wsn, None)


NORM_BAD = [({"G": 3}, EINVAL), ({"G": 0}, EINVAL), ({"C": 0}, EINVAL), ({"S": -1}, EINVAL), ({"xs": 63}, EINVAL),
            ({"zs": 1}, EINVAL), ({"x": None}, EINVAL), ({"w": None}, EINVAL), ({"eps": -1.0}, EINVAL),
            ({"eps": float("nan")}, EINVAL), ({"wd": 5}, EDTYPE), ({"bd": 5}, EDTYPE), ({"x": at(0) + 1}, EALIGN),
            ({"w": at(1) + 2}, EALIGN), ({"C": 32768, "G": 1, "xs": 32768, "zs": 32768, "dys": 32768}, EINVAL)]


@pytest.mark.parametrize("bad,code", [b for b in NORM_BAD if "dys" not in b[0]] + [
    ({"C": 32768, "G": 1, "xs": 32768, "zs": 32768}, EINVAL), ({"y": None}, EINVAL), ({"y": at(0)}, EINVAL),
    ({"y": at(3)}, EINVAL), ({"y": at(4) + 1}, EALIGN)])
def test_group_norm_silu_fwd_refuses(lib, bad, code):
    assert norm_fwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", NORM_BAD + [
    ({"dy": None}, EINVAL), ({"dx": None}, EINVAL), ({"dw": None}, EINVAL), ({"db": None}, EINVAL),
    ({"b": None}, EINVAL), ({"dz": None}, EINVAL), ({"z": None}, EINVAL), ({"dys": 8}, EINVAL),
    ({"dx": at(5)}, EINVAL), ({"dz": at(6)}, EINVAL), ({"wsn": 4}, EWORKSPACE), ({"ws": None}, EWORKSPACE),
    ({"ws": at(10) + 8}, EALIGN), ({"ws": at(6)}, EINVAL)])
def test_group_norm_silu_bwd_refuses(lib, bad, code):
    assert norm_bwd(lib, **bad) == code


def test_workspace_sizes(lib):
    w = lib.selective_scan_workspace_bytes
    assert w(FWD, 1, 64, 16, 1) == 0 and w(BWD, 1, 64, 16, 1) > 0
    for bad in ((2, 10, 64, 16, 1), (FWD, -1, 64, 16, 1), (FWD, 10, 64, 65, 1), (BWD, 10, 64, 16, 5)):
        assert w(*bad) == 0
    assert w(BWD, 0, 64, 16, 1) == 0
    assert lib.group_norm_silu_workspace_bytes(0, 64, 4) == 0
    assert lib.group_norm_silu_workspace_bytes(10, 64, 4) > 0


def test_host_tensors_and_shapes_are_refused():
    import varlen_depthwise_causal_amd as vdc
    k, _, cu = scan_inputs(1, [5], 8, 4, device="cpu")
    with pytest.raises(ValueError, match="device tensor"):
        vdc.selective_scan_fwd(k["x"], k["dt"], k["A"], k["B"], k["C"], cu)
    with pytest.raises(TypeError, match="bfloat16"):
        vdc.selective_scan_fwd(k["x"].float(), k["dt"], k["A"], k["B"], k["C"], cu)
    with pytest.raises(ValueError, match="rows, C"):
        vdc.selective_scan_fwd(k["x"][0], k["dt"], k["A"], k["B"], k["C"], cu)
    with pytest.raises(ValueError, match="needs a state"):
        vdc.selective_update(k["x"], k["dt"], k["A"], k["B"], k["C"], None)
    with pytest.raises(ValueError, match="groups must divide"):
        vdc.group_norm_silu_fwd(k["x"], k["D"], 3)
    with pytest.raises(ValueError, match="device tensor"):
        vdc.conv1d_update(k["x"], k["x"], k["A"])


# ------------------------------------- the definitions the GPU is held to --

def _scan_by_hand(p, docs):
    S, C = p["x"].shape
    per = C // p["B"].shape[1]
    d = torch.nn.functional.softplus(p["dt"] + p["dt_bias"])
    ys = [None] * S
    for lo, hi in docs:
        h = torch.zeros(C, p["A"].shape[1], dtype=torch.float64)
        for t in range(lo, hi):
            h = torch.exp(d[t][:, None] * p["A"]) * h + (d[t] * p["x"][t])[:, None] * p["B"][t].repeat_interleave(per, 0)
            y = (h * p["C"][t].repeat_interleave(per, 0)).sum(-1) + p["D"] * p["x"][t]
            ys[t] = y * torch.nn.functional.silu(p["z"][t])
    return torch.stack(ys)


def _scan_gradients():
    k, docs, _ = scan_inputs(1, [0, 5, 1, 9], 6, 3, 2, device="cpu")
    r = R.Scan(*(k[n] for n in ("x", "dt", "A", "B", "C")), docs, k["D"], k["z"], k["dt_bias"])
    dy = Maker(2, "cpu").normal(15, 6)
    return k, docs, r, dy, r.grads(dy)


def test_scan_definition_against_torch():
    k, docs, r, dy, g = _scan_gradients()
    p = {n: k[n].double().requires_grad_() for n in NAMES}
    y = _scan_by_hand(p, docs)
    torch.testing.assert_close(r.y, y.detach(), rtol=1e-12, atol=1e-13)
    want = torch.autograd.grad(y, [p[n] for n in NAMES], dy.double())
    for n, t in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), want):
        torch.testing.assert_close(g[n][0], t, rtol=1e-10, atol=1e-12)


def test_scan_definition_against_differences():
    k, docs, _, dy, g = _scan_gradients()
    p = {n: k[n].double() for n in NAMES}
    m = torch.Generator().manual_seed(3)
    for n, name in zip(NAMES, ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")):
        e = torch.randn(p[n].shape, generator=m, dtype=torch.float64)
        f = [float((_scan_by_hand({**p, n: p[n] + s * 1e-5 * e}, docs) * dy.double()).sum()) for s in (1, -1)]
        want = float((g[name][0] * e).sum())
        assert abs((f[0] - f[1]) / 2e-5 - want) <= 1e-6 * (1 + abs(want)), n


@pytest.mark.parametrize("gate", [True, False])
def test_norm_definition_against_torch_and_differences(gate):
    m = Maker(7, "cpu")
    x, z, dy = m.normal(9, 12, mean=0.3), m.normal(9, 12) if gate else None, m.normal(9, 12).double()
    w, b = m.uniform(12, lo=0.5, hi=1.5), m.normal(12, std=0.1, dtype=torch.float32)
    ref = R.Norm(x, w, 3, b, z)
    p = [t.double() for t in (x, w, b)] + ([z.double()] if gate else [])

    def by_hand(x, w, b, z=None):
        v = torch.nn.functional.group_norm(x, 3, w, b, 1e-5)
        return torch.nn.functional.silu(v) if z is None else v * torch.nn.functional.silu(z)

    torch.testing.assert_close(ref.y, by_hand(*p), rtol=1e-12, atol=1e-13)
    g = ref.grads(dy)
    gen = torch.Generator().manual_seed(3)
    for i, name in enumerate(("dx", "dweight", "dbias", "dz")[:len(p)]):
        e = torch.randn(p[i].shape, generator=gen, dtype=torch.float64)
        f = [float((by_hand(*(t + s * 1e-5 * e if j == i else t for j, t in enumerate(p))) * dy).sum()) for s in (1, -1)]
        want = float((g[name][0] * e).sum())
        assert abs((f[0] - f[1]) / 2e-5 - want) <= 1e-6 * (1 + abs(want)), name
