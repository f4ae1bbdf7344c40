"""The state space layer's autograd wrappers: the same bits as the direct
calls, gradients in the parameters' dtypes and only where they are needed, any
layout of the incoming gradient, and the scan's gradients against differences
of the kernel's own outputs."""
import pytest
import torch

from ssm_cases import Maker, scan_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _leaf(t):
    return t.detach().clone().requires_grad_()


def _scan(seed=201, params=torch.float32):
    k, _, cu = scan_inputs(seed, [40, 0, 170, 1], 136, 16, 2, device=DEV, params=params)
    return k, cu, Maker(seed + 1, DEV).normal(211, 136)


@pytest.mark.parametrize("params", [torch.float32, torch.bfloat16])
def test_selective_scan_matches_direct_calls(params):
    import varlen_depthwise_causal_amd as vdc
    from varlen_depthwise_causal_amd.autograd import selective_scan
    k, cu, dy = _scan(params=params)
    rest = {n: k[n] for n in ("D", "z", "dt_bias")}
    head = [k[n] for n in ("x", "dt", "A", "B", "C")]
    y0 = vdc.selective_scan_fwd(*head, cu, **rest)
    want = vdc.selective_scan_bwd(*head, cu, dy, **rest)
    # dense, another layout, FP32 with the same values
    for g in (dy, dy.t().contiguous().t(), dy.float()):
        v = {n: _leaf(k[n]) for n in NAMES}
        y = selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], cu, D=v["D"], z=v["z"], dt_bias=v["dt_bias"])
        assert torch.equal(y, y0)
        torch.autograd.backward(y, grad_tensors=g)
        for n, w in zip(NAMES, want):
            assert v[n].grad.dtype == v[n].dtype and torch.equal(v[n].grad, w), n


def test_selective_scan_only_what_is_needed():
    from varlen_depthwise_causal_amd.autograd import selective_scan
    k, cu, dy = _scan()
    A = _leaf(k["A"])
    y = selective_scan(k["x"], k["dt"], A, k["B"], k["C"], cu)
    assert y.requires_grad
    y.backward(dy)
    assert A.grad is not None and bool(torch.isfinite(A.grad).all())
    with pytest.raises(RuntimeError):  # once only
        (g,) = torch.autograd.grad(selective_scan(k["x"], k["dt"], A, k["B"], k["C"], cu), A, dy, create_graph=True)
        g.sum().backward()


def test_selective_scan_expanded_gradient_and_flat_states():
    """The gradient of a sum has no strides; B and C may come without groups."""
    import varlen_depthwise_causal_amd as vdc
    from varlen_depthwise_causal_amd.autograd import selective_scan
    k, _, cu = scan_inputs(211, [30, 60], 72, 8, 1, device=DEV)
    B, C = _leaf(k["B"][:, 0]), _leaf(k["C"][:, 0])
    selective_scan(k["x"], k["dt"], k["A"], B, C, cu).sum().backward()
    want = vdc.selective_scan_bwd(k["x"], k["dt"], k["A"], k["B"], k["C"], cu, torch.ones_like(k["x"]))
    assert torch.equal(B.grad, want[3][:, 0]) and torch.equal(C.grad, want[4][:, 0])


def test_selective_scan_against_differences_of_its_outputs():
    """A step e in A moves L = sum(w y) by e dL/dA, up to e^2 / 2 of its
    curvature and the rounding of y: every output is off by at most 2^-8 of
    itself, which adds over outputs of either sign like their root sum of
    squares, taken eight times."""
    from varlen_depthwise_causal_amd.autograd import selective_scan
    k, cu, dy = _scan(221)
    A = _leaf(k["A"])
    run = lambda a: selective_scan(k["x"], k["dt"], a, k["B"], k["C"], cu, D=k["D"], z=k["z"],  # noqa: E731
                                   dt_bias=k["dt_bias"])
    y = run(A)
    y.backward(dy)
    y = y.detach()
    way = -k["A"] * 0.25  # every decay slower or faster by a quarter
    up, down = run(k["A"] + way).double(), run(k["A"] - way).double()
    got = ((up - down) / 2 * dy.double()).sum()
    want = (A.grad.double() * way.double()).sum()
    noise = 8 * 2.0 ** -8 * float(((y.double() * dy.double()) ** 2).sum().sqrt())
    # third-order term of a central difference: bounded through the second
    # differences' change between the step and half of it
    half = ((run(k["A"] + way / 2).double() - run(k["A"] - way / 2).double()) * dy.double()).sum()
    curve = 2 * float((got - half).abs())
    off = abs(float(got - want))
    print("difference %.5g gradient %.5g off %.3g allowed %.3g" % (float(got), float(want), off, noise + curve))
    assert off <= noise + curve


@pytest.mark.parametrize("gate,bias,params", [(True, True, torch.float32), (False, True, torch.bfloat16),
                                              (True, False, torch.float32)])
def test_group_norm_silu_matches_direct_calls(gate, bias, params):
    import varlen_depthwise_causal_amd as vdc
    from varlen_depthwise_causal_amd.autograd import group_norm_silu
    m = Maker(231, DEV)
    x, dy = m.normal(50, 320), m.normal(50, 320)
    z = m.normal(50, 320) if gate else None
    w, b = m.uniform(320, lo=0.5, hi=1.5, dtype=params), m.normal(320, dtype=params) if bias else None
    y0 = vdc.group_norm_silu_fwd(x, w, 5, bias=b, z=z, eps=1e-3)
    want = vdc.group_norm_silu_bwd(x, w, 5, dy, bias=b, z=z, eps=1e-3)
    for g in (dy, dy.t().contiguous().t(), dy.float()):
        xl, wl = _leaf(x), _leaf(w)
        bl, zl = (_leaf(b) if bias else None), (_leaf(z) if gate else None)
        y = group_norm_silu(xl, wl, 5, bias=bl, z=zl, eps=1e-3)
        assert torch.equal(y, y0)
        torch.autograd.backward(y, grad_tensors=g)
        for t, w_ in zip((xl, wl, bl, zl), want):
            assert (t is None) == (w_ is None)
            if t is not None:
                assert t.grad.dtype == t.dtype and torch.equal(t.grad, w_)


def test_group_norm_silu_only_what_is_needed():
    from varlen_depthwise_causal_amd.autograd import group_norm_silu
    m = Maker(241, DEV)
    x, z, w = m.normal(9, 64), _leaf(m.normal(9, 64)), m.normal(64, dtype=torch.float32)
    group_norm_silu(x, w, 4, z=z).sum().backward()
    assert z.grad is not None and x.grad is None and w.grad is None


def test_training_step_in_a_graph():
    """A forward and backward pass of scan and norm captured once and replayed
    on other inputs gives the eager bits each time."""
    from varlen_depthwise_causal_amd.autograd import group_norm_silu, selective_scan
    sets = [_scan(seed) for seed in (251, 261, 271)]
    w = Maker(252, DEV).uniform(136, lo=0.5, hi=1.5)

    def step(v, cu, dy):
        y = selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], cu, D=v["D"], dt_bias=v["dt_bias"])
        out = group_norm_silu(y, w, 17, z=v["z"])
        return [out.detach()] + list(torch.autograd.grad(out, [v[n] for n in NAMES], dy))

    eager = [[t.clone() for t in step({n: _leaf(k[n]) for n in NAMES}, cu, dy)] for k, cu, dy in sets]
    k, cu, dy = sets[0]
    hold, hdy = {n: _leaf(k[n]) for n in NAMES}, dy.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(hold, cu, hdy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(hold, cu, hdy)
    for rep in (0, 1, 2, 0):
        k, _, dy = sets[rep]
        with torch.no_grad():
            for n in NAMES:
                hold[n].copy_(k[n])
        hdy.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, eager[rep])):
            assert torch.equal(a, b), "replay of set %d: output %d" % (rep, i)
        step({n: _leaf(k[n]) for n in NAMES}, cu, dy)
