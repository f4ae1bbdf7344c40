"""The recurrent layer's autograd wrappers: the same bits as the direct calls,
gradients in the parameters' dtypes and only where they are needed, any layout
of the incoming gradient, a stream with and without gradients of its own, and
the recurrence's gradients against differences of the kernel's outputs."""
import pytest
import torch

from layer_cases import norm_inputs, recur_inputs
from ssm_cases import Maker

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAMES = ("x", "r", "i", "decay", "z")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _leaf(t):
    return t.detach().clone().requires_grad_()


def _set(seed=301, params=torch.float32):
    k, _, cu = recur_inputs(seed, [40, 0, 170, 1], 136, device=DEV, params=params)
    return k, cu, Maker(seed + 1, DEV).normal(211, 136)


@pytest.mark.parametrize("params", [torch.float32, torch.bfloat16])
def test_gated_recurrence_matches_direct_calls(params):
    import varlen_depthwise_causal_amd as vdc
    from varlen_depthwise_causal_amd.autograd import gated_recurrence
    k, cu, dy = _set(params=params)
    head = [k[n] for n in NAMES[:4]]
    y0, keep = vdc.gated_recurrence_fwd(*head, cu, z=k["z"], scale=5.0, keep=True)
    want = vdc.gated_recurrence_bwd(*head, cu, dy, keep, z=k["z"], scale=5.0)
    for g in (dy, dy.t().contiguous().t(), dy.float()):
        v = {n: _leaf(k[n]) for n in NAMES}
        y = gated_recurrence(v["x"], v["r"], v["i"], v["decay"], cu, v["z"], 5.0)
        assert torch.equal(y, y0)
        torch.autograd.backward(y, grad_tensors=g)
        for n, w in zip(NAMES, want):
            assert v[n].grad.dtype == v[n].dtype and torch.equal(v[n].grad, w), n


def test_gated_recurrence_only_what_is_needed():
    from varlen_depthwise_causal_amd.autograd import gated_recurrence
    k, cu, dy = _set()
    decay = _leaf(k["decay"])
    gated_recurrence(k["x"], k["r"], k["i"], decay, cu).backward(dy)
    assert decay.grad is not None and bool(torch.isfinite(decay.grad).all())
    with pytest.raises(RuntimeError):  # once only
        (g,) = torch.autograd.grad(gated_recurrence(k["x"], k["r"], k["i"], decay, cu), decay, dy, create_graph=True)
        g.sum().backward()
    # one gate for both uses, and the gradient of a sum, which has no strides
    r = _leaf(k["r"])
    gated_recurrence(k["x"], r, r, k["decay"], cu).sum().backward()
    assert r.grad is not None and bool(torch.isfinite(r.grad).all())


@pytest.mark.parametrize("name", NAMES)
def test_gated_recurrence_against_differences_of_its_outputs(name):
    """Sums over the outputs' differences along a direction, whose size goes by
    what FP32 and the outputs' BF16 leave: each output is off by at most 2^-8 of
    itself, which adds over outputs of either sign like their root sum of squares,
    taken eight times, and the third-order term is bounded through half the step."""
    from varlen_depthwise_causal_amd.autograd import gated_recurrence
    k, cu, dy = _set(311)
    v = {n: _leaf(k[n]) for n in NAMES}
    run = lambda q: gated_recurrence(q["x"], q["r"], q["i"], q["decay"], cu, q["z"])  # noqa: E731
    y = run(v)
    y.backward(dy)
    grad = v[name].grad.double()
    # a direction the gradient answers to, in steps that BF16 holds exactly enough
    way = (torch.sign(grad) * (0.25 if name != "decay" else 0.5)).to(k[name].dtype)
    moved = lambda s: (k[name].double() + s * way.double()).to(k[name].dtype)  # noqa: E731
    out = {s: run({**k, name: moved(s)}).double() for s in (1, -1, 0.5, -0.5)}
    step = lambda s: (moved(s).double() - moved(-s).double()) / (2 * s)  # noqa: E731
    got = ((out[1] - out[-1]) / 2 * dy.double()).sum()
    half = ((out[0.5] - out[-0.5]) * dy.double()).sum()
    want = (grad * step(1)).sum()
    noise = 8 * 2.0 ** -8 * float(((y.double() * dy.double()) ** 2).sum().sqrt())
    # the rounded inputs' directions differ between the step and half of it
    curve = 2 * float((got - half).abs()) + 2 * float((grad * (step(1) - step(0.5))).sum().abs())
    off = float((got - want).abs())
    print("%s difference %.5g gradient %.5g off %.3g allowed %.3g" % (name, float(got), float(want), off, noise + curve))
    assert off <= noise + curve


@pytest.mark.parametrize("residual,bias,params", [(True, True, torch.float32), (False, True, torch.bfloat16),
                                                  (True, False, torch.float32), (False, False, torch.float32)])
def test_layer_norm_matches_direct_calls(residual, bias, params):
    import varlen_depthwise_causal_amd as vdc
    from varlen_depthwise_causal_amd.autograd import layer_norm
    k = norm_inputs(321, 50, 320, device=DEV, bias=bias, residual=residual, params=params)
    y0, s0 = vdc.layer_norm_fwd(k["x"], k["weight"], bias=k["bias"], residual=k["residual"], eps=1e-3)
    want = vdc.layer_norm_bwd(s0, k["weight"], k["dy"], bias=k["bias"], dstream=k["dstream"], eps=1e-3)
    for g in (k["dy"], k["dy"].t().contiguous().t(), k["dy"].float()):
        v = {n: _leaf(k[n]) for n in ("x", "weight", "bias", "residual") if k[n] is not None}
        out = layer_norm(v["x"], v["weight"], v.get("bias"), v.get("residual"), 1e-3)
        if residual:
            assert torch.equal(out[0], y0) and torch.equal(out[1], s0)
            torch.autograd.backward(out, grad_tensors=[g, k["dstream"]])
            assert torch.equal(v["residual"].grad, want[0])
        else:
            assert torch.equal(out, y0)
            torch.autograd.backward(out, grad_tensors=g)
        assert torch.equal(v["x"].grad, want[0]) and torch.equal(v["weight"].grad, want[1])
        assert v["weight"].grad.dtype == params
        if bias:
            assert torch.equal(v["bias"].grad, want[2])


def test_layer_norm_with_one_gradient_of_two():
    import varlen_depthwise_causal_amd as vdc
    from varlen_depthwise_causal_amd.autograd import layer_norm
    k = norm_inputs(331, 30, 72, device=DEV)
    x, res, w = _leaf(k["x"]), _leaf(k["residual"]), _leaf(k["weight"])
    y, s = layer_norm(x, w, k["bias"], res)
    y.backward(k["dy"])
    want = vdc.layer_norm_bwd(s.detach(), k["weight"], k["dy"], bias=k["bias"])
    assert torch.equal(x.grad, want[0]) and torch.equal(res.grad, want[0]) and torch.equal(w.grad, want[1])
    x, res, w = _leaf(k["x"]), _leaf(k["residual"]), _leaf(k["weight"])
    layer_norm(x, w, k["bias"], res)[1].backward(k["dstream"])
    assert torch.equal(x.grad, k["dstream"]) and torch.equal(res.grad, k["dstream"]) and w.grad is None
    # only the residual, and an input that is both
    res = _leaf(k["residual"])
    sum(t.sum() for t in layer_norm(k["x"], k["weight"], k["bias"], res)).backward()
    assert res.grad is not None
    both = _leaf(k["x"])
    layer_norm(both, k["weight"], k["bias"], both)[0].backward(k["dy"])
    y2, s2 = vdc.layer_norm_fwd(k["x"], k["weight"], bias=k["bias"], residual=k["x"])
    once = vdc.layer_norm_bwd(s2, k["weight"], k["dy"], bias=k["bias"])[0]
    assert torch.equal(both.grad, once + once)


def test_training_step_in_a_graph():
    """A forward and backward pass of norm, recurrence and norm captured once and
    replayed on other inputs gives the eager bits each time."""
    from varlen_depthwise_causal_amd.autograd import gated_recurrence, layer_norm
    sets = [_set(seed) for seed in (341, 351, 361)]
    w, b = Maker(342, DEV).uniform(136, lo=0.5, hi=1.5), Maker(343, DEV).normal(136, dtype=torch.float32)

    def step(v, cu, dy):
        y = layer_norm(v["x"], w, b)
        y = gated_recurrence(y, v["r"], v["i"], v["decay"], cu, v["z"])
        out, _ = layer_norm(y, w, b, v["x"])
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
        for i, (a, c) in enumerate(zip(out, eager[rep])):
            assert torch.equal(a, c), "replay of set %d: output %d" % (rep, i)
        step({n: _leaf(k[n]) for n in NAMES}, cu, dy)
