"""Gradients of the scan's and the norm's parameters against differences of the
kernels' own outputs, along directions that the outputs answer to: the loss is
sum(w y) with w the signs of what the outputs do in 64 bits, so that every output
adds to the difference.  What rounding and curvature leave open has to be less
than a tenth of it, or the test would show nothing."""
import pytest
import torch

import ssm_ref as R
from ssm_cases import Maker, scan_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def hold(name, run, there, p, way):
    """run(p): the kernels' outputs; there(p): those of the definition.

    Every output is off by at most 2^-8 of itself; over outputs that are off in
    either direction independently of w this adds like a root sum of squares,
    taken eight times.  Of a central difference the error goes with the step's
    square: that of the whole step is 4/3 of what halving it takes away, of
    which 2 are allowed."""
    w = torch.sign(there(p + way) - there(p - way))
    leaf = p.detach().clone().requires_grad_()
    y = run(leaf)
    y.backward(w.bfloat16())
    diff = lambda s: float(((run(p + s * way).double() - run(p - s * way).double()) * w).sum() / (2 * s))  # noqa: E731
    got, half = diff(1.0), diff(0.5)
    want = float((leaf.grad.double() * way.double()).sum())
    noise = 8 * 2.0 ** -8 * float(((y.detach().double() * w) ** 2).sum().sqrt())
    allowed = noise + 2 * abs(got - half)
    print("%-8s difference %.5g gradient %.5g allowed %.3g" % (name, got, want, allowed), flush=True)
    assert abs(want) >= 10 * allowed, "shows nothing"
    assert abs(got - want) <= allowed


@pytest.mark.parametrize("name", ["A", "D", "dt_bias"])
@pytest.mark.parametrize("C,N,G", [(136, 16, 2), (40, 13, 1)])
def test_selective_scan(name, C, N, G):
    from varlen_depthwise_causal_amd.autograd import selective_scan
    k, docs, cu = scan_inputs(221, [40, 0, 170, 1], C, N, G, device=DEV)

    def run(p):
        q = {**k, name: p}
        return selective_scan(q["x"], q["dt"], q["A"], q["B"], q["C"], cu, D=q["D"], z=q["z"], dt_bias=q["dt_bias"])

    def there(p):
        q = {**k, name: p}
        return R.Scan(q["x"], q["dt"], q["A"], q["B"], q["C"], docs, q["D"], q["z"], q["dt_bias"]).y

    hold(name, run, there, k[name], {"A": -k["A"] * 0.25, "D": k["D"] * 0.25,
                                     "dt_bias": torch.full_like(k["dt_bias"], 0.25)}[name])


@pytest.mark.parametrize("name", ["weight", "bias"])
@pytest.mark.parametrize("gate", [True, False])
def test_group_norm_silu(name, gate):
    from varlen_depthwise_causal_amd.autograd import group_norm_silu
    m = Maker(231, DEV)
    x, z = m.normal(50, 320), m.normal(50, 320) if gate else None
    k = {"weight": m.uniform(320, lo=0.5, hi=1.5), "bias": m.normal(320, dtype=torch.float32)}

    def run(p):
        q = {**k, name: p}
        return group_norm_silu(x, q["weight"], 5, bias=q["bias"], z=z)

    def there(p):
        q = {**k, name: p}
        return R.Norm(x, q["weight"], 5, q["bias"], z).y

    hold(name, run, there, k[name], torch.full_like(k[name], 0.25))
