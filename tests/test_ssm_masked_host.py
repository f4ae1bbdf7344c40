"""The definition of a masked step, on the CPU: a step of -inf has the size 0 in
torch's own softplus, the token leaves the state as it is, and a step of -1024,
with which the tests on the GPU evaluate the 64-bit definition, gives the same."""
import torch

import ssm_ref as R
from ssm_cases import Maker, scan_inputs


def test_a_masked_step_in_the_definition():
    k, docs, _ = scan_inputs(1, [4, 9], 6, 3, 2, device="cpu")
    dy = Maker(2, "cpu").normal(13, 6)
    where = torch.rand(13, 6, generator=torch.Generator().manual_seed(3)) < 0.4
    k["dt"] = k["dt"].masked_fill(where, -1024.0)
    r = R.Scan(*(k[n] for n in ("x", "dt", "A", "B", "C")), docs, k["D"], k["z"], k["dt_bias"])
    p = {n: t.double() for n, t in k.items()}
    p["dt"] = p["dt"].masked_fill(where, float("-inf")).requires_grad_()
    d = torch.nn.functional.softplus(p["dt"] + p["dt_bias"])
    assert bool((d[where] == 0).all())
    ys = []
    for lo, hi in docs:
        h = torch.zeros(6, 3, dtype=torch.float64)
        for t in range(lo, hi):
            h = torch.exp(d[t][:, None] * p["A"]) * h + (d[t] * p["x"][t])[:, None] * p["B"][t].repeat_interleave(3, 0)
            y = (h * p["C"][t].repeat_interleave(3, 0)).sum(-1) + p["D"] * p["x"][t]
            ys.append(y * torch.nn.functional.silu(p["z"][t]))
    y = torch.stack(ys)
    torch.testing.assert_close(r.y, y.detach(), rtol=1e-12, atol=1e-13)
    y.backward(dy.double())
    torch.testing.assert_close(r.grads(dy)["ddt"][0], p["dt"].grad, rtol=1e-10, atol=1e-12)
    assert bool((p["dt"].grad[where] == 0).all())
    for grad, bound in r.grads(dy).values():
        assert bool(torch.isfinite(grad).all()) and bool(torch.isfinite(bound).all())
