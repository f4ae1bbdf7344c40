"""The gated recurrence at the ends of its scale's range: finite, and the
definition's values."""
import pytest
import torch

import layer_ref as L
from layer_cases import recur_inputs
from ssm_cases import Maker
from ssm_ref import close

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAMES = ("x", "r", "i", "decay")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def vdc():
    import varlen_depthwise_causal_amd as v
    return v


@pytest.mark.parametrize("scale", [0.0, 1e-38, 1.6e38, 1.8e38, 3.4e38])
@pytest.mark.parametrize("lengths,C", [([20], 70), ([150, 3, 400], 64)])
def test_scales_at_the_ends_of_the_range(vdc, scale, lengths, C):
    """softplus(decay) counts as 0 below the normal numbers, and 0 times any scale
    is no step; a rate past 2^126 is a decay of 0 at any gate that is not closed."""
    k, docs, cu = recur_inputs(501, lengths, C, device=DEV)
    S = sum(lengths)
    decay = k["decay"]
    decay[::3] = -200.0
    decay[1::3] = torch.linspace(-4.0, 4.0, decay[1::3].numel(), device=DEV)
    decay[2::3] = float("-inf")
    none = torch.ones(C, dtype=torch.bool, device=DEV) if scale < 1.0 else decay < -100
    # Where a step would be taken from a softplus below the normal numbers, none is: in
    # 64 bits, softplus(-400) is 2^-577, and a step of it at any scale has m below 2^-224.
    used = decay.clone()
    used[none] = -400.0
    used_scale = scale if scale >= 1.0 else 8.0
    dy = Maker(502, DEV).normal(S, C)
    ref = L.Recurrence(k["x"], k["r"], k["i"], used, docs, k["z"], used_scale)
    head = [k[n] for n in NAMES]
    y, keep = vdc.gated_recurrence_fwd(*head, cu, z=k["z"], scale=scale, keep=True)
    # A scale of 1e-38 and a softplus of 5 at most: u below 2^-122 and m below 2^-61, of
    # which S tokens' worth reaches an output, times |x|, |dy| and |z| below 5 each (2^7).
    lost = S * 2.0 ** (7 - 61) if 0 < scale < 1 else 0.0
    assert max(float(t.abs().max()) for t in (k["x"], dy, k["z"])) < 5
    close("y", y, ref.y, ref.ey + lost)
    got = vdc.gated_recurrence_bwd(*head, cu, dy, keep, z=k["z"], scale=scale)
    for name, t in zip(("dx", "dr", "di", "ddecay", "dz"), got):
        w, e = ref.grads(dy)[name]
        close(name, t, w, e + (S if name == "ddecay" else 1) * lost)
    state = torch.zeros(S, C, device=DEV)
    y = vdc.gated_recurrence_update(*head, state, z=k["z"], scale=scale)
    one = L.Recurrence(k["x"], k["r"], k["i"], used, [(t, t + 1) for t in range(S)], k["z"], used_scale)
    close("y", y, one.y, one.ey + lost)
    if scale >= 1.0:
        assert bool((y[:, none] == 0).all())
