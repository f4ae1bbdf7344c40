"""The layer norm within bounds that follow its sums' order (layer_norm_tree.py):
rows whose mean is far from their spread, and wide rows of several tokens a
workgroup."""
import pytest
import torch

from layer_cases import norm_inputs
from layer_norm_tree import LayerNormTree, rows_far_from_zero
from ssm_cases import Maker
from ssm_ref import close

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def vdc():
    import varlen_depthwise_causal_amd as v
    return v


def check(vdc, s, w, b, dy, dstream, eps):
    ref = LayerNormTree(s, w, b, eps)
    y, _ = vdc.layer_norm_fwd(s, w, bias=b, eps=eps)
    close("y", y, ref.y, ref.ey)
    want = ref.grads(dy, dstream)
    for name, t in zip(("dx", "dweight", "dbias"), vdc.layer_norm_bwd(s, w, dy, bias=b, dstream=dstream, eps=eps)):
        close(name, t, *want[name])


@pytest.mark.parametrize("S,C", [(33, 40), (70, 65), (33, 128), (19, 200), (40, 520), (130, 1001), (65, 1024), (21, 1544),
                                 (40, 2056), (65, 4096), (20, 4100), (20, 8192), (11, 8190), (20, 16384), (6, 16381)])
def test_rows_far_from_zero(vdc, S, C):
    m = Maker(601, DEV)
    s = rows_far_from_zero(S, C, C, DEV)
    w, b = m.uniform(C, lo=0.5, hi=1.5), m.normal(C, std=0.1, dtype=F32)
    check(vdc, s, w, b, m.normal(S, C), None, 1e-12)


@pytest.mark.parametrize("S,C,params", [(1300, 8192, F32), (1100, 8190, BF), (600, 16384, F32), (530, 16381, BF),
                                        (2500, 4096, BF), (3000, 2048, F32), (4500, 1001, F32)])
@pytest.mark.parametrize("residual", [True, False])
def test_several_tokens_a_workgroup(vdc, S, C, params, residual):
    k = norm_inputs(611, S, C, device=DEV, params=params, residual=residual)
    y, s = vdc.layer_norm_fwd(k["x"], k["weight"], bias=k["bias"], residual=k["residual"])
    want = (k["x"].float() + k["residual"].float()).to(BF) if residual else k["x"]
    assert torch.equal(s, want)
    ref = LayerNormTree(s, k["weight"], k["bias"])
    close("y", y, ref.y, ref.ey)
    del ref
    check(vdc, s, k["weight"], k["bias"], k["dy"], k["dstream"], 1e-5)
