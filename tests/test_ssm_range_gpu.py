"""The state space layer's operators at sizes past 2^32 threads of a lane a
value: long packed rows with many states."""
import pytest
import torch

import ssm_ref as R
from ssm_cases import Maker, scan_inputs

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


@pytest.mark.parametrize("N", [16, 13])
def test_scan_fwd_of_a_row_past_2_28_tokens(vdc, N):
    """B and C read as they are (16 states) and by way of padded copies (13);
    the first tokens of the row and its last documents are held to the
    definition."""
    C, S, tail = 1, 2 ** 28 + 5000, 1500
    k, _, _ = scan_inputs(601, [8], C, N, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(602)
    act = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF)  # noqa: E731
    x, dt, z = act(S, C), act(S, C), act(S, C)
    B, Cm = act(S, 1, N), act(S, 1, N)
    e = [0, S - tail, S - 500, S]
    cu = torch.tensor(e, dtype=torch.int32, device=DEV)
    y = vdc.selective_scan_fwd(x, dt, k["A"], B, Cm, cu, D=k["D"], z=z, dt_bias=k["dt_bias"])
    assert vdc.selective_scan_workspace_bytes("fwd", S, C, N) > 0
    for lo, hi, docs in ((0, tail, [(0, tail)]), (S - tail, S, [(0, tail - 500), (tail - 500, tail)])):
        t = slice(lo, hi)
        ref = R.Scan(x[t], dt[t], k["A"], B[t], Cm[t], docs, k["D"], z[t], k["dt_bias"])
        R.close("y", y[t], ref.y, ref.ey)
    assert bool(torch.isfinite(y).all())
