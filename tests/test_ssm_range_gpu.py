"""The state space layer's operators at sizes past 2^32 threads of a lane a
value: long packed rows with many states, and many rows of single tokens."""
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


def test_update_of_rows_past_2_18(vdc):
    """262147 rows of 4096 channels, three of them with a slot."""
    rows, C, N = 2 ** 18 + 3, 4096, 16
    real = [0, 2 ** 18 - 1, rows - 1]
    k, _, _ = scan_inputs(611, [3], C, N, device=DEV)
    state = Maker(612, DEV).normal(4, C, N, dtype=F32)
    small = state[:3].clone()
    index = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    wide = {n: torch.zeros((rows,) + tuple(k[n].shape[1:]), dtype=BF, device=DEV) for n in ("x", "dt", "B", "C")}
    for i, r in enumerate(real):
        index[r] = i
        for n in wide:
            wide[n][r] = k[n][i]
    y = vdc.selective_update(wide["x"], wide["dt"], k["A"], wide["B"], wide["C"], state, D=k["D"],
                             dt_bias=k["dt_bias"], state_index=index)
    want = vdc.selective_update(k["x"], k["dt"], k["A"], k["B"], k["C"], small, D=k["D"], dt_bias=k["dt_bias"])
    assert torch.equal(y[real], want) and torch.equal(state[:3], small)
    y[real] = 0
    assert int(torch.count_nonzero(y)) == 0
