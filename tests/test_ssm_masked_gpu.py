"""Steps of the scan at the ends of their range.  A step of -inf (a masked
token, or a channel whose bias masks it) has the size 0: such a token leaves the
state as it is.  The 64-bit definition is evaluated at -1024 in its place, whose
softplus is 0 in 64 bits as well, so that the bounds stay numbers."""
import pytest
import torch

import ssm_ref as R
from ssm_cases import Maker, scan_inputs

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
DEV = "cuda:0"
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")
MASK = -1024.0  # exact in BF16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def vdc():
    import varlen_depthwise_causal_amd as v
    return v


def _head(k):
    return [k[n] for n in ("x", "dt", "A", "B", "C")]


def _rest(k):
    return {n: k[n] for n in ("D", "z", "dt_bias")}


def _masked(seed, lengths, C, N, G, how, low):
    """The inputs with some steps masked, and those the definition is given."""
    k, docs, cu = scan_inputs(seed, lengths, C, N, G, device=DEV)
    S = sum(lengths)
    given = dict(k)
    g = torch.Generator().manual_seed(seed)
    if how == "bias":
        where = (torch.rand(C, generator=g) < 0.3).to(DEV)
        k["dt_bias"] = k["dt_bias"].masked_fill(where, low)
        given["dt_bias"] = given["dt_bias"].masked_fill(where, MASK)
        return k, given, docs, cu
    if how == "tokens":  # of all channels: the first and the last of each document, and some more
        where = torch.rand(S, 1, generator=g) < 0.2
        for lo, hi in docs:
            if hi > lo:
                where[lo] = where[hi - 1] = True
    else:
        where = torch.rand(S, C, generator=g) < 0.2
    where = where.to(DEV)
    k["dt"], given["dt"] = k["dt"].masked_fill(where, low), given["dt"].masked_fill(where, MASK)
    return k, given, docs, cu


SIZES = [([1], 64, 16, 1), ([0, 37, 1, 0, 60, 2, 0], 130, 13, 2), ([129, 0, 500], 72, 16, 1), ([300, 5, 230], 40, 5, 1),
         ([560, 40], 24, 64, 1), ([330, 2], 33, 32, 1)]
HOWS = ["tokens", "channels", "bias"]
LOW = [float("-inf"), torch.finfo(BF).min]


@pytest.mark.parametrize("lengths,C,N,G", SIZES)
@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("low", LOW)
def test_scan_of_masked_steps(vdc, lengths, C, N, G, how, low):
    k, given, docs, cu = _masked(401, lengths, C, N, G, how, low)
    n = len(lengths)
    state = Maker(402, DEV).normal(n, C, N, dtype=F32)
    resume = [i % 2 == 0 for i in range(n)]
    ref = R.Scan(*_head(given), docs, given["D"], given["z"], given["dt_bias"], state=state, slots=list(range(n)),
                 resume=resume)
    y = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k), state=state, resume=torch.tensor(resume, device=DEV))
    R.close("y", y, ref.y, ref.ey)
    R.close("state", state, ref.after, ref.eafter)


@pytest.mark.parametrize("lengths,C,N,G", SIZES)
@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("low", LOW)
def test_scan_gradients_of_masked_steps(vdc, lengths, C, N, G, how, low):
    k, given, docs, cu = _masked(411, lengths, C, N, G, how, low)
    dy = Maker(412, DEV).normal(sum(lengths), C)
    want = R.Scan(*_head(given), docs, given["D"], given["z"], given["dt_bias"]).grads(dy)
    got = dict(zip(GRADS, vdc.selective_scan_bwd(*_head(k), cu, dy, **_rest(k))))
    for name, t in got.items():
        R.close(name, t, *want[name])
    if how == "bias":
        assert bool((got["ddt_bias"][k["dt_bias"] == low] == 0).all())


@pytest.mark.parametrize("C,N,G", [(64, 16, 1), (130, 13, 2), (40, 5, 1), (24, 64, 1), (33, 32, 1), (8, 1, 1)])
@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("low", LOW)
def test_update_of_masked_steps(vdc, C, N, G, how, low):
    rows = 9
    k, given, _, _ = _masked(421, [rows], C, N, G, how, low)
    k["dt"], given["dt"] = k["dt"].clone(), given["dt"].clone()
    k["dt"][4], given["dt"][4] = low, MASK
    state = Maker(422, DEV).normal(rows, C, N, dtype=F32)
    before = state.clone()
    ref = R.Scan(*_head(given), [(i, i + 1) for i in range(rows)], given["D"], given["z"], given["dt_bias"],
                 state=state, slots=list(range(rows)), resume=[True] * rows)
    y = vdc.selective_update(*_head(k), state, **_rest(k))
    R.close("y", y, ref.y, ref.ey)
    R.close("state", state, ref.after, ref.eafter)
    assert torch.equal(state[4], before[4]), "a masked token leaves the state as it is"


def test_nan_steps_stay(vdc):
    """A step that is no number gives none, from its token on."""
    k, docs, cu = scan_inputs(431, [20, 30], 64, 16, device=DEV)
    k["dt"][25, 7] = float("nan")
    y = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k))
    bad = torch.isnan(y)
    assert bool(bad[25:, 7].all()) and int(bad.sum()) == 25


@pytest.mark.parametrize("S,at", [(700, 64), (2500, 192)])
def test_states_that_vanish_and_decays_past_the_range(vdc, S, at):
    """Steps of either sign (dt_softplus off): 32 tokens that take the state to
    nothing are followed by 32 whose decay alone is past FP32's range.  What
    follows is finite, and as the definition has it."""
    C, N = 64, 8
    k, docs, cu = scan_inputs(521, [S], C, N, device=DEV, softplus=False, gate=False)
    k["A"] = torch.full((C, N), -1.0, device=DEV)
    k["x"], k["dt"] = k["x"].clone(), k["dt"].clone()
    k["x"][at:at + 64] = 0.0
    k["dt"][at:at + 32], k["dt"][at + 32:at + 64] = 40.0, -12.0
    ref = R.Scan(*_head(k), docs, k["D"], softplus_on=False)
    y = vdc.selective_scan_fwd(*_head(k), cu, D=k["D"], dt_softplus=False)
    R.close("y", y, ref.y, ref.ey)


@pytest.mark.parametrize("S", [100, 1200])
@pytest.mark.parametrize("step", [False, True])
def test_steps_of_a_bias_that_cancels(vdc, S, step):
    """Step sizes near softplus(0) from a dt and a bias some hundred times as
    large: with x = B = 1 a first token's state is the step size, in FP32."""
    C = 64
    m = Maker(441, DEV)
    bias = -m.uniform(C, lo=2.0, hi=400.0)
    raw = m.normal(S, C, std=8.0, dtype=F32).clamp(-40, 40)
    dt = (raw - bias).to(BF)
    one = torch.ones(S, 1, dtype=BF, device=DEV)
    x = torch.ones(S, C, dtype=BF, device=DEV)
    A = torch.full((C, 1), -1.0, device=DEV)
    state = torch.zeros(S, C, 1, device=DEV)
    if step:
        vdc.selective_update(x, dt, A, one, one, state, dt_bias=bias)
    else:
        cu = torch.arange(S + 1, dtype=torch.int32, device=DEV)
        vdc.selective_scan_fwd(x, dt, A, one, one, cu, dt_bias=bias, state=state)
    want, rel = R.softplus(dt.double() + bias.double())
    R.close("step size", state[:, :, 0], want, want * rel)
