"""The scan where the forward's choices change: rows at and past the longest
that take one launch, and longer rows whose B and C are read as they lie, with
every number of states the kernels are built for."""
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


def _one_launch(N):
    """Tokens that the forward takes in one launch."""
    return 160 if N <= 8 else 224 if N <= 16 else 320 if N <= 32 else 512


def _inputs(seed, lengths, C, N, G, layout):
    """layout: B and C dense, cut out of wider rows at multiples of 4 bytes, or
    at odd columns (which the forward copies first)."""
    k, docs, cu = scan_inputs(seed, lengths, C, N, G, device=DEV)
    pad, off = {"dense": (0, 0), "even": (10, 4), "odd": (9, 3)}[layout]
    if pad:
        both = torch.full((sum(lengths), 2 * G * N + pad), 7.0, dtype=BF, device=DEV)
        for n, at in (("B", off), ("C", off + G * N)):
            both[:, at:at + G * N] = k[n].flatten(1)
            k[n] = both[:, at:at + G * N].unflatten(1, (G, N))
    return k, docs, cu


def _run(vdc, k, docs, cu, resume):
    n, C, N = len(docs), k["A"].shape[0], k["A"].shape[1]
    state = Maker(702, DEV).normal(n, C, N, dtype=F32)
    head = [k[i] for i in ("x", "dt", "A", "B", "C")]
    ref = R.Scan(*head, docs, k["D"], k["z"], k["dt_bias"], state=state, slots=list(range(n)), resume=resume)
    y = vdc.selective_scan_fwd(*head, cu, D=k["D"], z=k["z"], dt_bias=k["dt_bias"], state=state,
                               resume=torch.tensor(resume, device=DEV))
    R.close("y", y, ref.y, ref.ey)
    R.close("state", state, ref.after, ref.eafter)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("past", [0, 1, 200])
@pytest.mark.parametrize("layout", ["dense", "even", "odd"])
def test_forward_at_and_past_one_launch(vdc, N, past, layout):
    S = _one_launch(N) + past
    lengths = [S // 2, 0, 1, S - S // 2 - 1, 0]
    k, docs, cu = _inputs(701, lengths, 136, N, 2, layout)
    assert (vdc.selective_scan_workspace_bytes("fwd", S, 136, N, 2) > 0) == (past > 0)
    for flip in (0, 1):
        _run(vdc, k, docs, cu, [i % 2 == flip for i in range(len(lengths))])


@pytest.mark.parametrize("N", [32, 64])
@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("layout", ["dense", "even"])
def test_gradients_of_many_states_read_as_they_lie(vdc, N, G, layout):
    lengths = [333, 0, 1, 166]
    k, docs, cu = _inputs(711, lengths, 120, N, G, layout)
    head = [k[i] for i in ("x", "dt", "A", "B", "C")]
    rest = {i: k[i] for i in ("D", "z", "dt_bias")}
    dy = Maker(712, DEV).normal(sum(lengths), 120)
    want = R.Scan(*head, docs, k["D"], k["z"], k["dt_bias"]).grads(dy)
    got = vdc.selective_scan_bwd(*head, cu, dy, **rest)
    for name, t in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), got):
        R.close(name, t, *want[name])
