"""The gated recurrence at sizes that take the kernels of large batches (more than
512 tiles of 64 tokens and 64 channels backward, tiles of 128 tokens forward)
against its 64-bit definition: documents over dozens of tiles, masked tokens, a
NaN, prefix sums in no order."""
import pytest
import torch

import layer_ref as L
from layer_cases import recur_inputs
from ssm_cases import Maker
from ssm_ref import close

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
DEV = "cuda:0"
NAMES = ("x", "r", "i", "decay")
GRADS = ("dx", "dr", "di", "ddecay", "dz")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def vdc():
    import varlen_depthwise_causal_amd as v
    return v


def head(k):
    return [k[n] for n in NAMES]


LARGE = [
    ([5000, 0, 4000], 264, {}),
    ([5000, 0, 4000], 264, {"gate": False, "wide": True, "params": BF}),
    ([1, 2300, 63, 700], 1032, {"low": 0.99, "high": 0.99999}),
    ([3100], 1089, {"low": 0.2, "high": 0.9999, "gate": False}),
    # 32 tiles of tokens and fewer, whose sums of the decay's gradient are handed on
    ([1200, 800], 1100, {}),
    ([700], 3008, {"gate": False, "params": BF}),
]


@pytest.mark.parametrize("lengths,C,more", LARGE, ids=["%d-%d-%d" % (sum(n), len(n), c) for n, c, _ in LARGE])
def test_large_batches(vdc, lengths, C, more):
    k, docs, cu = recur_inputs(701, lengths, C, device=DEV, **more)
    n, S = len(lengths), sum(lengths)
    assert (S + 63) // 64 * ((C + 63) // 64) > 512
    st = Maker(702, DEV).normal(n + 1, C, dtype=F32)
    slots = [n - j for j in range(n)]
    resume = [j % 2 == 0 for j in range(n)]
    ref = L.Recurrence(*head(k), docs, k["z"], 8.0, st, slots, resume)
    own = st.clone()
    y = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=own, state_index=torch.tensor(slots, dtype=torch.int32,
                                                                                             device=DEV),
                                 resume=torch.tensor(resume, device=DEV))
    close("y", y, ref.y, ref.ey)
    close("state", own, ref.after, ref.eafter)
    ref = L.Recurrence(*head(k), docs, k["z"])
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    close("y", y, ref.y, ref.ey)
    dy = Maker(703, DEV).normal(S, C)
    want = ref.grads(dy)
    for name, t in zip(GRADS, vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])):
        if t is not None:
            close(name, t, *want[name])


@pytest.mark.parametrize("junk", [0.0, float("inf"), float("nan")])
def test_masked_tokens(vdc, junk):
    lengths, C = [2500, 900], 640
    k, docs, cu = recur_inputs(711, lengths, C, device=DEV)
    S = sum(lengths)
    masked = torch.rand(S, generator=torch.Generator().manual_seed(1)) < 0.3
    masked[100:500] = masked[2300:2600] = masked[-70:] = True  # tiles without a token, over a border
    masked = masked.to(DEV)
    k["r"][masked] = torch.finfo(BF).min if junk else float("-inf")
    clean = {n: t.clone() for n, t in k.items()}
    clean["x"][masked] = 0
    k["x"][masked] = junk
    if junk:
        k["i"][masked] = -junk
    dy = Maker(712, DEV).normal(S, C)
    ref = L.Recurrence(*head(clean), docs, k["z"])
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    close("y", y, ref.y, ref.ey)
    want = ref.grads(dy)
    got = vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])
    for name, t in zip(GRADS, got):
        close(name, t, *want[name])
    for t in got[:3]:
        assert bool((t[masked] == 0).all())


def test_a_nan_stays_in_its_document(vdc):
    lengths, C = [1300, 1100, 0, 1000], 640
    k, docs, cu = recur_inputs(721, lengths, C, device=DEV)
    S = sum(lengths)
    dy = Maker(722, DEV).normal(S, C)
    bad = {n: t.clone() for n, t in k.items()}
    bad["x"][1400, 3], bad["i"][1301, 70], bad["r"][2399, 639], bad["x"][2000, 200] = (
        float("nan"), float("nan"), float("nan"), float("inf"))
    cols = torch.tensor([3, 70, 639, 200], device=DEV)
    ref = L.Recurrence(*head(k), docs, k["z"])
    want = ref.grads(dy)
    y, keep = vdc.gated_recurrence_fwd(*head(bad), cu, z=k["z"], keep=True)
    assert bool(y[1400:2400, 3].isnan().all()) and bool(y[1301:2400, 70].isnan().all()) and bool(y[2399, 639].isnan())
    assert not bool(torch.isfinite(y[2000, 200]))
    got = vdc.gated_recurrence_bwd(*head(bad), cu, dy, keep, z=k["z"])
    touched = torch.zeros(S, C, dtype=torch.bool, device=DEV)
    touched[1300:2400, cols] = True
    apart = torch.zeros((), dtype=BF, device=DEV)
    close("y", torch.where(touched, apart, y), torch.where(touched, 0.0, ref.y), ref.ey)
    for name, t in zip(GRADS, got):
        w, e = want[name]
        if name == "ddecay":
            rest = torch.ones(C, dtype=torch.bool, device=DEV)
            rest[cols] = False
            close(name, t[rest], w[rest], e[rest])
            assert bool(t[cols[:3]].isnan().all())
        else:
            close(name, torch.where(touched, apart, t), torch.where(touched, 0.0, w), e)


@pytest.mark.parametrize("ends", [[5, 3, 9000], [0, -7, 9000], [0, 9900, 100, 9000], [9000, 0], [0, 0], [0, 4000],
                                  [-2 ** 31, 2 ** 31 - 1]])
def test_prefix_sums_in_no_order(vdc, ends):
    """The results are unspecified, the call ends inside its buffers."""
    S, C = 9000, 264
    k, _, _ = recur_inputs(731, [S], C, device=DEV)
    cu, n = torch.tensor(ends, dtype=torch.int32, device=DEV), len(ends) - 1
    guard = torch.full((n + 2, C), 7.0, device=DEV)
    vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=guard[1:n + 1], resume=torch.ones(n, dtype=torch.bool, device=DEV))
    rows = torch.full((S + 2, C), 3.0, dtype=BF, device=DEV)
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True, out=rows[1:-1])
    vdc.gated_recurrence_bwd(*head(k), cu, y, keep, z=k["z"])
    torch.cuda.synchronize()
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())
    assert bool((rows[0] == 3).all()) and bool((rows[-1] == 3).all())
