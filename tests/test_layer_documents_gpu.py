"""The gated recurrence with many documents without tokens: the same bits as
without them, whichever tile has to look through them, and however long that
takes the tiles behind it."""
import pytest
import torch

from layer_cases import recur_inputs
from ssm_cases import Maker, edges

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


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# lengths of the documents with tokens, and how many empty ones go before each and
# behind the last; 8192 (16384) entries at a tile's tokens and more are searched
CASES = [
    ([9, 11], [0, 17000, 0], 40),
    ([40, 37], [20000, 30, 17000], 70),
    ([150, 150], [9000, 9000, 9000], 64),
    ([64, 1, 63, 200], [0, 12000, 0, 3, 12000], 130),
    ([128, 700, 1172], [8191, 8193, 20, 8500], 600),
]


@pytest.mark.parametrize("lengths,empty,C", CASES, ids=lambda v: str(v) if isinstance(v, int) else "-".join(map(str, v)))
@pytest.mark.parametrize("gate", [True, False])
def test_many_empty_documents(vdc, lengths, empty, C, gate):
    k, _, cu = recur_inputs(401, lengths, C, device=DEV, gate=gate)
    head, S = [k[n] for n in NAMES], sum(lengths)
    every, place = [], []
    for n, m in zip(lengths + [None], empty):
        every += [0] * m
        if n is not None:
            place.append(len(every))
            every.append(n)
    D = len(every)
    many = ints(edges(every))
    g = torch.Generator().manual_seed(402)
    # half of the empty documents have a slot, half of all resume
    slots = torch.randperm(D + 3, generator=g)[:D].int()
    slots[torch.rand(D, generator=g) < 0.5] = -1
    resume = torch.rand(D, generator=g) < 0.5
    slots[place[0]], resume[place[-1]] = D + 1, True
    state = Maker(403, DEV).normal(D + 3, C, dtype=torch.float32)
    slots[place[0] + 1:][slots[place[0] + 1:] == D + 1] = -1
    slots[:place[0]][slots[:place[0]] == D + 1] = -1
    want, got = state.clone(), state.clone()
    y0 = vdc.gated_recurrence_fwd(*head, cu, z=k["z"], state=want, state_index=slots[place].to(DEV),
                                  resume=resume[place].to(DEV))
    cleared = slots[(torch.tensor(every) == 0) & ~resume & (slots >= 0)].long().to(DEV)
    want[cleared] = 0
    y = vdc.gated_recurrence_fwd(*head, many, z=k["z"], state=got, state_index=slots.to(DEV), resume=resume.to(DEV))
    assert torch.equal(y, y0) and torch.equal(got, want)
    dy = Maker(404, DEV).normal(S, C)
    outs = []
    for c in (cu, many):
        y, keep = vdc.gated_recurrence_fwd(*head, c, z=k["z"], keep=True)
        outs.append([y, keep, *vdc.gated_recurrence_bwd(*head, c, dy, keep, z=k["z"])])
    for a, b in zip(*outs):
        assert (a is None and b is None) or torch.equal(a, b)


def test_so_many_empty_documents_that_they_take_long(vdc):
    """2^28 of them at one token, and all of those that leave zeros in the first
    tiles' parts: looked through before a tile hands its state on, they would take
    longer than the next tile waits."""
    S, C, D = 300, 64, 1 << 28
    k, _, cu = recur_inputs(411, [150, 150], C, device=DEV)
    head = [k[n] for n in NAMES]
    many = torch.full((D + 1,), 150, dtype=torch.int32, device=DEV)
    many[0], many[-1] = 0, S
    state = Maker(412, DEV).normal(9, C, dtype=torch.float32)
    slots = torch.full((D,), -1, dtype=torch.int32, device=DEV)
    resume = torch.zeros(D, dtype=torch.bool, device=DEV)
    resume[D // 2:] = True
    for d, s in ((0, 7), (1, 0), (5000, 1), (D // 3, 2), (D // 2 - 1, 3), (D // 2, 4), (D - 2, 5), (D - 1, 6)):
        slots[d] = s
    want, got = state.clone(), state.clone()
    y0 = vdc.gated_recurrence_fwd(*head, cu, z=k["z"], state=want, state_index=ints([7, 6]),
                                  resume=torch.tensor([False, True], device=DEV))
    want[:4] = 0
    y = vdc.gated_recurrence_fwd(*head, many, z=k["z"], state=got, state_index=slots, resume=resume)
    assert torch.equal(y, y0) and torch.equal(got, want)
    dy = Maker(413, DEV).normal(S, C)
    outs = []
    for c in (cu, many):
        y, keep = vdc.gated_recurrence_fwd(*head, c, z=k["z"], keep=True)
        outs.append([y, keep, *vdc.gated_recurrence_bwd(*head, c, dy, keep, z=k["z"])])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
