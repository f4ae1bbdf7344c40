"""The recurrent layer's operators at the largest sizes that they take, and their
refusal of one more: the last rows are bit for bit those of a call of their own."""
import pytest
import torch

import layer_ref as L

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


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def draw(*shape, seed, dtype=BF):
    return torch.randn(*shape, device=DEV, dtype=dtype, generator=torch.Generator(device=DEV).manual_seed(seed))


MOST = 2 ** 29 - 64  # 2^23 - 1 tiles of 64 tokens of one channel


def test_recurrence_of_the_most_tokens(vdc):
    """One document that ends 5 tiles of 128 and some tokens before the row does,
    and one behind it; its decay leaves nothing of the first tokens."""
    last = 5 * 128 + 17
    first = (MOST - last) // 128 * 128
    last = MOST - first
    x, decay = draw(MOST, 1, seed=801), torch.full((1,), -1.0, device=DEV)
    cu, state = ints([0, first, MOST]), torch.zeros(2, 1, device=DEV)
    y = vdc.gated_recurrence_fwd(x, x, x, decay, cu, state=state)
    tail = x[first:]
    one = torch.zeros(1, 1, device=DEV)
    want = vdc.gated_recurrence_fwd(tail, tail, tail, decay, ints([0, last]), state=one)
    assert torch.equal(y[first:], want) and torch.equal(state[1], one[0])
    # what the first document's last tokens leave, whose decays past 4096 tokens are 0
    near = x[first - 4096:first]
    ref = L.Recurrence(near, near, near, decay, [(0, 4096)])
    assert abs(float(state[0, 0]) - float(ref.h[-1])) <= float(L.MORE * ref.eh[-1]) + 1e-30
    y, keep = vdc.gated_recurrence_fwd(x, x, x, decay, cu, keep=True)
    got = vdc.gated_recurrence_bwd(x, x, x, decay, cu, x, keep)
    _, keep = vdc.gated_recurrence_fwd(tail, tail, tail, decay, ints([0, last]), keep=True)
    want = vdc.gated_recurrence_bwd(tail, tail, tail, decay, ints([0, last]), tail, keep)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[first:], b)
    assert bool(torch.isfinite(got[3]).all())


def test_single_tokens_of_the_most_rows(vdc):
    x, decay = draw(MOST, 1, seed=811), torch.full((1,), 0.5, device=DEV)
    state = draw(MOST, 1, seed=812, dtype=F32)
    at = torch.cat([torch.arange(100, device=DEV), torch.arange(MOST - 100, MOST, device=DEV)])
    some = state[at].clone()
    want = vdc.gated_recurrence_update(x[at], x[at], x[at], decay, some)
    y = vdc.gated_recurrence_update(x, x, x, decay, state)
    assert torch.equal(y[at], want) and torch.equal(state[at], some)


def test_more_tokens_are_refused(vdc):
    x = torch.zeros(MOST + 1, 1, dtype=BF, device=DEV)
    decay, cu = torch.zeros(1, device=DEV), ints([0, MOST + 1])
    with pytest.raises(vdc.VdcError):
        vdc.gated_recurrence_fwd(x, x, x, decay, cu)
    with pytest.raises(vdc.VdcError):
        vdc.gated_recurrence_update(x, x, x, decay, torch.zeros(MOST + 1, 1, device=DEV))


def test_layer_norm_of_the_most_tokens(vdc):
    S, C = 2 ** 31 - 1, 2
    x, w, b = draw(S, C, seed=821), draw(C, seed=822, dtype=F32), draw(C, seed=823, dtype=F32)
    y, same = vdc.layer_norm_fwd(x, w, bias=b)
    assert same is x
    tail = x[-300:]
    assert torch.equal(y[-300:], vdc.layer_norm_fwd(tail, w, bias=b)[0])
    dx, dw, db = vdc.layer_norm_bwd(x, w, y, bias=b)
    assert torch.equal(dx[-300:], vdc.layer_norm_bwd(tail, w, y[-300:], bias=b)[0])
    assert bool(torch.isfinite(dw).all())
    # FP32 over 256 turns and 32 teams, FP64 from there
    want = sum(y[i:i + (1 << 28)].double().sum(0) for i in range(0, S, 1 << 28))
    most = sum(y[i:i + (1 << 28)].double().abs().sum(0) for i in range(0, S, 1 << 28))
    assert bool(((db.double() - want).abs() <= (256 + 32 + 1) * 2.0 ** -24 * most).all())


def test_states_of_the_most_rows(vdc):
    rows, E = 2 ** 24 - 1, 64
    state = draw(rows, E, seed=831, dtype=F32)
    codes = torch.zeros(rows, E, dtype=torch.int8, device=DEV)
    scales = torch.zeros(rows, 1, device=DEV)
    vdc.state_quantize(state, codes, scales)
    for j in (0, rows // 2, rows - 1):
        q, scale = L.put_aside(state[j].double(), torch.int8)
        assert torch.equal(codes[j].float(), q.float()) and torch.equal(scales[j], scale)
    back = torch.zeros_like(state)
    vdc.state_dequantize(codes, scales, back)
    for j in (0, rows // 2, rows - 1):
        assert torch.equal(back[j], L.take_back(codes[j].float(), scales[j], F32))
    wide = torch.zeros(rows + 1, 1, device=DEV)
    with pytest.raises(vdc.VdcError):
        vdc.state_quantize(wide, torch.zeros(rows + 1, 1, dtype=torch.int8, device=DEV), torch.zeros(rows + 1, 1, device=DEV))
