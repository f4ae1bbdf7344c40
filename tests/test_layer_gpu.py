"""The recurrent layer's operators on the GPU against their 64-bit definitions
(layer_ref.py), element by element, each within its own bound."""
import pytest
import torch

import layer_ref as L
from layer_cases import norm_inputs, recur_inputs
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


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ---------------------------------------------- gated linear recurrence --

LONG = [0, 37, 1, 0, 260, 2, 0]
RECUR = [
    # lengths, C, options
    ([1], 1, {}),
    ([5], 65, {"wide": True}),
    (LONG, 130, {"wide": True}),
    (LONG, 130, {"gate": False}),
    (LONG, 129, {"params": BF}),
    ([300], 72, {"params": BF, "wide": True}),
    ([64, 64, 128, 63, 1, 65], 64, {}),       # documents that end with tiles
    ([129, 500], 520, {"gate": False}),
    ([1] * 700, 33, {}),
    ([2300], 136, {"low": 0.999, "high": 0.99999}),
    ([200, 3], 256, {"low": 1e-6, "high": 0.5}),
    ([1500, 40], 8, {"low": 0.5, "high": 0.9999, "params": BF}),
    ([0, 0, 0], 16, {}),
    ([], 16, {}),
    ([0] * 600 + [90] + [0] * 600, 24, {}),
]
IDS = ["-".join(map(str, (sum(c[0]), len(c[0]), c[1]))) for c in RECUR]


@pytest.mark.parametrize("lengths,C,more", RECUR, ids=IDS)
@pytest.mark.parametrize("stateful", [False, True])
def test_gated_recurrence_fwd(vdc, lengths, C, more, stateful):
    k, docs, cu = recur_inputs(11, lengths, C, device=DEV, **more)
    st, slots, resume, own = None, None, None, {}
    if stateful:
        n = len(lengths)
        st = Maker(12, DEV).normal(n + 2, C, dtype=F32)
        slots = [n + 1 - j for j in range(n)]
        if n > 3:
            slots[1], slots[3] = -1, n + 2
        resume = [j % 3 != 2 for j in range(n)]
        own = {"state": st.clone(), "state_index": ints(slots), "resume": torch.tensor(resume, dtype=torch.bool,
                                                                                       device=DEV)}
        slots = [s if 0 <= s < n + 2 else -1 for s in slots]
    ref = L.Recurrence(k["x"], k["r"], k["i"], k["decay"], docs, k["z"], 8.0, st, slots, resume)
    y = vdc.gated_recurrence_fwd(k["x"], k["r"], k["i"], k["decay"], cu, z=k["z"], **own)
    close("y", y, ref.y, ref.ey)
    if stateful:
        close("state", own["state"], ref.after, ref.eafter)


@pytest.mark.parametrize("lengths,C,more", RECUR, ids=IDS)
def test_gated_recurrence_bwd(vdc, lengths, C, more):
    k, docs, cu = recur_inputs(21, lengths, C, device=DEV, **more)
    dy = Maker(22, DEV).normal(k["x"].shape[0], C + 2)[:, 1:1 + C]
    ref = L.Recurrence(k["x"], k["r"], k["i"], k["decay"], docs, k["z"])
    y, keep = vdc.gated_recurrence_fwd(k["x"], k["r"], k["i"], k["decay"], cu, z=k["z"], keep=True)
    close("y", y, ref.y, ref.ey)
    # of the states at every 64th token those that a document goes on from
    rows = torch.tensor([t for t in range(0, k["x"].shape[0], 64) if not any(lo == t < hi for lo, hi in docs)],
                        dtype=torch.long, device=DEV)
    close("keep", keep[rows // 64], ref.before[rows], L.MORE * ref.ebefore[rows])
    got = vdc.gated_recurrence_bwd(k["x"], k["r"], k["i"], k["decay"], cu, dy, keep, z=k["z"])
    ref = ref.grads(dy)
    for name, t in zip(("dx", "dr", "di", "ddecay", "dz"), got):
        if t is None:
            assert name == "dz" and k["z"] is None
        else:
            close(name, t, *ref[name])


@pytest.mark.parametrize("rows,C,more", [(1, 1, {}), (5, 65, {"wide": True}), (33, 130, {"wide": True}),
                                         (9, 520, {"gate": False}), (3, 40, {"params": BF}), (700, 1030, {}),
                                         (0, 16, {}), (4, 4096, {}), (1000, 24, {"params": BF, "gate": False})])
@pytest.mark.parametrize("indexed", [True, False])
def test_gated_recurrence_update(vdc, rows, C, more, indexed):
    k, _, _ = recur_inputs(31, [rows], C, device=DEV, **more)
    st = Maker(32, DEV).normal(rows + 2, C, dtype=F32)
    slots = [rows + 1 - j for j in range(rows)] if indexed else list(range(rows))
    if rows > 3 and indexed:
        slots[1], slots[3] = -1, rows + 2
    given = [s if 0 <= s < rows + 2 else -1 for s in slots]
    ref = L.Recurrence(k["x"], k["r"], k["i"], k["decay"], [(j, j + 1) for j in range(rows)], k["z"], 8.0, st, given,
                       [True] * rows)
    for j, s in enumerate(given):
        if s < 0:
            ref.y[j], ref.ey[j] = 0, 0
    own = st.clone()
    y = vdc.gated_recurrence_update(k["x"], k["r"], k["i"], k["decay"], own, z=k["z"],
                                    state_index=ints(slots) if indexed else None)
    close("y", y, ref.y, ref.ey)
    close("state", own, ref.after, ref.eafter)


# ------------------------------------------------------------ layer norm --

NORM = [(1, 1, {}), (3, 7, {"wide": True}), (33, 64, {}), (70, 65, {"bias": False}), (257, 128, {"params": BF}),
        (19, 200, {"wide": True}), (33, 520, {}), (130, 1001, {"residual": False}), (64, 1024, {"wide": True}),
        (21, 1544, {"params": BF}), (5, 2056, {}), (300, 4096, {"residual": False, "bias": False}),
        (9, 4100, {"wide": True}), (12, 8192, {}), (4, 9000, {"residual": False}), (5, 16384, {"params": BF}),
        (2, 16381, {}), (0, 64, {}), (2100, 40, {}), (600, 2048, {"mean": 40.0, "std": 0.5})]
NORM_IDS = ["%d-%d" % c[:2] for c in NORM]


@pytest.mark.parametrize("S,C,more", NORM, ids=NORM_IDS)
def test_layer_norm(vdc, S, C, more):
    k = norm_inputs(51, S, C, device=DEV, **more)
    y, stream = vdc.layer_norm_fwd(k["x"], k["weight"], bias=k["bias"], residual=k["residual"])
    want = k["x"] if k["residual"] is None else (k["x"].float() + k["residual"].float()).to(BF)
    assert torch.equal(stream, want), "the sum is rounded once"
    ref = L.LayerNorm(want, k["weight"], k["bias"])
    close("y", y, ref.y, ref.ey)
    got = vdc.layer_norm_bwd(stream, k["weight"], k["dy"], bias=k["bias"], dstream=k["dstream"])
    ref = ref.grads(k["dy"], k["dstream"])
    for name, t in zip(("dx", "dweight", "dbias"), got):
        if t is None:
            assert name == "dbias" and k["bias"] is None
        else:
            close(name, t, *ref[name])


# ------------------------------------------------------ states put aside --

POOL = [(1, (1,)), (3, (64,)), (5, (63,)), (4, (3, 24)), (7, (130, 13)), (2, (520, 16)), (3, (4096,)), (2, (4099,)),
        (600, (40,)), (2, (1024, 64))]


@pytest.mark.parametrize("rows,tail", POOL)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_states_put_aside(vdc, rows, tail, dtype, code):
    m = Maker(61, DEV)
    slots, pool = 2 * rows + 3, rows + 4
    state = (m.normal(slots, *tail, dtype=F32) * torch.exp(m.normal(slots, *[1] * len(tail), std=4.0, dtype=F32)))
    state = state.to(dtype)
    E = state[0].numel()
    codes = torch.zeros(pool, E, dtype=torch.int8, device=DEV).view(code)
    scales = torch.full((pool, (E + 63) // 64), -1.0, device=DEV)
    leave, places = [(3 * j + 1) % slots for j in range(rows)], [pool - 1 - j for j in range(rows)]
    if len(set(leave)) < rows or slots % 3 == 0:
        leave = list(range(rows))
    skipped = set()
    if rows > 2:
        leave[1], places[2], skipped = -1, pool, {1, 2}
    vdc.state_quantize(state, codes, scales, state_index=ints(leave), pool_index=ints(places))
    for j in range(rows):
        if j in skipped:
            continue
        q, scale = L.put_aside(state[leave[j]].double().view(-1), code)
        if j < 40:
            assert torch.equal(scales[places[j]], scale)
            assert torch.equal(codes[places[j]].float(), q.float())
    held = {places[j] for j in range(rows) if j not in skipped}
    for p in set(range(pool)) - held:
        assert bool((scales[p] == -1).all()) and bool((codes[p].float() == 0).all()), "places left out stay"
    enter = [slots - 1 - j for j in range(rows)]
    back = state.clone()
    if rows > 2:
        enter[0] = slots
    vdc.state_dequantize(codes, scales, back, pool_index=ints(places), state_index=ints(enter))
    want = state.clone()
    for j in range(rows):
        if 0 <= places[j] < pool and 0 <= enter[j] < slots:
            want[enter[j]] = L.take_back(codes[places[j]].float(), scales[places[j]], dtype).view(tail)
    assert torch.equal(back, want)


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_codes_at_their_borders(vdc, code):
    """Quotients next to and at the middle of two codes, of either sign, at
    scales whose quotients are not exact."""
    mags = L.codes_of(code)
    middle = ((mags[1:] + mags[:-1]) / 2).float()
    rows = []
    for top in (1.0, 3.3, 1e-3, 7.7e15, 2.0 ** -60):
        scale = torch.tensor(top, dtype=torch.float64).float().double() / mags[-1]
        at = (middle.double() * scale.float().double()).float()
        bits = at.view(torch.int32)
        for off in (-2, -1, 0, 1, 2):
            v = (bits + off).view(torch.float32).clamp(max=top)
            v = torch.cat([v, -v])
            v = torch.cat([v, torch.zeros((-v.numel()) % 63)]).view(-1, 63)
            rows.append(torch.cat([torch.full((v.shape[0], 1), top), v], 1).view(-1))
    state = torch.stack(rows).to(DEV)
    n, E = state.shape
    codes = torch.zeros(n, E, dtype=torch.int8, device=DEV).view(code)
    scales = torch.zeros(n, E // 64, device=DEV)
    vdc.state_quantize(state, codes, scales)
    for j in range(n):
        q, scale = L.put_aside(state[j].double(), code)
        assert torch.equal(scales[j], scale)
        assert torch.equal(codes[j].float(), q.float()), j


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_blocks_of_unusual_values(vdc, code, dtype):
    """Zeros, the smallest and largest values, infinities and NaN: a block's
    fate is its own."""
    v = torch.zeros(1, 64 * 9 + 5, device=DEV)
    v[0, 70] = 2.0 ** -64
    v[0, 71] = 2.0 ** -72
    v[0, 130] = 2.0 ** -65
    v[0, 200] = float("inf")
    v[0, 300] = float("nan")
    v[0, 320:384] = torch.finfo(dtype).max
    v[0, 384:448] = torch.linspace(-1e-30, 1e30, 64)
    v[0, 448] = 1e-44
    v[0, 520] = -0.0
    v[0, 576:] = torch.tensor([5.0, -5.0, 2.5, 1.0, 0.01])
    v = v.to(dtype)
    codes = torch.zeros(1, v.shape[1], dtype=torch.int8, device=DEV).view(code)
    scales = torch.zeros(1, 10, device=DEV)
    vdc.state_quantize(v, codes, scales)
    q, scale = L.put_aside(v[0].double(), code)
    assert torch.equal(scales[0].isnan(), scale.isnan())
    assert torch.equal(scales[0].nan_to_num(-1), scale.nan_to_num(-1))
    assert torch.equal(codes[0].float(), q.float())
    back = torch.empty_like(v)
    vdc.state_dequantize(codes, scales, back)
    poisoned = torch.zeros(v.shape[1], dtype=torch.bool)
    poisoned[192:256] = poisoned[256:320] = True
    assert torch.equal(back[0].isnan().cpu(), poisoned)
