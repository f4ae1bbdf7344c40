"""The state space layer's operators on the GPU against their 64-bit
definitions (ssm_ref.py), element by element, each within its own bound."""
import pytest
import torch

import ssm_ref as R
from ssm_cases import Maker, edges, scan_inputs

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


# ------------------------------------------------------------ convolution --

CONV = [([1], 8, F32), ([0, 1, 2, 3, 4, 0, 5, 300], 520, F32), ([700, 0, 1, 1324], 1024, BF),
        ([2], 4096, BF), ([0, 0], 64, F32), ([3, 3, 3], 72, F32)]


@pytest.mark.parametrize("lengths,C,dtype", CONV)
@pytest.mark.parametrize("bias", [True, False])
def test_conv1d_prefill(vdc, lengths, C, dtype, bias):
    m = Maker(3, DEV)
    e, docs = edges(lengths), len(lengths)
    x = m.normal(e[-1], C)
    w = m.uniform(C, 4, lo=-0.5, hi=0.5, dtype=dtype)
    b = m.normal(C, std=0.1, dtype=dtype) if bias else None
    cu = torch.tensor(e, dtype=torch.int32, device=DEV)
    state = m.normal(docs + 3, 3, C)
    slots = [(5 * i + 2) % (docs + 3) for i in range(docs)] if docs % 5 else list(range(docs))
    if len(set(slots)) < docs:
        slots = list(range(docs))[::-1]
    if docs > 2:
        slots[1], slots[2] = -1, docs + 3  # no slot: below and above the cache
    resume = [i % 2 == 1 or i == 0 for i in range(docs)]
    given = [s if 0 <= s < docs + 3 else -1 for s in slots]
    y, bound, after = R.conv(x.double(), w, b, list(zip(e, e[1:])), state, given, resume)
    got = state.clone()
    out = vdc.conv1d_prefill(x, w, cu, got, bias=b, state_index=torch.tensor(slots, dtype=torch.int32, device=DEV),
                             resume=torch.tensor(resume, device=DEV))
    R.close("y", out, y, bound)
    assert torch.equal(got, after), "the carried inputs are exact"
    fresh = vdc.conv1d_prefill(x, w, cu, state.clone(), bias=b)
    if e[-1]:
        assert torch.equal(fresh, vdc.conv1d_fwd(x, w, cu, bias=b)), "fresh prompts are the packed forward's"


@pytest.mark.parametrize("rows,C,dtype", [(1, 8, F32), (7, 520, BF), (129, 4096, F32), (0, 64, F32)])
def test_conv1d_update(vdc, rows, C, dtype):
    m = Maker(4, DEV)
    x = m.normal(rows, C + 16)[:, 8:8 + C]
    w, b = m.uniform(C, 4, lo=-0.5, hi=0.5, dtype=dtype), m.normal(C, std=0.1, dtype=dtype)
    state = m.normal(rows + 4, 3, C)
    slots = [(rows + 3 - i) for i in range(rows)]
    if rows > 2:
        slots[1], slots[2] = -7, rows + 4
    given = [s if 0 <= s < rows + 4 else -1 for s in slots]
    y, bound, after = R.conv(x.double(), w, b, [(i, i + 1) for i in range(rows)], state, given, [True] * rows)
    for i, s in enumerate(given):
        if s < 0:
            y[i], bound[i] = 0, 0
    out = vdc.conv1d_update(x, state, w, bias=b, state_index=torch.tensor(slots, dtype=torch.int32, device=DEV))
    R.close("y", out, y, bound)
    assert torch.equal(state, after)


def test_conv1d_tokens_after_a_prompt(vdc):
    """A prompt cut anywhere and continued, by prompts or by single tokens, is
    the whole prompt, bit for bit."""
    m = Maker(5, DEV)
    C, S = 264, 23
    x, w, b = m.normal(S, C), m.uniform(C, 4, lo=-0.5, hi=0.5), m.normal(C, std=0.1, dtype=F32)
    whole = vdc.conv1d_fwd(x, w, torch.tensor([0, S], dtype=torch.int32, device=DEV), bias=b)
    for cuts in ([0, 1, 23], [0, 2, 4, 23], [0, 20, 20, 23]):
        state, ys = m.normal(1, 3, C), []
        for lo, hi in zip(cuts, cuts[1:]):
            cu = torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV)
            ys.append(vdc.conv1d_prefill(x[lo:hi], w, cu, state, bias=b, resume=torch.tensor([lo > 0], device=DEV)))
        assert torch.equal(torch.cat(ys), whole)
    state = torch.zeros(1, 3, C, dtype=BF, device=DEV)
    ys = [vdc.conv1d_update(x[t:t + 1], state, w, bias=b) for t in range(S)]
    assert torch.equal(torch.cat(ys), whole)
    assert torch.equal(state[0], x[-3:])


# ------------------------------------------------------------------- scan --

LONG = [0, 37, 1, 0, 260, 2, 0]
SCAN = [
    # lengths, C, N, G, options
    ([1], 1, 1, 1, {}),
    ([5], 65, 16, 1, {}),
    (LONG, 130, 16, 1, {"wide": True}),
    (LONG, 130, 16, 2, {"gate": False, "D": False}),
    ([300], 72, 8, 3, {"params": BF}),
    ([32, 32, 64, 31, 1, 33], 64, 16, 1, {}),            # documents that end with chunks
    ([129, 500], 40, 13, 2, {"wide": True, "params": BF}),
    (LONG, 96, 32, 2, {"bias": False}),
    (LONG, 48, 64, 4, {"wide": True}),
    ([77], 20, 3, 1, {"softplus": False, "wide": True}),
    ([1] * 70, 64, 16, 1, {}),
    ([0, 0, 0], 16, 16, 1, {}),
]
IDS = ["-".join(map(str, (sum(c[0]), len(c[0])) + c[1:4])) for c in SCAN]


@pytest.mark.parametrize("lengths,C,N,G,more", SCAN, ids=IDS)
@pytest.mark.parametrize("stateful", [False, True])
def test_selective_scan_fwd(vdc, lengths, C, N, G, more, stateful):
    soft = more.get("softplus", True)
    k, docs, cu = scan_inputs(11, lengths, C, N, G, device=DEV, **more)
    st, slots, resume, own = None, None, None, {}
    if stateful:
        n = len(lengths)
        st = Maker(12, DEV).normal(n + 2, C, N, dtype=F32)
        slots = [n + 1 - i for i in range(n)]
        if n > 3:
            slots[1], slots[3] = -1, n + 2
        resume = [i % 3 != 2 for i in range(n)]
        own = {"state": st.clone(), "state_index": torch.tensor(slots, dtype=torch.int32, device=DEV),
               "resume": torch.tensor(resume, device=DEV)}
        slots = [s if 0 <= s < n + 2 else -1 for s in slots]
    ref = R.Scan(k["x"], k["dt"], k["A"], k["B"], k["C"], docs, k["D"], k["z"], k["dt_bias"], soft, st, slots,
                 resume)
    y = vdc.selective_scan_fwd(k["x"], k["dt"], k["A"], k["B"], k["C"], cu, D=k["D"], z=k["z"],
                               dt_bias=k["dt_bias"], dt_softplus=soft, **own)
    R.close("y", y, ref.y, ref.ey)
    if stateful:
        R.close("state", own["state"], ref.after, ref.eafter)


@pytest.mark.parametrize("lengths,C,N,G,more", SCAN, ids=IDS)
def test_selective_scan_bwd(vdc, lengths, C, N, G, more):
    soft = more.get("softplus", True)
    k, docs, cu = scan_inputs(21, lengths, C, N, G, device=DEV, **more)
    dy = Maker(22, DEV).normal(k["x"].shape[0], C)
    ref = R.Scan(k["x"], k["dt"], k["A"], k["B"], k["C"], docs, k["D"], k["z"], k["dt_bias"], soft).grads(dy)
    got = vdc.selective_scan_bwd(k["x"], k["dt"], k["A"], k["B"], k["C"], cu, dy, D=k["D"], z=k["z"],
                                 dt_bias=k["dt_bias"], dt_softplus=soft)
    got = dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), got))
    for name, t in got.items():
        if t is None:
            assert name == "ddt_bias" or name not in ref
        else:
            R.close(name, t, *ref[name])


@pytest.mark.parametrize("rows,C,N,G,more", [(1, 1, 1, 1, {}), (5, 65, 16, 1, {}), (33, 130, 16, 2, {"wide": True}),
                                             (9, 48, 64, 4, {"gate": False}), (3, 40, 13, 2, {"params": BF}),
                                             (4, 96, 32, 1, {"D": False}), (6, 24, 3, 1, {"softplus": False}),
                                             (7, 24, 8, 1, {"bias": False}), (0, 16, 16, 1, {})])
def test_selective_update(vdc, rows, C, N, G, more):
    soft = more.get("softplus", True)
    k, _, _ = scan_inputs(31, [rows], C, N, G, device=DEV, **more)
    st = Maker(32, DEV).normal(rows + 2, C, N, dtype=F32)
    slots = [rows + 1 - i for i in range(rows)]
    if rows > 3:
        slots[1], slots[3] = -1, rows + 2
    given = [s if 0 <= s < rows + 2 else -1 for s in slots]
    ref = R.Scan(k["x"], k["dt"], k["A"], k["B"], k["C"], [(i, i + 1) for i in range(rows)], k["D"], k["z"],
                 k["dt_bias"], soft, st, given, [True] * rows)
    for i, s in enumerate(given):
        if s < 0:
            ref.y[i], ref.ey[i] = 0, 0
    own = st.clone()
    y = vdc.selective_update(k["x"], k["dt"], k["A"], k["B"], k["C"], own, D=k["D"], z=k["z"],
                             dt_bias=k["dt_bias"], dt_softplus=soft,
                             state_index=torch.tensor(slots, dtype=torch.int32, device=DEV))
    R.close("y", y, ref.y, ref.ey)
    R.close("state", own, ref.after, ref.eafter)


def test_selective_scan_keeps_documents_apart(vdc):
    """A NaN or an infinity stays in its document, and in its channel where
    the formula does not mix channels."""
    lengths = [40, 90, 70]
    k, _, cu = scan_inputs(41, lengths, 64, 16, device=DEV)
    dy = Maker(42, DEV).normal(200, 64)
    args = (k["A"], k["B"], k["C"], cu)
    rest = {"D": k["D"], "z": k["z"], "dt_bias": k["dt_bias"]}
    clean = vdc.selective_scan_fwd(k["x"], k["dt"], *args, **rest)
    cleang = vdc.selective_scan_bwd(k["x"], k["dt"], *args, dy, **rest)
    x, dt = k["x"].clone(), k["dt"].clone()
    x[60, 3], dt[100, 5] = float("nan"), float("inf")
    y = vdc.selective_scan_fwd(x, dt, *args, **rest)
    assert bool(torch.isnan(y[60:130, 3]).all())
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[60:130, 3], keep[100:130, 5] = False, False
    assert torch.equal(y[keep], clean[keep])
    dx, ddt, _, dB, dC, _, dz, _ = vdc.selective_scan_bwd(x, dt, *args, dy, **rest)
    out = torch.ones(200, dtype=torch.bool, device=DEV)
    out[40:130] = False
    for a, b in ((dx, cleang[0]), (ddt, cleang[1]), (dB, cleang[3]), (dC, cleang[4]), (dz, cleang[6])):
        assert torch.equal(a[out], b[out])


# ------------------------------------------------------------- group norm --

NORM = [(1, 8, 1, F32, True), (33, 520, 8, F32, False), (5, 6, 2, BF, True), (64, 4096, 32, F32, True),
        (3, 16384, 1, BF, False), (9, 1000, 1, F32, True), (200, 65, 65, F32, True), (0, 64, 4, F32, True),
        (17, 2048, 1, BF, True), (2, 5000, 1, F32, False), (40, 264, 3, F32, True), (70, 512, 2, F32, False),
        (70, 1024, 2, BF, True), (13, 8192, 2, F32, True), (1100, 64, 1, F32, True)]


@pytest.mark.parametrize("S,C,G,dtype,gate", NORM)
@pytest.mark.parametrize("wide", [False, True])
def test_group_norm_silu(vdc, S, C, G, dtype, gate, wide):
    m = Maker(51, DEV)
    pad = 5 if wide else 0
    x = m.normal(S, C + pad, mean=0.3)[:, pad // 2:pad // 2 + C]
    z = m.normal(S, C + pad)[:, pad // 2:pad // 2 + C] if gate else None
    dy = m.normal(S, C + pad)[:, pad // 2:pad // 2 + C]
    if S > 2:
        x[1] = 1.5     # no variance
        x[2] *= 1e-3   # little, against eps
    w, b = m.uniform(C, lo=0.5, hi=1.5, dtype=dtype), m.normal(C, std=0.1, dtype=dtype) if C != 5000 else None
    ref = R.Norm(x, w, G, b, z)
    R.close("y", vdc.group_norm_silu_fwd(x, w, G, bias=b, z=z), ref.y, ref.ey)
    want = ref.grads(dy)
    got = dict(zip(("dx", "dweight", "dbias", "dz"), vdc.group_norm_silu_bwd(x, w, G, dy, bias=b, z=z)))
    for name, t in got.items():
        if t is not None:
            R.close(name, t, *want[name])
    assert (got["dz"] is None) == (z is None) and (got["dbias"] is None) == (b is None)


# ------------------------------------- streams, graphs, reproducible sums --

def _everything(vdc, k, cu, dy, z, states):
    rest = {"D": k["D"], "z": k["z"], "dt_bias": k["dt_bias"]}
    args = (k["A"], k["B"], k["C"])
    out = [vdc.selective_scan_fwd(k["x"], k["dt"], *args, cu, **rest),
           vdc.selective_scan_fwd(k["x"], k["dt"], *args, cu, state=states[0], **rest), states[0],
           vdc.selective_update(k["x"], k["dt"], *args, states[1], **rest), states[1]]
    out += vdc.selective_scan_bwd(k["x"], k["dt"], *args, cu, dy, **rest)
    w, b = k["D"], k["dt_bias"]
    out.append(vdc.group_norm_silu_fwd(k["x"], w, 4, bias=b, z=z))
    out += vdc.group_norm_silu_bwd(k["x"], w, 4, dy, bias=b, z=z)
    cw = k["A"][:, :4].contiguous()
    out += [vdc.conv1d_prefill(k["x"], cw, cu, states[2], bias=b), states[2],
            vdc.conv1d_update(k["x"], states[3], cw, bias=b), states[3]]
    return out


def _set(seed):
    lengths = [90, 0, 33, 200]
    k, _, cu = scan_inputs(seed, lengths, 128, 16, device=DEV)
    m = Maker(seed + 1, DEV)
    S = sum(lengths)
    dy, z = m.normal(S, 128), m.normal(S, 128)
    states = [m.normal(4, 128, 16, dtype=F32), m.normal(S, 128, 16, dtype=F32), m.normal(4, 3, 128), m.normal(S, 3, 128)]
    return k, cu, dy, z, states


def test_same_bits_on_any_stream_and_in_graphs(vdc):
    sets = [_set(s) for s in (61, 71, 81)]
    eager = [[t.clone() for t in _everything(vdc, k, cu, dy, z, [s.clone() for s in st])] for k, cu, dy, z, st in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k, cu, dy, z, st = sets[0]
    with torch.cuda.stream(side):
        again = _everything(vdc, k, cu, dy, z, [s.clone() for s in st])
    side.synchronize()
    for a, b in zip(again, eager[0]):
        assert torch.equal(a, b)
    hold = {n: t.clone() for n, t in k.items()}
    hz, hdy, hst = z.clone(), dy.clone(), [s.clone() for s in st]
    with torch.cuda.stream(side):
        _everything(vdc, hold, cu, hdy, hz, hst)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _everything(vdc, hold, cu, hdy, hz, hst)
    for rep in (0, 1, 2, 0):
        k, _, dy, z, st = sets[rep]
        for n in hold:
            hold[n].copy_(k[n])
        hz.copy_(z)
        hdy.copy_(dy)
        for a, b in zip(hst, st):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, eager[rep])):
            assert torch.equal(a, b), "replay of set %d: output %d" % (rep, i)
        _everything(vdc, k, cu, dy, z, [s.clone() for s in st])
