"""The recurrent layer's operators where they can go wrong: any stream and
workspace, graphs, many tiles and documents, masked tokens, infinities and NaN,
prefix sums that do not end with the row, strides, offsets past 32 bits."""
import pytest
import torch

import layer_ref as L
from layer_cases import norm_inputs, recur_inputs
from ssm_cases import Maker, edges
from ssm_ref import close

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
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


def head(k):
    return [k[n] for n in NAMES]


# --------------------------------------- streams, graphs, workspaces, bits --

def _set(seed, lengths=(90, 0, 33, 700), C=136):
    k, _, cu = recur_inputs(seed, list(lengths), C, device=DEV)
    m, S = Maker(seed + 1, DEV), sum(lengths)
    states = [m.normal(4, C, dtype=F32), m.normal(S, C, dtype=F32), m.normal(5, C, 3, dtype=F32)]
    return k, cu, norm_inputs(seed + 2, S, C, device=DEV), m.normal(S, C), states


def _everything(vdc, k, cu, n, dy, states):
    out = [vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=states[0]), states[0],
           vdc.gated_recurrence_update(*head(k), states[1], z=k["z"]), states[1]]
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    out += [y, keep, *vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])]
    y, s = vdc.layer_norm_fwd(n["x"], n["weight"], bias=n["bias"], residual=n["residual"])
    out += [y, s, *vdc.layer_norm_bwd(s, n["weight"], n["dy"], bias=n["bias"], dstream=n["dstream"])]
    for code in (torch.int8, torch.float8_e4m3fn):
        E = states[2][0].numel()
        codes = torch.zeros(5, E, dtype=torch.int8, device=DEV).view(code)
        scales = torch.zeros(5, (E + 63) // 64, device=DEV)
        vdc.state_quantize(states[2], codes, scales)
        vdc.state_dequantize(codes, scales, states[2])
        out += [codes.view(torch.int8), scales, states[2].clone()]
    return out


def test_same_bits_on_any_stream_and_in_graphs(vdc):
    sets = [_set(s) for s in (61, 71, 81)]
    eager = [[t.clone() for t in _everything(vdc, k, cu, n, dy, [s.clone() for s in st])] for k, cu, n, dy, st in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k, cu, n, dy, st = sets[0]
    with torch.cuda.stream(side):
        again = _everything(vdc, k, cu, n, dy, [s.clone() for s in st])
    side.synchronize()
    for a, b in zip(again, eager[0]):
        assert torch.equal(a, b)
    hold = [{q: t.clone() for q, t in d.items()} for d in (k, n)]
    hdy, hst = dy.clone(), [s.clone() for s in st]
    with torch.cuda.stream(side):
        _everything(vdc, hold[0], cu, hold[1], hdy, hst)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _everything(vdc, hold[0], cu, hold[1], hdy, hst)
    for rep in (0, 1, 2, 0):
        k, _, n, dy, st = sets[rep]
        for h, d in zip(hold, (k, n)):
            for q in h:
                h[q].copy_(d[q])
        hdy.copy_(dy)
        for a, b in zip(hst, st):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, eager[rep])):
            assert torch.equal(a, b), "replay of set %d: output %d" % (rep, i)
        _everything(vdc, k, cu, n, dy, [s.clone() for s in st])


@pytest.mark.parametrize("S,C", [(9000, 264), (33000, 1032), (40000, 40)])
def test_same_bits_whatever_finishes_first(vdc, S, C):
    """What a tile finds of those before it differs from run to run, its result
    does not; neither with garbage in the workspace, nor beside other work."""
    k, _, cu = recur_inputs(91, [S // 3, S - S // 3], C, device=DEV, low=0.99, high=0.99999)
    dy = Maker(92, DEV).normal(S, C)
    y0, keep0 = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    want = vdc.gated_recurrence_bwd(*head(k), cu, dy, keep0, z=k["z"])
    side, noise = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    for rep in range(6):
        ws = [torch.full((vdc.gated_recurrence_workspace_bytes(d, S, C),), 0xA5 if rep % 2 else 0, dtype=torch.uint8,
                         device=DEV) for d in ("fwd", "bwd")]
        torch.cuda.synchronize()
        if rep > 2:
            with torch.cuda.stream(side):
                for _ in range(rep):
                    noise = noise * 1.0001
        y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True, workspace=ws[0])
        got = vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"], workspace=ws[1])
        assert torch.equal(y, y0) and torch.equal(keep, keep0)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_two_calls_at_once(vdc):
    """Calls on two streams with workspaces of their own."""
    sets = [_set(s, (3000, 5, 1200), 520) for s in (101, 111)]
    want = [_everything(vdc, k, cu, n, dy, [s.clone() for s in st]) for k, cu, n, dy, st in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        copies = [[s.clone() for s in st] for *_, st in sets]
        torch.cuda.synchronize()
        got = []
        for (k, cu, n, dy, _), st, stream in zip(sets, copies, streams):
            with torch.cuda.stream(stream):
                got.append(_everything(vdc, k, cu, n, dy, st))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


# ------------------------------------------------ tiles, documents, prompts --

@pytest.mark.parametrize("lengths", [[127], [128], [129], [64], [65], [128, 128], [127, 1, 128], [1, 255, 64], [256, 0, 1],
                                     [15, 1, 16, 17, 15, 64, 1, 1, 126], [2049], [130, 0, 0, 2000, 1]],
                         ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("C,gate", [(66, True), (257, False)])
def test_documents_around_tiles(vdc, lengths, C, gate):
    k, docs, cu = recur_inputs(121, lengths, C, device=DEV, gate=gate)
    n = len(lengths)
    st = Maker(122, DEV).normal(n, C, dtype=F32)
    resume = [j % 2 == 0 for j in range(n)]
    ref = L.Recurrence(*head(k), docs, k["z"], 8.0, st, list(range(n)), resume)
    own = st.clone()
    y = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=own, resume=torch.tensor(resume, device=DEV))
    close("y", y, ref.y, ref.ey)
    close("state", own, ref.after, ref.eafter)
    ref = L.Recurrence(*head(k), docs, k["z"])
    dy = Maker(123, DEV).normal(sum(lengths), C)
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    want = ref.grads(dy)
    for name, t in zip(("dx", "dr", "di", "ddecay", "dz"), vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])):
        if t is not None:
            close(name, t, *want[name])


@pytest.mark.parametrize("seed", range(4))
def test_many_documents(vdc, seed):
    g = torch.Generator().manual_seed(seed)
    lengths = [int(v) for v in torch.randint(0, (3, 9, 40, 2)[seed], (1500,), generator=g)]
    C = 40 + 31 * seed
    k, docs, cu = recur_inputs(131 + seed, lengths, C, device=DEV, wide=seed % 2 == 1, params=BF if seed == 2 else F32)
    n = len(lengths)
    st = Maker(141, DEV).normal(n + 9, C, dtype=F32)
    slots = torch.randperm(n + 9, generator=g)[:n]
    slots[5], slots[77] = -3, n + 9
    given = [int(s) if 0 <= s < n + 9 else -1 for s in slots]
    resume = torch.randint(0, 2, (n,), generator=g).bool()
    ref = L.Recurrence(*head(k), docs, k["z"], 8.0, st, given, resume.tolist())
    own = st.clone()
    y = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=own, state_index=slots.int().to(DEV), resume=resume.to(DEV))
    close("y", y, ref.y, ref.ey)
    close("state", own, ref.after, ref.eafter)


def test_prompts_in_parts_and_tokens_after_them(vdc):
    C, S = 200, 700
    k, docs, cu = recur_inputs(151, [S], C, device=DEV)
    ref = L.Recurrence(*head(k), docs, k["z"])
    for cuts in ([0, 1, S], [0, 300, 300, 301, S], [0, 128, 500, S]):
        state, ys = Maker(152, DEV).normal(1, C, dtype=F32), []
        for lo, hi in zip(cuts, cuts[1:]):
            part = [k[n][lo:hi] for n in ("x", "r", "i")]
            ys.append(vdc.gated_recurrence_fwd(*part, k["decay"], ints([0, hi - lo]), z=k["z"][lo:hi], state=state,
                                               resume=torch.tensor([lo > 0], device=DEV)))
        close("y", torch.cat(ys), ref.y, ref.ey)
        close("state", state[0], ref.h[-1], L.MORE * ref.eh[-1])
    state = torch.zeros(1, C, device=DEV)
    ys = [vdc.gated_recurrence_update(k["x"][t:t + 1], k["r"][t:t + 1], k["i"][t:t + 1], k["decay"], state,
                                      z=k["z"][t:t + 1]) for t in range(S)]
    close("y", torch.cat(ys), ref.y, ref.ey)


def test_documents_without_tokens(vdc):
    st = Maker(161, DEV).normal(6, 70, dtype=F32)
    own = st.clone()
    x = torch.zeros(0, 70, dtype=BF, device=DEV)
    y = vdc.gated_recurrence_fwd(x, x, x, torch.zeros(70, device=DEV), ints([0, 0, 0, 0]), state=own,
                                 state_index=ints([4, 1, 9]), resume=torch.tensor([False, True, False], device=DEV))
    want = st.clone()
    want[4] = 0
    assert y.shape == (0, 70) and torch.equal(own, want)


# ---------------------------------------------- masks, infinities and NaN --

LOW = [float("-inf"), torch.finfo(BF).min]


@pytest.mark.parametrize("low", LOW)
@pytest.mark.parametrize("junk", [0.0, float("inf"), float("nan")])
@pytest.mark.parametrize("lengths,C", [([5, 300, 1], 70), ([700], 200)])
def test_masked_tokens_are_not_there(vdc, lengths, C, low, junk):
    """Tokens with a closed decay gate leave the state exactly as it is, whatever
    their inputs hold, and have no gradients."""
    k, docs, cu = recur_inputs(171, lengths, C, device=DEV)
    S = sum(lengths)
    g = torch.Generator().manual_seed(1)
    masked = torch.rand(S, generator=g) < 0.4
    masked[:3] = True
    masked[-150:-20] = True
    masked = masked.to(DEV)
    k["r"][masked] = low
    clean = {n: t.clone() for n, t in k.items()}
    clean["x"][masked] = 0
    k["x"][masked] = junk
    if junk:
        k["i"][masked] = -junk
    dy = Maker(172, DEV).normal(S, C)
    st = Maker(173, DEV).normal(len(lengths), C, dtype=F32)
    resume = torch.ones(len(lengths), dtype=torch.bool, device=DEV)
    ref = L.Recurrence(*head(clean), docs, k["z"], 8.0, st, list(range(len(lengths))), [True] * len(lengths))
    own = st.clone()
    y = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=own, resume=resume)
    close("y", y, ref.y, ref.ey)
    close("state", own, ref.after, ref.eafter)
    ref = L.Recurrence(*head(clean), docs, k["z"]).grads(dy)
    _, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    dx, dr, di, dd, dz = vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])
    for name, t in (("dx", dx), ("dr", dr), ("di", di), ("ddecay", dd), ("dz", dz)):
        close(name, t, *ref[name])
    for t in (dx, dr, di):
        assert bool((t[masked] == 0).all())
    # one row at a time
    state = st[:1].repeat(S, 1)
    was = state.clone()
    vdc.gated_recurrence_update(*head(k), state, z=k["z"])
    assert torch.equal(state[masked], was[masked])


def test_rows_that_are_masked_altogether(vdc):
    C, S = 130, 400
    k, _, cu = recur_inputs(181, [S], C, device=DEV)
    k["r"][:], k["x"][:] = float("-inf"), float("nan")
    st = Maker(182, DEV).normal(1, C, dtype=F32)
    own = st.clone()
    y = vdc.gated_recurrence_fwd(*head(k), cu, state=own, resume=torch.ones(1, dtype=torch.bool, device=DEV))
    assert torch.equal(own, st) and torch.equal(y, st.to(BF).expand(S, C))
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, keep=True)
    assert bool((y == 0).all())
    got = vdc.gated_recurrence_bwd(*head(k), cu, torch.ones_like(y), keep)
    for t in got[:4]:
        assert bool((t == 0).all())


def test_infinities_and_nan_stay_in_their_documents(vdc):
    lengths, C = [40, 90, 700, 70], 68
    k, _, cu = recur_inputs(191, lengths, C, device=DEV)
    S = sum(lengths)
    dy = Maker(192, DEV).normal(S, C)
    y0, keep0 = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    g0 = vdc.gated_recurrence_bwd(*head(k), cu, dy, keep0, z=k["z"])
    bad = {n: t.clone() for n, t in k.items()}
    bad["x"][60, 3], bad["r"][100, 5], bad["x"][500, 7], bad["i"][129, 9] = (float("nan"), float("nan"), float("inf"),
                                                                              float("nan"))
    y, keep = vdc.gated_recurrence_fwd(*head(bad), cu, z=k["z"], keep=True)
    assert bool(y[60:130, 3].isnan().all()) and bool(y[100:130, 5].isnan().all()) and bool(y[129, 9].isnan())
    assert not bool(torch.isfinite(y[500:600, 7]).any())
    touched = torch.zeros(S, C, dtype=torch.bool, device=DEV)
    touched[40:130, [3, 5, 9]] = True
    touched[130:830, 7] = True
    assert torch.equal(y[~touched], y0[~touched])
    bdy = dy.clone()
    bdy[70, 20] = float("nan")
    touched[40:130, 20] = True
    got = vdc.gated_recurrence_bwd(*head(bad), cu, bdy, keep, z=k["z"])
    for j in (0, 1, 2, 4):
        assert torch.equal(got[j][~touched], g0[j][~touched])
    cols = torch.ones(C, dtype=torch.bool, device=DEV)
    cols[[3, 5, 7, 9, 20]] = False
    assert torch.equal(got[3][cols], g0[3][cols])


def test_decays_at_the_ends_of_the_range(vdc):
    """A decay that is too strong or too weak to be told from 0 and 1, and a gate
    that is far open or closed: finite and within the bounds."""
    S, C = 300, 64
    k, docs, cu = recur_inputs(201, [S], C, device=DEV)
    k["decay"] = torch.linspace(-100, 90, C, device=DEV)
    k["r"] = torch.linspace(-80, 80, S, device=DEV).to(BF)[:, None].expand(S, C).contiguous()
    dy = Maker(202, DEV).normal(S, C)
    ref = L.Recurrence(*head(k), docs, k["z"])
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    # softplus(decay) and u count as 0 below the normal numbers: a token with u up to
    # 16 * 2^-126 may add nothing, where m = sqrt(u) is 2^-61 at most.  Up to S
    # tokens' worth of that reaches an output, times inputs and gradients: their
    # largest products of |x| sigmoid(i), |dy| and |z| are below 5 * 5 * 5 < 2^7.
    # The decay's gradient sums S of these.
    assert max(float(t.abs().max()) for t in (k["x"], dy, k["z"])) < 5
    lost = S * 2.0 ** (7 - 61)
    close("y", y, ref.y, ref.ey + lost)
    want = ref.grads(dy)
    for name, t in zip(("dx", "dr", "di", "ddecay", "dz"), vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])):
        close(name, t, want[name][0], want[name][1] + (S if name == "ddecay" else 1) * lost)


def test_layer_norm_of_unusual_rows(vdc):
    k = norm_inputs(211, 9, 700, device=DEV)
    s = (k["x"].float() + k["residual"].float()).to(BF)
    s[0] = 3.0                       # no variance
    s[1] *= 1e-4                     # little, against eps
    s[2] = 1000.0
    s[2, ::7] = 1008.0               # a mean far from 0
    s[3, 0] = 3e38                   # one value that is the whole of it
    ref = L.LayerNorm(s, k["weight"], k["bias"])
    y, same = vdc.layer_norm_fwd(s, k["weight"], bias=k["bias"])
    assert same is s
    rows = [0, 1, 2, 4, 5, 6, 7, 8]
    close("y", y[rows], ref.y[rows], ref.ey[rows])
    s[3] = 1.0
    s[4, 5], s[5, 6] = float("nan"), float("inf")
    y, _ = vdc.layer_norm_fwd(s, k["weight"], bias=k["bias"])
    assert bool(y[4].isnan().all()) and bool(y[5].isnan().any())
    rest = [0, 1, 2, 3, 6, 7, 8]
    ref = L.LayerNorm(s[rest], k["weight"], k["bias"])
    close("y", y[rest], ref.y, ref.ey)
    dx, _, _ = vdc.layer_norm_bwd(s, k["weight"], k["dy"], bias=k["bias"])
    close("dx", dx[rest], *ref.grads(k["dy"][rest])["dx"])


# ------------------------------------------------- prefix sums, own buffers --

@pytest.mark.parametrize("S,C", [(3, 64), (100, 72), (700, 136)])
@pytest.mark.parametrize("past", [1, 50, 2 ** 31 - 1])
def test_an_end_past_the_last_token(vdc, S, C, past):
    """Comes out as a document that ends with the row and leaves its slot alone."""
    k, _, _ = recur_inputs(221, [S], C, device=DEV)
    st = Maker(222, DEV).normal(2, C, dtype=F32)
    want, got, go_on = st.clone(), st.clone(), torch.ones(2, dtype=torch.bool, device=DEV)
    y = vdc.gated_recurrence_fwd(*head(k), ints([0, S // 3, S]), z=k["z"], state=want, resume=go_on)
    bad = vdc.gated_recurrence_fwd(*head(k), ints([0, S // 3, min(S + past, 2 ** 31 - 1)]), z=k["z"], state=got,
                                   resume=go_on)
    assert torch.equal(bad, y) and torch.equal(got[0], want[0]) and torch.equal(got[1], st[1])


@pytest.mark.parametrize("ends", [[5, 3, 700], [0, -7, 700], [0, 900, 100, 700], [700, 0], [0, 0], [3], [-2 ** 31, 2 ** 31 - 1]])
def test_prefix_sums_in_no_order(vdc, ends):
    """The results are unspecified, the call ends inside its buffers."""
    S, C = 700, 200
    k, _, _ = recur_inputs(231, [S], C, device=DEV)
    n = len(ends) - 1
    guard = torch.full((n + 2, C), 7.0, device=DEV)
    cu = ints(ends if n else ends * 2)
    n = max(n, 1)
    guard = torch.full((n + 2, C), 7.0, device=DEV)
    vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], state=guard[1:n + 1], resume=torch.ones(n, dtype=torch.bool, device=DEV))
    y, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    vdc.gated_recurrence_bwd(*head(k), cu, y, keep, z=k["z"])
    torch.cuda.synchronize()
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())


def test_own_outputs_and_refused_shapes(vdc):
    k, _, cu = recur_inputs(241, [200], 72, device=DEV)
    n = norm_inputs(242, 200, 72, device=DEV)
    out, keep = torch.full((200, 72), 5.0, dtype=BF, device=DEV), torch.zeros(4, 72, device=DEV)
    y, kept = vdc.gated_recurrence_fwd(*head(k), cu, keep=keep, out=out)
    assert y is out and kept is keep
    assert torch.equal(y, vdc.gated_recurrence_fwd(*head(k), cu))
    stream = torch.empty_like(out)
    a, b = vdc.layer_norm_fwd(n["x"], n["weight"], residual=n["residual"], out=out, stream_out=stream)
    assert a is out and b is stream
    state = torch.zeros(3, 72, device=DEV)
    codes, scales = torch.zeros(2, 72, dtype=torch.int8, device=DEV), torch.zeros(2, 2, device=DEV)
    for call, error in (
            (lambda: vdc.gated_recurrence_fwd(*head(k), cu, keep=True, state=state), ValueError),
            (lambda: vdc.gated_recurrence_fwd(*head(k), cu, resume=torch.zeros(1, dtype=torch.bool, device=DEV)), ValueError),
            (lambda: vdc.gated_recurrence_fwd(k["x"], k["r"][:100], k["i"], k["decay"], cu), ValueError),
            (lambda: vdc.gated_recurrence_fwd(k["x"], k["r"].float(), k["i"], k["decay"], cu), TypeError),
            (lambda: vdc.gated_recurrence_fwd(k["x"], k["r"].t().contiguous().t(), k["i"], k["decay"], cu), ValueError),
            (lambda: vdc.gated_recurrence_fwd(*head(k), cu.long()), ValueError),
            (lambda: vdc.gated_recurrence_fwd(*head(k), cu, scale=-1.0), vdc.VdcError),
            (lambda: vdc.gated_recurrence_bwd(*head(k), cu, k["x"], keep[:3]), ValueError),
            (lambda: vdc.gated_recurrence_bwd(*head(k), cu, k["x"], keep.cpu()), ValueError),
            (lambda: vdc.gated_recurrence_update(*head(k), state), ValueError),
            (lambda: vdc.layer_norm_fwd(n["x"], n["weight"][:5]), ValueError),
            (lambda: vdc.layer_norm_fwd(n["x"], n["weight"], stream_out=stream), ValueError),
            (lambda: vdc.layer_norm_fwd(n["x"], n["weight"], eps=-1.0), vdc.VdcError),
            (lambda: vdc.layer_norm_fwd(n["x"][:, :0], n["weight"][:0]), vdc.VdcError),
            (lambda: vdc.state_quantize(state, codes, scales), ValueError),
            (lambda: vdc.state_quantize(state, codes[:, :70], scales, state_index=ints([0])), ValueError),
            (lambda: vdc.state_quantize(state, codes.float(), scales, state_index=ints([0])), TypeError),
            (lambda: vdc.state_quantize(state.t(), codes, scales), ValueError),
            (lambda: vdc.state_dequantize(codes, scales, state, pool_index=ints([0]), state_index=ints([0, 1])),
             ValueError)):
        with pytest.raises(error):
            call()


def test_rows_far_apart(vdc):
    """Row strides at their limit."""
    S, C, stride = 20, 64, 1 << 25
    wide = torch.empty(S * stride, dtype=BF, device=DEV)
    k, docs, cu = recur_inputs(251, [S], C, device=DEV)
    far = {}
    for j, n in enumerate(("x", "r", "i", "z")):
        far[n] = wide.as_strided((S, C), (stride, 1), j * 128)
        far[n].copy_(k[n])
    y = vdc.gated_recurrence_fwd(far["x"], far["r"], far["i"], k["decay"], cu, z=far["z"])
    assert torch.equal(y, vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"]))
    dy = Maker(252, DEV).normal(S, C)
    _, keep = vdc.gated_recurrence_fwd(*head(k), cu, z=k["z"], keep=True)
    for a, b in zip(vdc.gated_recurrence_bwd(far["x"], far["r"], far["i"], k["decay"], cu, dy, keep, z=far["z"]),
                    vdc.gated_recurrence_bwd(*head(k), cu, dy, keep, z=k["z"])):
        assert torch.equal(a, b)
    with pytest.raises(Exception):
        vdc.gated_recurrence_fwd(wide.as_strided((2, C), (stride + 1, 1)), k["r"][:2], k["i"][:2], k["decay"], ints([0, 2]))


def test_offsets_past_32_bits(vdc):
    """The last document of a long row, whose first token begins a tile, is bit
    for bit the document alone."""
    C, last = 4096, 1000
    first = (2 ** 31 // C // 128 + 3) * 128
    S = first + last
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.randn(S, C, device=DEV, generator=g, dtype=BF)
    decay = Maker(261, DEV).uniform(C, lo=-9.0, hi=-4.0)
    cu = ints([0, 100, first, S])
    st = torch.zeros(3, C, device=DEV)
    one = torch.zeros(1, C, device=DEV)
    tail = x[first:]
    y = vdc.gated_recurrence_fwd(x, x, x, decay, cu, z=x, state=st)
    assert torch.equal(y[first:], vdc.gated_recurrence_fwd(tail, tail, tail, decay, ints([0, last]), z=tail, state=one))
    assert torch.equal(st[2], one[0])
    y, keep = vdc.gated_recurrence_fwd(x, x, x, decay, cu, z=x, keep=True)
    got = vdc.gated_recurrence_bwd(x, x, x, decay, cu, x, keep, z=x)
    _, keep = vdc.gated_recurrence_fwd(tail, tail, tail, decay, ints([0, last]), z=tail, keep=True)
    want = vdc.gated_recurrence_bwd(tail, tail, tail, decay, ints([0, last]), tail, keep, z=tail)
    for j in (0, 1, 2, 4):
        assert torch.equal(got[j][first:], want[j])
    del got, want, y, keep
    w = torch.ones(C, device=DEV)
    y, s = vdc.layer_norm_fwd(x, w, residual=x)
    assert torch.equal(y[first:], vdc.layer_norm_fwd(tail, w, residual=tail)[0])
    dx, _, _ = vdc.layer_norm_bwd(s, w, x, dstream=x)
    assert torch.equal(dx[first:], vdc.layer_norm_bwd(s[first:], w, tail, dstream=tail)[0])


def test_caches_past_32_bits(vdc):
    C, slots = 65536, 2 ** 31 // 65536 + 9
    state = torch.zeros(slots, C, device=DEV)
    row = Maker(271, DEV).normal(2, C, dtype=F32)
    state[-2:] = row
    k, _, _ = recur_inputs(272, [2], C, device=DEV)
    own = row.clone()
    y = vdc.gated_recurrence_update(*head(k), state, z=k["z"], state_index=ints([slots - 2, slots - 1]))
    assert torch.equal(y, vdc.gated_recurrence_update(*head(k), own, z=k["z"])) and torch.equal(state[-2:], own)
    state[-2:] = row
    y = vdc.gated_recurrence_fwd(*head(k), ints([0, 1, 2]), state=state, state_index=ints([slots - 2, slots - 1]),
                                 resume=torch.ones(2, dtype=torch.bool, device=DEV))
    own = row.clone()
    assert torch.equal(y, vdc.gated_recurrence_fwd(*head(k), ints([0, 1, 2]), state=own,
                                                   resume=torch.ones(2, dtype=torch.bool, device=DEV)))
    assert torch.equal(state[-2:], own)
    codes, scales = torch.zeros(slots, C, dtype=torch.int8, device=DEV), torch.zeros(slots, C // 64, device=DEV)
    vdc.state_quantize(state, codes, scales, state_index=ints([slots - 1]), pool_index=ints([slots - 1]))
    q, scale = L.put_aside(own[1].double(), torch.int8)
    assert torch.equal(codes[-1].float(), q.float()) and torch.equal(scales[-1], scale)
    vdc.state_dequantize(codes, scales, state, pool_index=ints([slots - 1]), state_index=ints([slots - 2]))
    assert torch.equal(state[-2], L.take_back(q, scale, F32))
    assert not bool(state[:-2].any()) and torch.equal(state[-1], own[1])


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_states_at_any_alignment(vdc, shift):
    """Vectors where the buffers allow them, the same values where not."""
    m, E = Maker(281, DEV), 256
    for dtype in (F32, BF):
        flat = torch.zeros(6 * E + 8, dtype=dtype, device=DEV)
        state = flat[shift:shift + 6 * E].view(6, E)
        state.copy_(m.normal(6, E, dtype=F32))
        for code in (torch.int8, torch.float8_e4m3fn):
            raw = torch.zeros(6 * E + 8, dtype=torch.int8, device=DEV)
            codes, scales = raw[shift:shift + 6 * E].view(6, E).view(code), torch.zeros(6, E // 64, device=DEV)
            was = state.clone()
            vdc.state_quantize(state, codes, scales)
            for j in range(6):
                q, scale = L.put_aside(was[j].double(), code)
                assert torch.equal(codes[j].float(), q.float()) and torch.equal(scales[j], scale)
            back = torch.zeros_like(flat)[shift:shift + 6 * E].view(6, E)
            vdc.state_dequantize(codes, scales, back)
            assert torch.equal(back, torch.stack([L.take_back(codes[j].float(), scales[j], dtype) for j in range(6)]))
            assert not bool(raw[:shift].any()) and not bool(raw[shift + 6 * E:].any())
        assert not bool(flat[:shift].any()) and not bool(flat[shift + 6 * E:].any())


def test_memory_that_is_not_there_is_its_own_error(vdc):
    """An output that does not fit raises what torch raises, and the next call works."""
    x = torch.randn(4096, 4096, device=DEV).bfloat16()
    w = torch.ones(4096, device=DEV)
    want = vdc.layer_norm_fwd(x, w)[0]
    torch.cuda.empty_cache()
    total = torch.cuda.mem_get_info()[1]
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            held = [vdc.layer_norm_fwd(x, w)[0] for _ in range(64)]  # reserved memory has room for some
            del held
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(vdc.layer_norm_fwd(x, w)[0], want)


def test_more_rows_than_one_launch_has_waves_for(vdc):
    """2^24 rows and some of one channel, in turns of 2^24: each row is its own sequence."""
    rows = (1 << 24) + 77
    x = torch.randn(rows, 1, device=DEV).bfloat16()
    r, i = torch.randn(rows, 1, device=DEV).bfloat16(), torch.randn(rows, 1, device=DEV).bfloat16()
    decay = torch.full((1,), 0.5, device=DEV)
    state = torch.randn(rows, 1, device=DEV)
    at = torch.cat([torch.arange(200, device=DEV), torch.arange(rows - 200, rows, device=DEV)])
    some = state[at].clone()
    want = vdc.gated_recurrence_update(x[at], r[at], i[at], decay, some)
    got = vdc.gated_recurrence_update(x, r, i, decay, state)
    assert torch.equal(got[at], want) and torch.equal(state[at], some)
