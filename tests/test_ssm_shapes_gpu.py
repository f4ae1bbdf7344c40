"""The state space layer's operators where sizes decide what runs: prompts at
the border between one launch and three, chunks of many blocks, many documents,
prompts in parts, caches and strides past 32 bits, the caller's own outputs and
workspaces."""
import pytest
import torch

import ssm_ref as R
from ssm_cases import Maker, scan_inputs

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
DEV = "cuda:0"
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")


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


def _ref(k, docs, **more):
    return R.Scan(*_head(k), docs, k["D"], k["z"], k["dt_bias"], **more)


@pytest.mark.parametrize("lengths", [[80], [81], [39, 0, 41], [7, 72, 0, 2], [8] * 10, [88], [95, 1]])
@pytest.mark.parametrize("N", [5, 16, 48])
def test_scan_fwd_around_one_launch(vdc, lengths, N):
    C = 70
    k, docs, cu = scan_inputs(301, lengths, C, N, 2, device=DEV)
    n = len(lengths)
    state = Maker(302, DEV).normal(n, C, N, dtype=F32)
    resume = [i % 2 == 0 for i in range(n)]
    ref = _ref(k, docs, state=state, slots=list(range(n)), resume=resume)
    y = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k), state=state, resume=torch.tensor(resume, device=DEV))
    R.close("y", y, ref.y, ref.ey)
    R.close("state", state, ref.after, ref.eafter)


@pytest.mark.parametrize("N,S", [(5, 160), (5, 161), (16, 224), (16, 225), (24, 320), (24, 321), (64, 512),
                                 (64, 513)])
def test_scan_fwd_around_longer_launches(vdc, N, S):
    """Documents that end with the parts of a row, inside them, and run over
    several; resumed ones among them."""
    C, lengths = 40, [20, 0, S // 2 - 20, 3, 0, 1, S - S // 2 - 4, 0]
    k, docs, cu = scan_inputs(305, lengths, C, N, 1, device=DEV, wide=True)
    n = len(lengths)
    for flip in (0, 1):
        state = Maker(306, DEV).normal(n, C, N, dtype=F32)
        resume = [i % 2 == flip for i in range(n)]
        ref = _ref(k, docs, state=state, slots=list(range(n)), resume=resume)
        y = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k), state=state,
                                   resume=torch.tensor(resume, device=DEV))
        R.close("y", y, ref.y, ref.ey)
        R.close("state", state, ref.after, ref.eafter)


def test_scan_chunks_of_many_blocks(vdc):
    """32768 channels leave few chunks, each of many blocks; three of the 512
    groups are held to the definition."""
    C, N, G = 32768, 16, 512
    lengths = [700, 0, 1, 211, 588]
    k, docs, cu = scan_inputs(311, lengths, C, N, G, device=DEV)
    dy = Maker(312, DEV).normal(1500, C)
    y = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k))
    got = dict(zip(GRADS, vdc.selective_scan_bwd(*_head(k), cu, dy, **_rest(k))))
    for g in (0, 300, 511):
        c, per = slice(g * 64, g * 64 + 64), slice(g, g + 1)
        part = {
            "x": k["x"][:, c], "dt": k["dt"][:, c], "z": k["z"][:, c], "A": k["A"][c], "D": k["D"][c],
            "dt_bias": k["dt_bias"][c], "B": k["B"][:, per], "C": k["C"][:, per]}
        ref = _ref(part, docs)
        R.close("y", y[:, c], ref.y, ref.ey)
        for name, (want, bound) in ref.grads(dy[:, c]).items():
            t = got[name]
            t = t[:, per] if name in ("dB", "dC") else t[c] if name in ("dA", "dD", "ddt_bias") else t[:, c]
            R.close(name, t, want, bound)


@pytest.mark.parametrize("seed", [1, 2])
def test_scan_many_documents(vdc, seed):
    """Thousands of documents, most of them empty or of one token."""
    C, N = 16, 8
    g = torch.Generator().manual_seed(seed)
    lengths = torch.randint(0, 3, (5000,), generator=g).tolist()
    for i in torch.randint(0, 5000, (8,), generator=g).tolist():
        lengths[i] = 60
    k, docs, cu = scan_inputs(320 + seed, lengths, C, N, device=DEV)
    state = Maker(321, DEV).normal(5000, C, N, dtype=F32)
    resume = [i % 3 == 0 for i in range(5000)]
    ref = _ref(k, docs, state=state, slots=list(range(5000)), resume=resume)
    y = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k), state=state, resume=torch.tensor(resume, device=DEV))
    R.close("y", y, ref.y, ref.ey)
    R.close("state", state, ref.after, ref.eafter)
    dy = Maker(322, DEV).normal(k["x"].shape[0], C)
    want = _ref(k, docs).grads(dy)
    for name, t in zip(GRADS, vdc.selective_scan_bwd(*_head(k), cu, dy, **_rest(k))):
        R.close(name, t, *want[name])


@pytest.mark.parametrize("C,N,G", [(66, 16, 1), (40, 12, 2), (24, 64, 1)])
def test_prompts_in_parts_and_tokens_after_them(vdc, C, N, G):
    """The state carries a sequence over any cuts: the outputs stay within the
    bounds of the whole sequence's."""
    k, docs, _ = scan_inputs(331, [260], C, N, G, device=DEV)
    ref = _ref(k, docs)
    state = torch.full((3, C, N), float("nan"), device=DEV)
    slot = torch.tensor([1], dtype=torch.int32, device=DEV)
    ys, lo = [], 0
    for hi in (33, 33, 150, 151, 230):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV)
        part = {n: (k[n] if n in ("A", "D", "dt_bias") else k[n][lo:hi]) for n in k}
        ys.append(vdc.selective_scan_fwd(*_head(part), cu, **_rest(part), state=state, state_index=slot,
                                         resume=torch.tensor([lo > 0], device=DEV)))
        lo = hi
    for t in range(230, 260):
        part = {n: (k[n] if n in ("A", "D", "dt_bias") else k[n][t:t + 1]) for n in k}
        ys.append(vdc.selective_update(*_head(part), state, **_rest(part), state_index=slot))
    R.close("y", torch.cat(ys), ref.y, ref.ey)
    R.close("state", state[1], ref.h[-1], ref.eh[-1])
    assert bool(torch.isnan(state[0]).all()) and bool(torch.isnan(state[2]).all())


def test_last_token_past_the_range_leaves_decay_gradients(vdc):
    """dA does not read a sequence's last input: an infinity there leaves it as
    it was, also where the row of tokens ends inside a block."""
    k, _, cu = scan_inputs(341, [13], 64, 16, device=DEV)
    dy = Maker(342, DEV).normal(13, 64)
    clean = vdc.selective_scan_bwd(*_head(k), cu, dy, **_rest(k))
    x = k["x"].clone()
    x[12, 7] = float("inf")
    got = vdc.selective_scan_bwd(x, *_head(k)[1:], cu, dy, **_rest(k))
    assert torch.equal(got[2], clean[2])


def test_rows_far_apart(vdc):
    """Activations cut out of rows 1 MB long: offsets past 32 bits."""
    S, C, N, wide = 4600, 136, 16, 2 ** 19 - 8
    k, _, cu = scan_inputs(351, [4000, 600], C, N, device=DEV)
    dy = Maker(352, DEV).normal(S, C)
    big = torch.empty(S, wide, dtype=BF, device=DEV)
    assert big.numel() * 2 > 2 ** 32
    far, at = dict(k), 0
    for n in ("x", "dt", "z"):
        big[:, at:at + C] = k[n]
        far[n] = big[:, at:at + C]
        at += 200
    for n in ("B", "C"):
        big[:, at:at + N] = k[n][:, 0]
        far[n] = big[:, at:at + N].unflatten(1, (1, N))
        at += 200
    big[:, at:at + C] = dy
    fdy = big[:, at:at + C]
    assert torch.equal(vdc.selective_scan_fwd(*_head(far), cu, **_rest(far)),
                       vdc.selective_scan_fwd(*_head(k), cu, **_rest(k)))
    for a, b in zip(vdc.selective_scan_bwd(*_head(far), cu, fdy, **_rest(far)),
                    vdc.selective_scan_bwd(*_head(k), cu, dy, **_rest(k))):
        assert torch.equal(a, b)
    w = k["D"]
    assert torch.equal(vdc.group_norm_silu_fwd(far["x"], w, 17, z=far["z"]),
                       vdc.group_norm_silu_fwd(k["x"], w, 17, z=k["z"]))
    for a, b in zip(vdc.group_norm_silu_bwd(far["x"], w, 17, fdy, z=far["z"]),
                    vdc.group_norm_silu_bwd(k["x"], w, 17, dy, z=k["z"])):
        assert a is b or torch.equal(a, b)


def test_caches_past_32_bits(vdc):
    """The last slots of caches of more than 4 GiB."""
    m, C, N, slots = Maker(361, DEV), 2048, 16, 33000
    cache = torch.empty(slots, C, N, device=DEV)
    assert cache.numel() * 4 > 2 ** 32
    k, _, cu = scan_inputs(362, [100, 28], C, N, device=DEV)
    first = m.normal(2, C, N, dtype=F32)
    small = first.clone()
    cache[-2:] = first
    index = torch.tensor([slots - 2, slots - 1], dtype=torch.int32, device=DEV)
    resume = torch.ones(2, dtype=torch.bool, device=DEV)
    a = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k), state=cache, state_index=index, resume=resume)
    b = vdc.selective_scan_fwd(*_head(k), cu, **_rest(k), state=small, resume=resume)
    assert torch.equal(a, b) and torch.equal(cache[-2:], small)
    part = {n: (k[n] if n in ("A", "D", "dt_bias") else k[n][:2]) for n in k}
    a = vdc.selective_update(*_head(part), cache, **_rest(part), state_index=index)
    b = vdc.selective_update(*_head(part), small, **_rest(part))
    assert torch.equal(a, b) and torch.equal(cache[-2:], small)
    del cache
    C, slots = 4096, 180000
    cache = torch.empty(slots, 3, C, dtype=BF, device=DEV)
    assert cache.numel() * 2 > 2 ** 32
    first = m.normal(2, 3, C)
    small = first.clone()
    cache[-2:] = first
    index = torch.tensor([slots - 1, slots - 2], dtype=torch.int32, device=DEV)
    small = small.flip(0).contiguous()
    x, w = m.normal(128, C), m.normal(C, 4, dtype=F32)
    a = vdc.conv1d_prefill(x, w, cu, cache, state_index=index, resume=resume)
    b = vdc.conv1d_prefill(x, w, cu, small, resume=resume)
    assert torch.equal(a, b) and torch.equal(cache[-2:].flip(0), small)
    a = vdc.conv1d_update(x[:2], cache, w, state_index=index)
    b = vdc.conv1d_update(x[:2], small, w)
    assert torch.equal(a, b) and torch.equal(cache[-2:].flip(0), small)


def test_own_outputs_and_workspaces(vdc):
    """The caller's outputs and workspaces, whatever they held, give the same
    bits, and a workspace too small is refused before anything runs."""
    k, _, cu = scan_inputs(371, [300, 45], 136, 16, device=DEV)
    dy = Maker(372, DEV).normal(345, 136)
    head, rest = _head(k), _rest(k)
    want = vdc.selective_scan_fwd(*head, cu, **rest)
    wantg = vdc.selective_scan_bwd(*head, cu, dy, **rest)
    wantn = vdc.group_norm_silu_bwd(k["x"], k["D"], 4, dy, z=k["z"])
    need = [vdc.selective_scan_workspace_bytes("fwd", 345, 136, 16), vdc.selective_scan_workspace_bytes("bwd", 345, 136, 16),
            vdc.group_norm_silu_workspace_bytes(345, 136, 4)]
    for fill in (0x00, 0x7f, 0xff):
        ws = [torch.full((n,), fill, dtype=torch.uint8, device=DEV) for n in need]
        out = torch.full_like(want, float("nan"))
        assert vdc.selective_scan_fwd(*head, cu, **rest, out=out, workspace=ws[0]) is out
        assert torch.equal(out, want)
        for a, b in zip(vdc.selective_scan_bwd(*head, cu, dy, **rest, workspace=ws[1]), wantg):
            assert torch.equal(a, b)
        for a, b in zip(vdc.group_norm_silu_bwd(k["x"], k["D"], 4, dy, z=k["z"], workspace=ws[2]), wantn):
            assert a is b or torch.equal(a, b)
    for n in need:
        small = torch.empty(n - 1, dtype=torch.uint8, device=DEV)
        with pytest.raises(vdc.VdcError):
            if n == need[0]:
                vdc.selective_scan_fwd(*head, cu, **rest, workspace=small)
            elif n == need[1]:
                vdc.selective_scan_bwd(*head, cu, dy, **rest, workspace=small)
            else:
                vdc.group_norm_silu_bwd(k["x"], k["D"], 4, dy, z=k["z"], workspace=small)


@pytest.mark.parametrize("S,C,G", [(70, 7, 1), (33, 63, 7), (700, 65, 1), (40, 4 * 129, 4), (21, 3 * 513, 3), (9, 1025, 1),
                                   (600, 2047, 1), (5, 4099, 1), (9, 8193, 1), (5, 10007, 1), (3, 16384, 1)])
@pytest.mark.parametrize("gate,shift", [(True, 1), (False, 0), (True, 0)])
def test_norm_groups_of_any_size(vdc, S, C, G, gate, shift):
    """Groups that end in a part of a vector, at every size of a team, on
    aligned and unaligned rows; nothing outside the rows is written."""
    m = Maker(381, DEV)
    cut = lambda: m.normal(S, C + shift)[:, shift:]  # noqa: E731
    x, z, dy = cut(), cut() if gate else None, cut()
    w, b = m.uniform(C, lo=0.5, hi=1.5), m.normal(C, std=0.1, dtype=F32)
    ref = R.Norm(x, w, G, b, z)
    room = torch.full((S * C + 64,), 7.0, dtype=BF, device=DEV)
    out = room[32:32 + S * C].view(S, C)
    R.close("y", vdc.group_norm_silu_fwd(x, w, G, bias=b, z=z, out=out), ref.y, ref.ey)
    assert bool((room[:32] == 7).all()) and bool((room[32 + S * C:] == 7).all())
    want = ref.grads(dy)
    for name, t in zip(("dx", "dweight", "dbias", "dz"), vdc.group_norm_silu_bwd(x, w, G, dy, bias=b, z=z)):
        if t is not None:
            R.close(name, t, *want[name])
