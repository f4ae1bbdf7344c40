"""Infinities and NaN of one document do not reach another, nor the tokens that
the formulas keep from them, through what the scan's kernels share: chunks of the
packed row that a document's start cuts, states past the last of a channel and
columns past the last of a group."""
import pytest
import torch

from ssm_cases import Maker, scan_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")
TOKENS = {"dx": 0, "ddt": 1, "dB": 3, "dC": 4, "dz": 6}  # gradients by token, and where they are


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


# One document each with and without room for more states, groups of 64
# channels and others.
SIZES = [(64, 16, 1), (64, 13, 1), (130, 16, 2), (130, 5, 2), (65, 24, 1), (40, 40, 1), (520, 64, 2)]


@pytest.mark.parametrize("C,N,G", SIZES)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("which", ["x", "dt", "B", "C", "z", "dy"])
def test_gradients_of_the_documents_around(vdc, C, N, G, value, which):
    """The second document starts and ends where chunks do (multiples of 32
    tokens are multiples of every chunk's length here); its first, a middle and
    its last token have the value in one channel, or in one state."""
    lengths = [96, 64, 64]
    lo, hi = 96, 160
    k, _, cu = scan_inputs(501, lengths, C, N, G, device=DEV)
    k["dy"] = Maker(502, DEV).normal(sum(lengths), C)
    run = lambda q: (vdc.selective_scan_fwd(*_head(q), cu, **_rest(q)),  # noqa: E731
                     vdc.selective_scan_bwd(*_head(q), cu, q["dy"], **_rest(q)))
    clean, cleang = run(k)
    bad = dict(k)
    bad[which] = k[which].clone()
    for t in (lo, lo + 17, hi - 1):
        bad[which][t].view(-1)[3] = value
    y, got = run(bad)
    out = torch.ones(sum(lengths), dtype=torch.bool, device=DEV)
    out[lo:hi] = False
    assert torch.equal(y[out], clean[out])
    for name, i in TOKENS.items():
        assert torch.equal(got[i][out], cleang[i][out]), name


@pytest.mark.parametrize("C,N,G", SIZES)
@pytest.mark.parametrize("t", [128, 133])
def test_an_endless_step_cuts_its_document(vdc, C, N, G, t):
    """A step of +inf forgets all that was: the gradients of the tokens before
    it are those of a document that ends there."""
    lengths, dy = [96, 104, 24], Maker(512, DEV).normal(224, C)
    k, _, cu = scan_inputs(511, lengths, C, N, G, device=DEV)
    cut = torch.tensor([0, 96, t, 200, 224], dtype=torch.int32, device=DEV)
    want = vdc.selective_scan_bwd(*_head(k), cut, dy, **_rest(k))
    k["dt"] = k["dt"].clone()
    k["dt"][t] = INF
    got = vdc.selective_scan_bwd(*_head(k), cu, dy, **_rest(k))
    for name, i in TOKENS.items():
        assert torch.equal(got[i][:t], want[i][:t]), name
