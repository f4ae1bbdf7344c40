"""Prefix sums that do not end with the row.  The results are unspecified but
the kernels stay inside their buffers: a document whose end lies past the last
token comes out as one that ends with it and leaves its slot alone, and tokens
past the last document's end as a document of their own."""
import pytest
import torch

from ssm_cases import Maker, scan_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def vdc():
    import varlen_depthwise_causal_amd as v
    return v


def _run(vdc, k, ends, state, resume=True):
    cu = torch.tensor(ends, dtype=torch.int32, device=DEV)
    head = [k[i] for i in ("x", "dt", "A", "B", "C")]
    rest = {i: k[i] for i in ("D", "z", "dt_bias")}
    n = len(ends) - 1
    return vdc.selective_scan_fwd(*head, cu, **rest, state=state,
                                  resume=torch.full((n,), resume, dtype=torch.bool, device=DEV))


# Rows of one launch, of many chunks, and of one chunk that takes no first pass.
@pytest.mark.parametrize("S,C,N", [(3, 64, 16), (100, 72, 5), (700, 72, 16), (700, 40, 64), (200, 262144, 8)])
@pytest.mark.parametrize("past", [1, 50, 2 ** 31 - 1])
def test_an_end_past_the_last_token(vdc, S, C, N, past):
    k, _, _ = scan_inputs(801, [S], C, N, device=DEV)
    state = Maker(802, DEV).normal(2, C, N, dtype=torch.float32)
    first = S // 3
    want, got = state.clone(), state.clone()
    y = _run(vdc, k, [0, first, S], want)
    bad = _run(vdc, k, [0, first, min(S + past, 2 ** 31 - 1)], got)
    assert torch.equal(bad, y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], state[1])


@pytest.mark.parametrize("S,C,N", [(100, 72, 5), (700, 72, 16)])
def test_tokens_past_the_last_end(vdc, S, C, N):
    k, _, _ = scan_inputs(811, [S], C, N, device=DEV)
    state = Maker(812, DEV).normal(2, C, N, dtype=torch.float32)
    want, got = state.clone(), state[:1].clone()
    y = _run(vdc, k, [0, S // 2, S], want, resume=False)
    assert torch.equal(_run(vdc, k, [0, S // 2], got, resume=False), y)
    assert torch.equal(got[0], want[0])
