"""The layer norm's parameter gradients of long inputs: FP32 sums of at most 256
terms one after another, whatever the number of tokens."""
import pytest
import torch

from ssm_ref import U

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("S,C", [(2048 * 512 * 32 + 5, 64), (2048 * 512 + 1, 4096), (2048 * 256, 8192)])
@pytest.mark.parametrize("dstream", [True, False])
def test_sums_of_many_tokens(S, C, dstream):
    """Every token the same, so that the sums are S times a term and FP32 rounds
    each addition of a range the same way."""
    import varlen_depthwise_causal_amd as vdc
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(C)
    row, grad = torch.randn(C, generator=g).bfloat16(), torch.randn(C, generator=g).bfloat16()
    w = torch.rand(C, generator=g).to(DEV) + 0.5
    s = row.to(DEV).expand(S, C).contiguous()
    dy = grad.to(DEV).expand(S, C).contiguous()
    dx, dw, db = vdc.layer_norm_bwd(s, w, dy, bias=torch.zeros(C, device=DEV), dstream=s if dstream else None)
    x = row.double()
    mean = x.mean()
    rstd = ((x - mean) ** 2).mean().add(1e-5) ** -0.5
    xh = (x - mean) * rstd
    # A term: the mean, the difference, the variance and its root, 64 roundings of the
    # values' largest at most in any order of summing (8 K + 6 + waves and a few, K = 2).
    # The sums: 256 turns, 32 teams, the last rounding from FP64.
    term = 64 * U * (x.abs().max() * rstd + xh.abs())
    chain = (256 + 32 + 1) * U
    want, bound = S * grad.double() * xh, S * grad.double().abs() * (term + chain * xh.abs())
    for name, got, w_, b in (("dweight", dw, want, bound),
                             ("dbias", db, S * grad.double(), S * grad.double().abs() * chain)):
        off = (got.double().cpu() - w_).abs() / b.clamp(min=1e-30)
        print("%s: relative L2 %.2e, worst %.3f of its bound" % (
            name, float((got.double().cpu() - w_).norm() / w_.norm()), float(off.max())), flush=True)
        assert float(off.max()) <= 1.0
    assert torch.equal(dx[:1], dx[-1:]) and torch.equal(dx[: 1 << 16], dx[-(1 << 16):])
