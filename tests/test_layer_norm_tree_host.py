"""The bounds of layer_norm_tree.py on the CPU: they hold for sums in the kernel's
order in FP32, and reject a variance from one pass over the row."""
import pytest
import torch

from layer_norm_tree import LayerNormTree, rows_far_from_zero, tree
from ssm_ref import close

F32 = torch.float32
SIZES = [40, 130, 520, 1001, 2048, 4096, 8192, 16384]


def emulated(s, weight, bias, eps, one_pass):
    """y in FP32: sums of a lane's channels, over its wave's lanes, over the waves, or
    of the values and their squares alone."""
    S, C = s.shape
    L, K, W = tree(C)
    x = torch.zeros(S, L * K * 8, dtype=F32)
    x[:, :C] = s.float()
    has = torch.zeros(L * K * 8, dtype=torch.bool)
    has[:C] = True
    # [rows, K, waves, lanes, 8]
    x, has = x.view(S, K, W, L // W, 8), has.view(K, W, L // W, 8)

    def wave_sum(v):
        t = torch.zeros(S, W, L // W)
        for k in range(K):
            for i in range(8):
                t = t + v[:, k, :, :, i]
        while t.shape[-1] > 1:
            t = t[..., ::2] + t[..., 1::2]
        return t[..., 0]

    n = has.sum((0, 2, 3)).float()
    if one_pass:
        mean = sum(wave_sum(x).unbind(1)) / C
        square = sum(wave_sum(x * x).unbind(1)) / C
        var, d = square - mean * mean, x - mean.view(S, 1, 1, 1, 1)
    else:
        inv = torch.where(n > 0, 1 / n.clamp(min=1), torch.zeros_like(n))
        mw = wave_sum(x) * inv
        d = torch.where(has, x - mw.view(S, 1, W, 1, 1), torch.zeros(()))
        sq = wave_sum(d * d)
        mean = sum((n * mw).unbind(1)) / C if W > 1 else mw[:, 0]
        off = mw - mean[:, None]
        var = sum((sq + n * off * off).unbind(1)) / C
        d = d + off.view(S, 1, W, 1, 1)
    y = d * (1 / (var + eps).sqrt()).view(S, 1, 1, 1, 1)
    return (y.reshape(S, -1)[:, :C] * weight + bias).to(torch.bfloat16)


def case(C):
    s = rows_far_from_zero(10, C, C, "cpu")
    g = torch.Generator().manual_seed(C + 1)
    return s, torch.rand(C, generator=g) + 0.5, torch.randn(C, generator=g) * 0.1


@pytest.mark.parametrize("C", SIZES)
def test_the_kernels_order_is_within_the_bounds(C):
    s, w, b = case(C)
    ref = LayerNormTree(s, w, b, 1e-12)
    close("y", emulated(s, w, b, 1e-12, False), ref.y, ref.ey)


@pytest.mark.parametrize("C", SIZES)
def test_one_pass_is_not(C):
    s, w, b = case(C)
    ref = LayerNormTree(s, w, b, 1e-12)
    y = emulated(s, w, b, 1e-12, True)
    off = (y.double() - ref.y).abs() > ref.ey * 1.01 + 2.0 ** -8 * ref.y.abs()
    bad = off.any(1) | ~torch.isfinite(y).all(1)
    assert bool(bad.float().mean() > 0.5), bad
