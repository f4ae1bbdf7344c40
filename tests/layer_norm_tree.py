"""Bounds of the layer norm that follow the order in which the kernel sums: a lane's
8 K channels one after another, the lanes of a wave in halves, the waves one after
another, squares about the wave's own mean.  They grow with the logarithm of the
row, where layer_ref's are those of a sum in any order, so that a mean far from the
values' spread, which costs a sum of squares its digits, shows.

With u = 2^-24, x the row, mu its mean, m_w a wave's mean as computed and `all` the
row's:
- a wave's sum has 8 K - 1 roundings in a lane, 6 over lanes, its mean 2 more (the
  reciprocal's and the product's): |m_w - mean_w| <= ew = (8 K + 7) u max|x|; the
  row's mean has one for each wave and 3 more (the products' come in FMAs):
  |all - mu| <= em = ew + (W + 3) u max|x|.
- x - all comes as (x - m_w) + (m_w - all): three roundings, of values up to twice
  the largest difference from mu and the means' errors.
- sum (x - all)^2 = sum_w [sum (x - m_w)^2 + 2 (m_w - all) sum (x - m_w) + n_w (m_w -
  all)^2], of which the kernel leaves out the middle: at most 2 ew |m_w - all| a
  channel, and the mean of |m_w - all| is no more than the root of the mean square,
  which is no more than that of (x - all)^2 and ew.
- the squares' sums have 8 K + 6 + W + 4 roundings, and 2 of the differences.
"""
import torch

from layer_ref import MORE, LayerNorm
from ssm_ref import U, f64


def tree(C):
    """Lanes, vectors of 8 a lane and waves of a row's team."""
    n = (C + 7) // 8
    lanes = 8 if n <= 8 else 16 if n <= 16 else 32 if n <= 32 else 64 if n <= 128 else 256 if n <= 512 else \
        512 if n <= 1024 else 1024
    vecs = 2 if 64 < n <= 128 or n > 256 else 1
    return lanes, vecs, max(1, lanes // 64)


class LayerNormTree(LayerNorm):
    """LayerNorm's values with these bounds."""

    def __init__(self, s, weight, bias=None, eps=1e-5):
        super().__init__(s, weight, bias, eps)
        x = f64(s)
        _, K, W = tree(self.C)
        self.n = 8 * K + 6 + W + 4
        most = x.abs().amax(-1, keepdim=True)
        ew = (8 * K + 7) * U * most
        em = ew + ((W + 3) * U * most if W > 1 else 0)
        d = x - x.mean(-1, keepdim=True)
        ed = em + 3 * U * (2 * self.top + em + ew)
        var = (d * d).mean(-1, keepdim=True)
        about = var + em * em  # mean (x - all)^2
        evar = (self.n + 2) * U * about + em * em
        if W > 1:
            evar = evar + 2 * ew * (about.sqrt() + ew)
        share = (evar + U * eps) / (var + eps)
        assert float(share.max()) < 0.5, "no bound: the variance has no digits"
        # 1 / sqrt(1 - share) - 1 <= share below a half
        self.er = 6 * U + share
        self.exh = ed * self.rstd * (1 + self.er) + self.xh.abs() * (self.er + 2 * U)
        self.ey = MORE * (self.w.abs() * self.exh + 2 * U * ((self.w * self.xh).abs() + self.b.abs()))

    def grads(self, dy, dstream=None):
        dy, n = f64(dy), self.n
        out = super().grads(dy, dstream)
        q = dy * self.xh
        rows = (self.S + 4) * U
        out["dweight"] = (out["dweight"][0], MORE * ((dy.abs() * self.exh + U * q.abs()).sum(0) + rows * q.abs().sum(0)))
        r = dy * self.w
        er = U * r.abs()
        m1 = r.mean(-1, keepdim=True)
        e1 = er.mean(-1, keepdim=True) + n * U * r.abs().mean(-1, keepdim=True)
        rx = r * self.xh
        m2 = rx.mean(-1, keepdim=True)
        # sums about the waves' means, whose terms are up to twice the largest difference,
        # and the row's: as many roundings each, one more for the factor rstd
        e2 = ((er * self.xh.abs() + r.abs() * self.exh + U * rx.abs()).mean(-1, keepdim=True)
              + (n + 4) * U * (r.abs() * 3 * self.top * self.rstd).mean(-1, keepdim=True)
              + self.er * rx.abs().mean(-1, keepdim=True))
        parts = r.abs() + m1.abs() + (self.xh * m2).abs()
        inner = r - m1 - self.xh * m2
        einner = er + e1 + self.exh * m2.abs() + self.xh.abs() * e2 + 4 * U * parts
        dx = self.rstd * inner
        edx = self.rstd * einner * (1 + self.er) + dx.abs() * (self.er + 2 * U)
        if dstream is not None:
            dx = dx + f64(dstream)
            edx = edx + U * dx.abs()
        out["dx"] = (dx, MORE * edx)
        return out


def rows_far_from_zero(S, C, seed, device):
    """BF16 rows whose mean is 500 to 4000 times their spread: one value, and the
    next one or the one before it here and there."""
    g = torch.Generator().manual_seed(seed)
    base = torch.tensor([256.0, -1000.0, 3.0e4, 1.0, -2.0e-3])[torch.arange(S) % 5]
    step = base.abs() * 2.0 ** -7  # one or two steps of BF16
    often = torch.rand(S, 1, generator=g) * 0.04 + 0.002
    off = (torch.rand(S, C, generator=g) < often).float() * torch.sign(torch.randn(S, C, generator=g))
    off[:, C // 2] = 1.0
    return (base[:, None] + step[:, None] * off).to(torch.bfloat16).to(device)
