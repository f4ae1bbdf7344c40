"""64-bit definitions of the recurrent layer's operators, token by token, and
bounds on what FP32 kernels may differ from them by, in the manner of ssm_ref
(whose constants, sigmoid and softplus they use): u = 2^-24 for each rounding to
FP32, a few of them for an exponential, reciprocal or root, n u times the sum
of the magnitudes for a sum of n terms in any order.  Products of two such
errors are left out, for which every bound is a tenth larger (MORE)."""
import torch

from ssm_ref import U, dsilu, f64, sigmoid, softplus

MORE = 1.1


class Recurrence:
    """The gated linear recurrence and its gradients, with bounds."""

    def __init__(self, x, r, i, decay, docs, z=None, scale=8.0, state=None, slots=None, resume=None):
        x, r, i, decay = f64(x), f64(r), f64(i), f64(decay)
        self.S, self.C = x.shape
        self.docs, self.decay = docs, decay
        self.soft, self.es = softplus(decay)
        self.sr, self.er = sigmoid(r)
        self.si, self.ei = sigmoid(i)
        self.er = torch.where(self.sr == 0, torch.zeros_like(self.er), self.er)  # no infinite error of a zero
        self.u = 2 * scale * self.soft * self.sr
        self.eu = self.es + self.er + 4 * U
        self.a = torch.exp(-self.u / 2)
        self.ea = 4 * U + self.u / 2 * (self.eu + 3 * U)
        self.v = -torch.expm1(-self.u)
        # the series below u = 1/4; above it 1 - a^2, which cancels by v
        safe = self.v.clamp(min=1e-300)
        self.ev = torch.where(self.u < 0.26, self.eu + 8 * U, torch.zeros_like(self.u))
        self.ev = torch.where(self.u > 0.24, torch.maximum(self.ev, 2 * self.a ** 2 * self.ea / safe + 2 * U), self.ev)
        self.m = self.v.sqrt()
        none = self.v == 0
        # a token without a step adds nothing, whatever x holds
        self.gx = torch.where(none, torch.zeros_like(x), self.si * x)
        self.none = none
        self.b = self.m * self.gx
        eb = self.b.abs() * (self.ev / 2 + self.ei + 6 * U)
        self.z = f64(z)
        if z is None:
            self.gate, self.eg = torch.ones_like(x), torch.zeros_like(x)
        else:
            s, e = sigmoid(self.z)
            self.gate, self.eg = self.z * s, e + 2 * U
        new = lambda: torch.zeros_like(x)  # noqa: E731
        self.h, self.eh, self.before, self.ebefore = new(), new(), new(), new()
        self.after = None if state is None else state.double().clone()
        self.eafter = None if state is None else torch.zeros_like(self.after)
        for d, (lo, hi) in enumerate(docs):
            h = torch.zeros(self.C, dtype=torch.float64, device=x.device)
            m, e = h.clone(), h.clone()
            slot = -1 if slots is None else slots[d]
            if slot >= 0 and resume is not None and resume[d]:
                h = state[slot].double()
                m = h.abs()
            for t in range(lo, hi):
                self.before[t], self.ebefore[t] = h, e
                e = self.a[t] * (e + self.ea[t] * m) + eb[t]
                h = self.a[t] * h + self.b[t]
                m = self.a[t] * m + self.b[t].abs()
                # a step's own rounding, that of the products of decays, a join
                e = e + torch.where(none[t], 0.0, 4 * U) * m
                self.h[t], self.eh[t] = h, e
            if slot >= 0 and self.after is not None and (hi > lo or not (resume and resume[d])):
                self.after[slot], self.eafter[slot] = h, MORE * e
        self.y = self.h * self.gate
        self.ey = MORE * (self.eh * self.gate.abs() + self.y.abs() * (self.eg + 2 * U))

    def grads(self, dy):
        """{name: (gradient, bound)} for y's gradient dy."""
        dy = f64(dy)
        g = dy * self.gate
        eg = g.abs() * (self.eg + U)
        lam, el = torch.zeros_like(g), torch.zeros_like(g)
        for lo, hi in self.docs:
            L = torch.zeros(self.C, dtype=torch.float64, device=g.device)
            m = e = L
            for t in range(hi - 1, lo - 1, -1):
                m, L = m + g[t].abs(), L + g[t]
                e = e + eg[t] + 4 * U * m
                lam[t], el[t] = L, e
                e = self.a[t] * (e + self.ea[t] * m)
                L, m = self.a[t] * L, self.a[t] * m
        out = {}
        em = self.ev / 2 + 4 * U
        dx = lam * self.m * self.si
        out["dx"] = (dx, el * self.m * self.si + dx.abs() * (em + self.ei + 3 * U))
        rest, erest = 1 - self.si, self.si * self.ei + U
        base = lam * self.b
        out["di"] = (base * rest, rest * (el * self.b.abs() + base.abs() * (em + self.ei + 5 * U))
                     + base.abs() * erest)
        half = self.u / 2
        w = torch.where(self.none, torch.zeros_like(half), half / self.m.clamp(min=1e-300))
        t1, t2 = self.gx * self.a ** 2 * w, half * self.a * self.before
        inner = t1 - t2
        einner = (t1.abs() * (self.ei + 2 * self.ea + self.eu + self.ev / 2 + 8 * U)
                  + t2.abs() * (self.eu + self.ea + 5 * U) + half * self.a * self.ebefore)
        E = lam * inner
        eE = el * inner.abs() + lam.abs() * einner + 2 * U * E.abs()
        keep = 1 - self.sr
        out["dr"] = (E * keep, eE * keep + E.abs() * (self.sr * self.er + 3 * U))
        s, e = sigmoid(self.decay)
        ratio = torch.where(self.soft > 0, s / self.soft.clamp(min=1e-300), torch.ones_like(s))
        total = E.sum(0)
        out["ddecay"] = (ratio * total, ratio * (eE.sum(0) + (self.S + 4) * U * E.abs().sum(0)
                                                 + total.abs() * (self.es + e + 4 * U)))
        if self.z is not None:
            k, ek = dsilu(self.z)
            dz = dy * self.h * k
            out["dz"] = (dz, dy.abs() * (self.eh * k.abs() + self.h.abs() * ek) + 4 * U * dz.abs())
        return {n: (t, MORE * e) for n, (t, e) in out.items()}


class LayerNorm:
    """The layer norm of what the stream holds (BF16) and its gradients."""

    def __init__(self, s, weight, bias=None, eps=1e-5):
        x = f64(s)
        self.S, self.C = x.shape
        C = self.C
        self.w = f64(weight)
        self.b = torch.zeros_like(self.w) if bias is None else f64(bias)
        mean = x.mean(-1, keepdim=True)
        em = (C + 4) * U * x.abs().mean(-1, keepdim=True)
        d = x - mean
        self.top = d.abs().amax(-1, keepdim=True)
        # a wave's mean is off the row's by no more than the largest difference
        ed = 2 * em + 4 * U * (d.abs() + self.top)
        var = (d * d).mean(-1, keepdim=True)
        evar = (2 * (d.abs() * ed).mean(-1, keepdim=True) + (ed * ed).mean(-1, keepdim=True) + (C + 8) * U * var
                + 2 * ed.amax(-1, keepdim=True) * em)
        self.rstd = (var + eps) ** -0.5
        self.er = 8 * U + (evar + U * eps) / (var + eps)  # eps itself is an FP32 argument
        self.xh = d * self.rstd
        self.exh = ed * self.rstd * (1 + self.er) + self.xh.abs() * (self.er + 2 * U)
        self.y = self.w * self.xh + self.b
        self.ey = MORE * (self.w.abs() * self.exh + 2 * U * ((self.w * self.xh).abs() + self.b.abs()))

    def grads(self, dy, dstream=None):
        dy, C, n = f64(dy), self.C, self.S + 4
        out = {}
        q = dy * self.xh
        eq = dy.abs() * self.exh + U * q.abs()
        out["dweight"] = (q.sum(0), eq.sum(0) + n * U * q.abs().sum(0))
        out["dbias"] = (dy.sum(0), n * U * dy.abs().sum(0))
        r = dy * self.w
        er = U * r.abs()
        m1 = r.mean(-1, keepdim=True)
        e1 = er.mean(-1, keepdim=True) + (C + 4) * U * r.abs().mean(-1, keepdim=True)
        rx = r * self.xh
        erx = er * self.xh.abs() + r.abs() * self.exh + U * rx.abs()
        m2 = rx.mean(-1, keepdim=True)
        # sums about the waves' means: their terms are up to the largest difference
        e2 = erx.mean(-1, keepdim=True) + (C + 8) * U * 2 * (r.abs() * self.top * self.rstd).mean(-1, keepdim=True)
        inner = r - m1 - self.xh * m2
        parts = r.abs() + m1.abs() + (self.xh * m2).abs()
        einner = er + e1 + self.exh * m2.abs() + self.xh.abs() * e2 + 4 * U * parts
        dx = self.rstd * inner
        edx = self.rstd * einner * (1 + self.er) + dx.abs() * (self.er + 2 * U)
        if dstream is not None:
            dx = dx + f64(dstream)
            edx = edx + U * dx.abs()
        out["dx"] = (dx, edx)
        return {k: (t, MORE * e) for k, (t, e) in out.items()}


POOL_BLOCK = 64


def codes_of(dtype):
    """The magnitudes that a code can stand for, in order."""
    if dtype == torch.int8:
        return torch.arange(128).double()
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def put_aside(flat, dtype):
    """Values in a row (float64 of FP32 or BF16 values) -> signed magnitudes that
    their codes stand for, and the scale of each block of 64 (float32)."""
    mags = codes_of(dtype).to(flat.device)
    n = (flat.numel() + POOL_BLOCK - 1) // POOL_BLOCK
    v = torch.zeros(n * POOL_BLOCK, dtype=torch.float64, device=flat.device)
    v[:flat.numel()] = flat
    v = v.view(n, POOL_BLOCK)
    top = v.abs().amax(1)  # a NaN stays
    bad, zero = ~torch.isfinite(top), top < 2.0 ** -64
    scale = (top / mags[-1]).float()
    scale = torch.where(zero, 0.0, torch.where(bad, float("nan"), scale))
    t = torch.where((bad | zero)[:, None], 0.0, v.abs() / torch.where(bad | zero, 1.0, scale.double())[:, None])
    middle = (mags[1:] + mags[:-1]) / 2
    k = torch.searchsorted(middle, t)
    k = k + ((t == middle[k.clamp(max=middle.numel() - 1)]) & (k % 2 == 1)).long()
    q = mags[k] * torch.sign(torch.where(bad[:, None], 0.0, v))
    return q.view(-1)[:flat.numel()], scale


def take_back(q, scale, dtype):
    """code * scale in FP32, rounded to the cache's dtype."""
    return (q.float() * scale.repeat_interleave(POOL_BLOCK)[:q.numel()]).to(dtype)
