"""64-bit definitions of the state space layer's operators, token by token,
and bounds on what FP32 kernels may differ from them by.

Each result comes with a bound of its own, carried through the same formulas:
u = 2^-24 is the most a rounding to FP32 is off, relative to the value; the
hardware's exponential, reciprocal and root are off by a few of those; a sum of
n terms by at most n u times the sum of their magnitudes in any order.  Results
in BF16 may be half a step off on top, 2^-8 of the value (``close``).
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -120  # results below the normal range are flushed


def f64(t):
    return None if t is None else t.detach().double()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(name, got, want, bound):
    """Every element within its bound and half a step of its type."""
    assert tuple(got.shape) == tuple(want.shape), (name, got.shape, want.shape)
    g = got.double()
    assert bool(torch.isfinite(g).all()), "%s: not finite" % name
    off = (g - want).abs()
    allowed = bound * (1 + half_step(got.dtype)) + half_step(got.dtype) * want.abs() + TINY
    worst = float((off / allowed).max()) if off.numel() else 0.0
    print("%-10s n=%-9d worst %.3f of its bound" % (name, off.numel(), worst), flush=True)
    assert worst <= 1.0, "%s: %.3f times its bound" % (name, worst)


def sigmoid(z):
    """sigmoid(z) and the relative error of 1 / (1 + exp2(-z log2 e)) in FP32."""
    return torch.sigmoid(z), (8 + 3 * z.abs()) * U


def dsilu(z):
    """silu'(z) and its absolute error: s (1 + z (1 - s)) cancels near -1.28."""
    s, e = sigmoid(z)
    return s * (1 + z * (1 - s)), s * (1 + z.abs()) * (8 * U + 2 * e)


def softplus(raw):
    """softplus(raw) and its relative error: raw itself is a rounded sum."""
    d = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    return d, (24 + 2 * raw.abs()) * U


def spans(cu):
    e = [int(v) for v in cu]
    return list(zip(e, e[1:]))


# ------------------------------------------------------------ convolution --

def conv(x, weight, bias, docs, state=None, slots=None, resume=None):
    """y, its bound and the states after each document (x float64 [S, C])."""
    w, S, C = f64(weight), x.shape[0], x.shape[1]
    b = torch.zeros(C, dtype=torch.float64, device=x.device) if bias is None else f64(bias)
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    after = None if state is None else state.clone()
    for i, (lo, hi) in enumerate(docs):
        slot = -1 if slots is None else slots[i]
        past = torch.zeros(3, C, dtype=torch.float64, device=x.device)
        if slot >= 0 and resume is not None and resume[i]:
            past = state[slot].double()
        seq = torch.cat([past, x[lo:hi]])
        for k in range(4):
            p[lo:hi] += w[:, k] * seq[k:k + hi - lo]
            m[lo:hi] += (w[:, k] * seq[k:k + hi - lo]).abs()
        if slot >= 0 and after is not None:
            after[slot] = seq[hi - lo:].to(after.dtype)
    p, m = p + b, m + b.abs()
    s, e = sigmoid(p)
    return p * s, 1.1 * 5 * U * m + (p * s).abs() * (e + 2 * U), after


# ------------------------------------------------------------------- scan --

class Scan:
    """The scan and its gradients, with bounds.  B, C: [S, G, N]."""

    def __init__(self, x, dt, A, B, C, docs, D=None, z=None, dt_bias=None, softplus_on=True, state=None,
                 slots=None, resume=None):
        x, dt, A, B, Cm = f64(x), f64(dt), f64(A), f64(B), f64(C)
        self.S, self.Cn = x.shape
        self.N, self.G = A.shape[1], B.shape[1]
        per = self.Cn // self.G
        self.x, self.A, self.docs = x, A, docs
        self.D = f64(D)
        self.B, self.C = B.repeat_interleave(per, 1), Cm.repeat_interleave(per, 1)
        self.raw = dt if dt_bias is None else dt + f64(dt_bias)
        self.soft = softplus_on
        if softplus_on:
            self.d, ed = softplus(self.raw)
        else:
            self.d, ed = self.raw, torch.full_like(dt, 2 * U)
        self.ed = ed
        self.z = f64(z)
        if z is None:
            self.gate, self.eg = torch.ones_like(x), torch.zeros_like(x)
        else:
            s, e = sigmoid(self.z)
            self.gate, self.eg = self.z * s, e + 2 * U
        dA = self.d[..., None] * A
        self.a = torch.exp(dA)
        # the decay's exponential and the rounding of its argument; the joins
        # of chunks (sums of step sizes, one more exponential) within it
        self.ea = 4 * U + dA.abs() * (ed[..., None] + 6 * U)
        self.u = (self.d * x)[..., None] * self.B
        shape = (self.S, self.Cn, self.N)
        new = lambda: torch.zeros(shape, dtype=torch.float64, device=x.device)  # noqa: E731
        self.h, self.eh, self.before, self.ebefore = new(), new(), new(), new()
        self.after = None if state is None else state.double().clone()
        self.eafter = None if state is None else torch.zeros_like(self.after)
        eu = self.u.abs() * (ed[..., None] + 3 * U)
        for i, (lo, hi) in enumerate(docs):
            h = torch.zeros(shape[1:], dtype=torch.float64, device=x.device)
            m, e = h.clone(), h.clone()
            slot = -1 if slots is None else slots[i]
            if slot >= 0 and resume is not None and resume[i]:
                h = state[slot].double()
                m = h.abs()
            for t in range(lo, hi):
                self.before[t], self.ebefore[t] = h, e
                e = self.a[t] * (e + self.ea[t] * m) + eu[t]
                h = self.a[t] * h + self.u[t]
                m = self.a[t] * m + self.u[t].abs()
                e = e + 4 * U * m
                self.h[t], self.eh[t] = h, e
            if slot >= 0 and self.after is not None:
                self.after[slot], self.eafter[slot] = h, e
        Dx = 0 if self.D is None else self.D * x
        terms = (self.C * self.h).abs().sum(-1) + (0 if self.D is None else Dx.abs())
        self.y0 = (self.C * self.h).sum(-1) + Dx
        self.ey0 = (self.C.abs() * self.eh).sum(-1) + (self.N + 4) * U * terms
        self.y = self.y0 * self.gate
        self.ey = self.ey0 * self.gate.abs() + self.y.abs() * (self.eg + 2 * U)

    def grads(self, dy):
        """{name: (gradient, bound)} for y's gradient dy."""
        dy = f64(dy)
        S, Cn, N, G = self.S, self.Cn, self.N, self.G
        per = Cn // G
        g = dy * self.gate
        eg = g.abs() * (self.eg + U)
        lam, el = torch.zeros_like(self.h), torch.zeros_like(self.h)
        for lo, hi in self.docs:
            L = torch.zeros_like(self.h[0]) if S else None
            m = e = L
            for t in range(hi - 1, lo - 1, -1):
                own = self.C[t] * g[t][:, None]
                m = m + own.abs()
                L = L + own
                e = e + self.C[t].abs() * eg[t][:, None] + 4 * U * m
                lam[t], el[t] = L, e
                e = self.a[t] * (e + self.ea[t] * m)
                L, m = self.a[t] * L, self.a[t] * m
        ah = self.a * self.before
        eah = self.a * (self.ebefore + (self.ea + 2 * U) * self.before.abs())
        v = lam * ah
        ev = lam.abs() * eah + ah.abs() * el + 2 * U * v.abs()
        dx_ = self.d * self.x
        edx = dx_.abs() * (self.ed + U)
        slb = (lam * self.B).sum(-1)
        eslb = (el * self.B.abs()).sum(-1) + (N + 2) * U * (lam * self.B).abs().sum(-1)
        sva = (v * self.A).sum(-1)
        esva = (ev * self.A.abs()).sum(-1) + (N + 2) * U * (v * self.A).abs().sum(-1)
        out = {}
        Dg = 0 if self.D is None else self.D * g
        eDg = 0 if self.D is None else self.D.abs() * eg + U * Dg.abs()
        out["dx"] = (Dg + self.d * slb, eDg + self.d.abs() * (eslb + slb.abs() * (self.ed + 2 * U)))
        dd = self.x * slb + sva
        edd = self.x.abs() * eslb + esva + 3 * U * ((self.x * slb).abs() + sva.abs())
        if self.soft:
            s, e = sigmoid(self.raw)
            ddt, eddt = dd * s, edd * s + (dd * s).abs() * (e + 2 * U + 2 * U * self.raw.abs())
        else:
            ddt, eddt = dd, edd
        out["ddt"] = (ddt, eddt)
        group = lambda q: q.view(S, G, per, N).sum(2)  # noqa: E731
        dB = lam * dx_[..., None]
        eB = el * dx_.abs()[..., None] + lam.abs() * edx[..., None]
        out["dB"] = (group(dB), group(eB) + (per + 4) * U * group(dB.abs()))
        dC = self.h * g[..., None]
        eC = self.eh * g.abs()[..., None] + self.h.abs() * eg[..., None]
        out["dC"] = (group(dC), group(eC) + (per + 4) * U * group(dC.abs()))
        q = v * self.d[..., None]
        eq = ev * self.d.abs()[..., None] + q.abs() * (self.ed[..., None] + U)
        out["dA"] = (q.sum(0), eq.sum(0) + (S + 4) * U * q.abs().sum(0))
        out["ddt_bias"] = (ddt.sum(0), eddt.sum(0) + (S + 4) * U * ddt.abs().sum(0))
        if self.D is not None:
            q = g * self.x
            out["dD"] = (q.sum(0), (eg * self.x.abs()).sum(0) + (S + 4) * U * q.abs().sum(0))
        if self.z is not None:
            k, ek = dsilu(self.z)
            dz = dy * self.y0 * k
            out["dz"] = (dz, dy.abs() * (self.ey0 * k.abs() + self.y0.abs() * ek) + 3 * U * dz.abs())
        return out


# ------------------------------------------------------------- group norm --

class Norm:
    def __init__(self, x, weight, groups, bias=None, z=None, eps=1e-5):
        x = f64(x)
        self.S, self.C = x.shape
        P = self.C // groups
        self.P, self.shape = P, (self.S, groups, P)
        g = x.view(self.shape)
        mean = g.mean(-1, keepdim=True)
        em = (P + 2) * U * g.abs().mean(-1, keepdim=True)
        d = g - mean
        ed = em + U * d.abs()
        var = (d * d).mean(-1, keepdim=True)
        evar = 2 * (d.abs() * ed).mean(-1, keepdim=True) + (ed * ed).mean(-1, keepdim=True) + (P + 4) * U * var
        self.rstd = (var + eps) ** -0.5
        # eps itself is an FP32 argument
        self.er = 8 * U + (evar + U * eps) / (var + eps)
        self.xh = d * self.rstd
        self.exh = ed * self.rstd * (1 + self.er) + self.xh.abs() * (self.er + 2 * U)
        self.w = f64(weight).view(self.shape[1:])
        self.b = torch.zeros_like(self.w) if bias is None else f64(bias).view(self.shape[1:])
        self.v = self.w * self.xh + self.b
        self.ev = self.w.abs() * self.exh + 2 * U * ((self.w * self.xh).abs() + self.b.abs())
        self.z = None if z is None else f64(z).view(self.shape)
        u = self.v if z is None else self.z
        s, e = sigmoid(u)
        if z is None:
            self.y = self.v * s
            self.ey = 1.1 * self.ev + self.y.abs() * (e + 2 * U)
        else:
            self.gate, self.eg = u * s, (u * s).abs() * (e + 2 * U)
            self.y = self.v * self.gate
            self.ey = self.ev * self.gate.abs() + self.v.abs() * self.eg + 2 * U * self.y.abs()
        flat = (self.S, self.C)
        self.y, self.ey = self.y.view(flat), self.ey.view(flat)

    def grads(self, dy):
        dy, P = f64(dy).view(self.shape), self.P
        flat, out = (self.S, self.C), {}
        if self.z is None:
            k, ek = dsilu(self.v)
            # silu'' is at most 1/2
            dv, edv = dy * k, dy.abs() * (ek + 0.5 * self.ev) + 2 * U * (dy * k).abs()
        else:
            dv, edv = dy * self.gate, dy.abs() * self.eg + 2 * U * (dy * self.gate).abs()
            k, ek = dsilu(self.z)
            dz = dy * self.v * k
            out["dz"] = (dz.view(flat), (dy.abs() * (self.ev * k.abs() + self.v.abs() * ek)
                                         + 3 * U * dz.abs()).view(flat))
        q = dv * self.xh
        eq = edv * self.xh.abs() + dv.abs() * self.exh + U * q.abs()
        n = self.S + 4
        out["dweight"] = (q.sum(0).reshape(-1), (eq.sum(0) + n * U * q.abs().sum(0)).reshape(-1))
        out["dbias"] = (dv.sum(0).reshape(-1), (edv.sum(0) + n * U * dv.abs().sum(0)).reshape(-1))
        r = dv * self.w
        er = edv * self.w.abs() + U * r.abs()
        m1 = r.mean(-1, keepdim=True)
        e1 = er.mean(-1, keepdim=True) + (P + 2) * U * r.abs().mean(-1, keepdim=True)
        rx = r * self.xh
        erx = er * self.xh.abs() + r.abs() * self.exh + U * rx.abs()
        m2 = rx.mean(-1, keepdim=True)
        e2 = erx.mean(-1, keepdim=True) + (P + 2) * U * rx.abs().mean(-1, keepdim=True)
        inner = r - m1 - self.xh * m2
        parts = r.abs() + m1.abs() + (self.xh * m2).abs()
        einner = er + e1 + self.exh * m2.abs() + self.xh.abs() * e2 + 4 * U * parts
        dx = self.rstd * inner
        out["dx"] = (dx.view(flat), (self.rstd * einner * (1 + self.er) + dx.abs() * (self.er + 2 * U)).view(flat))
        return out
