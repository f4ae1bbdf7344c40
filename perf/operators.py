"""The operators of a selective state space layer around the packed causal
convolution, measured: the convolution with a carried state (prompts and
single tokens), the selective scan (prompts, training, single tokens) and the
gated group norm.

``run`` computes them in plain torch operations, or, where ``own`` is true,
through this package's entry points.  ``exact`` computes the same outputs from
the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One sequence decoding one token: the latency of a single call.
        {"name": "conv_step_1", "kind": "conv_step", "batch": 1, "C": 2048, "params": "f32"},
        # A full serving batch, one token each, slots scattered over a cache.
        {"name": "conv_step_1000", "kind": "conv_step", "batch": 1000, "C": 8192, "params": "bf16"},
        # A ragged batch of short prompts, half of them continuing a sequence;
        # rows that are not a multiple of a cache line.
        {"name": "conv_prompt_ragged", "kind": "conv_prompt", "S": 5003, "docs": 37, "C": 520,
         "params": "f32"},
        # A long prefill batch at the convolution's headline width.
        {"name": "conv_prompt_long", "kind": "conv_prompt", "S": 65536, "docs": 22, "C": 4096,
         "params": "f32"},
        # One short prompt: latency again, too few rows to fill the machine.
        {"name": "scan_prompt_short", "kind": "scan_prompt", "S": 77, "docs": 1, "C": 2048, "N": 16,
         "groups": 1, "gate": True, "params": "f32"},
        # A prefill batch of long prompts.
        {"name": "scan_prompt_long", "kind": "scan_prompt", "S": 32768, "docs": 5, "C": 4096, "N": 16,
         "groups": 1, "gate": True, "params": "f32"},
        # A small training batch: odd length, ragged documents, small states,
        # two groups, parameters kept in bfloat16, no gate.
        {"name": "scan_train_ragged", "kind": "scan_train", "S": 1543, "docs": 11, "C": 520, "N": 8,
         "groups": 2, "gate": False, "params": "bf16"},
        # A training batch of packed documents.
        {"name": "scan_train_large", "kind": "scan_train", "S": 16384, "docs": 6, "C": 4096, "N": 16,
         "groups": 1, "gate": True, "params": "f32"},
        # One sequence decoding one token.
        {"name": "state_step_1", "kind": "state_step", "batch": 1, "C": 2048, "N": 16, "groups": 1,
         "gate": True, "params": "f32"},
        # A full serving batch: the whole state is read and written.
        {"name": "state_step_512", "kind": "state_step", "batch": 512, "C": 4096, "N": 16, "groups": 1,
         "gate": True, "params": "f32"},
        # The output norm of a decoding batch, groups of 65 channels, no gate.
        {"name": "norm_serve", "kind": "norm", "S": 33, "C": 520, "groups": 8, "gate": False,
         "train": False, "params": "f32"},
        # The gated output norm of a training batch, forward and backward.
        {"name": "norm_train", "kind": "norm", "S": 16384, "C": 4096, "groups": 32, "gate": True,
         "train": True, "params": "f32"},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number spread over [lo, hi] by its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    kind = rng.choice(["conv_step", "conv_prompt", "scan_prompt", "scan_train", "state_step", "norm"])
    params = rng.choice(["f32", "bf16"])
    if kind == "conv_step":
        return {"kind": kind, "batch": _spread(rng, 1, 1000), "C": _spread(rng, 64, 8192, 8),
                "params": params}
    if kind == "conv_prompt":
        C = _spread(rng, 64, 8192, 8)
        S = _spread(rng, 1, min(65536, 65536 * 4096 // C))
        return {"kind": kind, "S": S, "docs": _spread(rng, 1, 64), "C": C, "params": params}
    groups = rng.choice([1, 1, 2, 4])
    N = rng.choice([16, 16, 16, 8, 13, 32, 64])
    gate = rng.random() < 0.5
    if kind == "scan_prompt" or kind == "scan_train":
        C = _spread(rng, 64, 6144, groups)
        most = (32768 if kind == "scan_prompt" else 16384) * 4096 * 16 // (C * N)
        S = _spread(rng, 1, min(32768, most))
        return {"kind": kind, "S": S, "docs": _spread(rng, 1, 48), "C": C, "N": N, "groups": groups,
                "gate": gate, "params": params}
    if kind == "state_step":
        C = _spread(rng, 64, 6144, groups)
        return {"kind": kind, "batch": _spread(rng, 1, min(512, 512 * 4096 * 16 // (C * N))), "C": C,
                "N": N, "groups": groups, "gate": gate, "params": params}
    groups = rng.choice([1, 2, 8, 32])
    C = _spread(rng, 8 * groups, 6144, 8 * groups)
    return {"kind": "norm", "S": _spread(rng, 1, 16384 * 4096 // max(C, 4096)), "C": C, "groups": groups,
            "gate": gate, "train": rng.random() < 0.5, "params": params}


# ----------------------------------------------------------------- inputs --

def _lengths(case):
    """Document lengths of a case: ragged, empty ones among them where there
    are many documents; they go by the case alone."""
    S, docs = case["S"], case["docs"]
    rng = random.Random("%d %d %d" % (S, docs, case["C"]))
    cuts = sorted(rng.randint(0, S) for _ in range(docs - 1))
    edges = [0] + cuts + [S]
    return [b - a for a, b in zip(edges, edges[1:])]


def _slots(count, rng):
    """More slots than sequences, taken in no order."""
    slots = count + count // 4 + 3
    return slots, rng.sample(range(slots), count)


class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEVICE)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, mean=0.0):
        return torch.randn(*shape, device=DEVICE, generator=self.g) * std + mean

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device=DEVICE, generator=self.g) * (hi - lo) + lo


def prepare(case, seed):
    m, host = _Maker(seed), random.Random(seed)
    kind, C = case["kind"], case["C"]
    bf = torch.bfloat16
    pt = bf if case["params"] == "bf16" else torch.float32
    s = {"kind": kind}
    if kind in ("conv_prompt", "scan_prompt", "scan_train"):
        lens = _lengths(case)
        edges = [0]
        for n in lens:
            edges.append(edges[-1] + n)
        s["cu"] = torch.tensor(edges, dtype=torch.int32, device=DEVICE)
        s["longest"] = max(lens)
    if kind in ("conv_step", "conv_prompt"):
        s["weight"] = m.uniform(C, 4, lo=-0.5, hi=0.5).to(pt)
        s["bias"] = m.normal(C, std=0.1).to(pt)
        count = case["batch"] if kind == "conv_step" else case["docs"]
        s["x"] = m.normal(case["batch"] if kind == "conv_step" else case["S"], C).to(bf)
        slots, index = _slots(count, host)
        s["state"] = m.normal(slots, 3, C).to(bf)
        s["index"] = torch.tensor(index, dtype=torch.int32, device=DEVICE)
        if kind == "conv_prompt":
            s["resume"] = torch.tensor([i % 2 for i in range(count)], dtype=torch.bool, device=DEVICE)
        return s
    if kind == "norm":
        S = case["S"]
        s["groups"], s["train"], s["eps"] = case["groups"], case["train"], 1e-5
        s["x"] = m.normal(S, C, mean=0.3).to(bf)
        s["z"] = m.normal(S, C).to(bf) if case["gate"] else None
        s["dy"] = m.normal(S, C).to(bf) if case["train"] else None
        s["weight"] = m.uniform(C, lo=0.5, hi=1.5).to(pt)
        s["bias"] = m.normal(C, std=0.1).to(pt)
        return s
    # The scan: step sizes of 0.001 to 0.1 on the channel's bias, decays of 1 to N,
    # the three projections' results cut out of wider rows as a layer has them.
    N, G = case["N"], case["groups"]
    rows = case["batch"] if kind == "state_step" else case["S"]
    s["x"] = m.normal(rows, C).to(bf)
    s["dt"] = m.normal(rows, C, std=0.5).to(bf)
    s["z"] = m.normal(rows, 2 * C).to(bf)[:, C:] if case["gate"] else None
    rank = 2 * max(1, C // 32)
    wide = m.normal(rows, rank + 2 * G * N).to(bf)
    s["B"] = wide[:, rank:rank + G * N].unflatten(1, (G, N))
    s["C"] = wide[:, rank + G * N:].unflatten(1, (G, N))
    s["A"] = (-(torch.arange(1, N + 1, device=DEVICE) * torch.exp(m.normal(C, N, std=0.1)))).to(pt)
    s["D"] = m.normal(C, mean=1.0, std=0.1).to(pt)
    step = torch.exp(m.uniform(C, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = (step + torch.log(-torch.expm1(-step))).to(pt)
    if kind == "scan_train":
        s["dy"] = m.normal(rows, C).to(bf)
        return s
    count = rows if kind == "state_step" else case["docs"]
    slots, index = _slots(count, host)
    s["state"] = m.normal(slots, C, N, std=0.1)
    s["index"] = torch.tensor(index, dtype=torch.int32, device=DEVICE)
    if kind == "scan_prompt":
        s["resume"] = torch.tensor([i % 2 for i in range(count)], dtype=torch.bool, device=DEVICE)
    return s


# --------------------------------------------- the framework's entry points --

def _run_own(s):
    import varlen_depthwise_causal_amd as vdc
    kind = s["kind"]
    if kind == "conv_step":
        y = vdc.conv1d_update(s["x"], s["state"], s["weight"], bias=s["bias"], state_index=s["index"])
        return {"y": y, "state": s["state"]}
    if kind == "conv_prompt":
        y = vdc.conv1d_prefill(s["x"], s["weight"], s["cu"], s["state"], bias=s["bias"],
                               state_index=s["index"], resume=s["resume"])
        return {"y": y, "state": s["state"]}
    if kind == "scan_prompt":
        y = vdc.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
                                   dt_bias=s["dt_bias"], state=s["state"], state_index=s["index"],
                                   resume=s["resume"])
        return {"y": y, "state": s["state"]}
    if kind == "state_step":
        y = vdc.selective_update(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"],
                                 z=s["z"], dt_bias=s["dt_bias"], state_index=s["index"])
        return {"y": y, "state": s["state"]}
    if kind == "scan_train":
        y = vdc.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
                                   dt_bias=s["dt_bias"])
        dx, ddt, dA, dB, dC, dD, dz, ddt_bias = vdc.selective_scan_bwd(
            s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["dy"], D=s["D"], z=s["z"],
            dt_bias=s["dt_bias"])
        out = {"y": y, "dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": dD,
               "ddt_bias": ddt_bias}
        return out if s["z"] is None else {**out, "dz": dz}
    y = vdc.group_norm_silu_fwd(s["x"], s["weight"], s["groups"], bias=s["bias"], z=s["z"], eps=s["eps"])
    if not s["train"]:
        return {"y": y}
    dx, dw, db, dz = vdc.group_norm_silu_bwd(s["x"], s["weight"], s["groups"], s["dy"], bias=s["bias"],
                                             z=s["z"], eps=s["eps"])
    out = {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    return out if s["z"] is None else {**out, "dz": dz}


# ------------------------------------------------------------- plain forms --

def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    g = torch.sigmoid(v)
    return g * (1 + v * (1 - g))


def _plain_conv_step(s):
    x, w = s["x"].float(), s["weight"].float()
    index = s["index"].long()
    rows = torch.cat([s["state"][index].float(), x[:, None]], 1)      # [batch, 4, C]
    y = _silu((rows * w.t()).sum(1) + s["bias"].float())
    s["state"][index] = rows[:, 1:].to(torch.bfloat16)
    return {"y": y.to(torch.bfloat16), "state": s["state"]}


def _plain_conv_prompt(s):
    # One buffer holds each document behind its three rows of history.
    x, w, cu = s["x"], s["weight"].float(), s["cu"].long()
    index = s["index"].long()
    S, C = x.shape
    docs = cu.numel() - 1
    history = s["state"][index] * s["resume"][:, None, None]
    t = torch.arange(S, device=x.device)
    at = t + 3 * (torch.searchsorted(cu[1:], t, right=True) + 1)       # a token's row
    first = cu[:-1] + 3 * torch.arange(docs, device=x.device)          # a document's first history row
    three = torch.arange(3, device=x.device)
    buf = torch.empty(S + 3 * docs, C, dtype=torch.float32, device=x.device)
    buf[at] = x.float()
    buf[first[:, None] + three] = history.float()
    p = w[:, 0] * buf[at - 3] + w[:, 1] * buf[at - 2] + w[:, 2] * buf[at - 1] + w[:, 3] * buf[at]
    y = _silu(p + s["bias"].float())
    s["state"][index] = buf[(first + cu[1:] - cu[:-1])[:, None] + three].to(torch.bfloat16)
    return {"y": y.to(torch.bfloat16), "state": s["state"]}


def _doubling(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] over the first axis, by doubled steps; a is 0
    at the first token of a document, none of which is longer than `longest`."""
    k = 1
    while k < longest:
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _scan_terms(s):
    x, raw, A = s["x"].float(), s["dt"].float() + s["dt_bias"].float(), s["A"].float()
    step = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw)))
    rows, (C, N) = x.shape[0], A.shape
    G = s["B"].shape[1]
    wide = (rows, G, C // G)                                           # channels by group
    x, step, raw, A = x.view(wide), step.view(wide), raw.view(wide), A.view(G, C // G, N)
    return x, step, raw, A, s["B"].float()[:, :, None], s["C"].float()[:, :, None]


def _gated(s, y0):
    return y0 if s["z"] is None else y0 * _silu(s["z"].float())


def _plain_state_step(s):
    x, step, _, A, B, Cm = _scan_terms(s)
    index = s["index"].long()
    rows, (C, N) = x.shape[0], s["A"].shape
    h = s["state"][index].view(*x.shape, N)
    h = torch.exp(step[..., None] * A) * h + (step * x)[..., None] * B
    s["state"][index] = h.view(rows, C, N)
    y = (h * Cm).sum(-1).view(rows, C) + s["D"].float() * s["x"].float()
    return {"y": _gated(s, y).to(torch.bfloat16), "state": s["state"]}


def _plain_scan_prompt(s):
    x, step, _, A, B, Cm = _scan_terms(s)
    cu, index = s["cu"].long(), s["index"].long()
    rows, (C, N) = x.shape[0], s["A"].shape
    some = cu[1:] > cu[:-1]                                            # documents with tokens
    begin = s["state"][index] * s["resume"][:, None, None]
    a = torch.exp(step[..., None] * A)
    b = (step * x)[..., None] * B
    first = cu[:-1][some]
    b[first] += a[first] * begin[some].view(-1, *x.shape[1:], N)
    a[first] = 0
    h = _doubling(a, b, s["longest"])
    begin[some] = h[cu[1:][some] - 1].view(-1, C, N)
    s["state"][index] = begin
    y = (h * Cm).sum(-1).view(rows, C) + s["D"].float() * s["x"].float()
    return {"y": _gated(s, y).to(torch.bfloat16), "state": s["state"]}


def _plain_scan_train(s):
    bf = torch.bfloat16
    x, step, raw, A, B, Cm = _scan_terms(s)
    cu = s["cu"].long()
    rows, (C, N) = x.shape[0], s["A"].shape
    D = s["D"].float().view(x.shape[1:])
    a = torch.exp(step[..., None] * A)
    a[cu[:-1][cu[1:] > cu[:-1]]] = 0
    h = _doubling(a, (step * x)[..., None] * B, s["longest"])
    y0 = (h * Cm).sum(-1) + D * x
    y = _gated(s, y0.view(rows, C))
    # backward
    g = s["dy"].float()
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        dz = (g * y0.view(rows, C) * _dsilu(z)).to(bf)
        g = g * _silu(z)
    g = g.view(x.shape)
    after = torch.cat([a[1:], torch.zeros_like(a[:1])])
    lam = _doubling(after.flip(0), (g[..., None] * Cm).flip(0), s["longest"]).flip(0)
    del after
    dC = (g[..., None] * h).sum(2)
    v = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * a * lam         # lambda times the decayed state
    del h, a
    dB = (lam * (step * x)[..., None]).sum(2)
    along = (lam * B).sum(-1)
    del lam
    dstep = x * along + (v * A).sum(-1)
    draw = dstep * torch.sigmoid(raw)
    out = {"y": y.to(bf), "dx": (D * g + step * along).view(rows, C).to(bf),
           "ddt": draw.view(rows, C).to(bf),
           "dA": (v * step[..., None]).sum(0, dtype=torch.float64).view(C, N).to(s["A"].dtype),
           "dB": dB.to(bf), "dC": dC.to(bf),
           "dD": (g * x).sum(0, dtype=torch.float64).view(C).to(s["D"].dtype),
           "ddt_bias": draw.sum(0, dtype=torch.float64).view(C).to(s["dt_bias"].dtype)}
    return out if dz is None else {**out, "dz": dz}


def _plain_norm(s):
    bf = torch.bfloat16
    S, C = s["x"].shape
    G = s["groups"]
    x, w, b = s["x"].float().view(S, G, C // G), s["weight"].float(), s["bias"].float()
    mid = x - x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((mid * mid).mean(-1, keepdim=True) + s["eps"])
    xhat = mid * rstd
    v = xhat.view(S, C) * w + b
    z = None if s["z"] is None else s["z"].float()
    y = _silu(v) if z is None else v * _silu(z)
    if not s["train"]:
        return {"y": y.to(bf)}
    dy = s["dy"].float()
    dv = dy * _dsilu(v) if z is None else dy * _silu(z)
    dw = (dv * xhat.view(S, C)).sum(0, dtype=torch.float64)
    db = dv.sum(0, dtype=torch.float64)
    dh = (dv * w).view(S, G, C // G)
    dx = rstd * (dh - dh.mean(-1, keepdim=True) - xhat * (dh * xhat).mean(-1, keepdim=True))
    out = {"y": y.to(bf), "dx": dx.view(S, C).to(bf), "dweight": dw.to(s["weight"].dtype),
           "dbias": db.to(s["bias"].dtype)}
    return out if z is None else {**out, "dz": (dy * v * _dsilu(z)).to(bf)}


_PLAIN = {"conv_step": _plain_conv_step, "conv_prompt": _plain_conv_prompt,
          "state_step": _plain_state_step, "scan_prompt": _plain_scan_prompt,
          "scan_train": _plain_scan_train, "norm": _plain_norm}


def run(state):
    return _run_own(state) if own else _PLAIN[state["kind"]](state)


# -------------------------------------------------- the definitions, 64 bits --

def _edges(s):
    e = s["cu"].tolist()
    return list(zip(e, e[1:]))


def _exact_conv(s):
    w, bias = s["weight"].double(), s["bias"].double()
    after = s["state"].double()
    index = s["index"].tolist()
    if s["kind"] == "conv_step":
        # every row is a sequence of one token: all of them together
        past = after[s["index"].long()]
        seq = torch.cat([past, s["x"].double()[:, None]], 1)
        p = torch.einsum("bkc,ck->bc", seq, w) + bias
        after[s["index"].long()] = seq[:, 1:]
        return {"y": p / (1 + torch.exp(-p)), "state": after}
    docs, go_on = _edges(s), s["resume"].tolist()
    y = torch.empty(s["x"].shape, dtype=torch.float64, device=DEVICE)
    for d, (lo, hi) in enumerate(docs):
        past = after[index[d]] if go_on[d] else torch.zeros_like(after[0])
        seq = torch.cat([past, s["x"][lo:hi].double()])
        n = hi - lo
        p = bias.expand(n, -1).clone()
        for k in range(4):
            p += w[:, k] * seq[k:k + n]
        y[lo:hi] = p / (1 + torch.exp(-p))
        after[index[d]] = seq[n:]
    return {"y": y, "state": after}


def _exact_scan(s):
    x, dt = s["x"].double(), s["dt"].double() + s["dt_bias"].double()
    A, D = s["A"].double(), s["D"].double()
    rows, C = x.shape
    N, G = A.shape[1], s["B"].shape[1]
    step = torch.logaddexp(dt, torch.zeros_like(dt))
    B = s["B"].double().repeat_interleave(C // G, 1)                    # [rows, C, N]
    H = B * (step * x)[..., None]
    del B
    a = torch.exp(step[..., None] * A)
    z = None if s["z"] is None else s["z"].double()
    gate = torch.ones_like(x) if z is None else z / (1 + torch.exp(-z))
    after = None
    if s["kind"] == "state_step":
        after = s["state"].double()
        at = s["index"].long()
        H += a * after[at]
        after[at] = H
        docs = []
    else:
        docs = _edges(s)
    for d, (lo, hi) in enumerate(docs):
        h = torch.zeros(C, N, dtype=torch.float64, device=DEVICE)
        if s["kind"] == "scan_prompt":
            after = s["state"].double() if after is None else after
            at = int(s["index"][d])
            if bool(s["resume"][d]):
                h = after[at].clone()
        for t in range(lo, hi):                                         # one token after another
            h = torch.addcmul(H[t], a[t], h, out=H[t])
        if s["kind"] == "scan_prompt":
            after[at] = h
    Cm = s["C"].double()
    y0 = torch.matmul(H.view(rows, G, C // G, N), Cm[..., None]).view(rows, C) + D * x
    if s["kind"] != "scan_train":
        return {"y": y0 * gate, "state": after}
    dy = s["dy"].double()
    g = dy * gate
    out = {"y": y0 * gate, "dD": (g * x).sum(0)}
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        out["dz"] = dy * y0 * (sig + z * sig * (1 - sig))
    gw = g.view(rows, G, 1, C // G)
    out["dC"] = torch.matmul(gw, H.view(rows, G, C // G, N)).view(rows, G, N)
    # v: the state of the token before, decayed into this one
    v = torch.zeros_like(H)
    for lo, hi in docs:
        v[lo + 1:hi] = a[lo + 1:hi] * H[lo:max(lo, hi - 1)]
    L = H.zero_()
    L.view(rows, G, C // G, N).copy_(g.view(rows, G, C // G, 1) * Cm[:, :, None])
    for lo, hi in docs:
        for t in range(hi - 2, lo - 1, -1):                             # and back
            L[t].addcmul_(a[t + 1], L[t + 1])
    del a
    out["dB"] = torch.matmul((step * x).view(rows, G, 1, C // G), L.view(rows, G, C // G, N)).view(rows, G, N)
    along = torch.matmul(L.view(rows, G, C // G, N), s["B"].double()[..., None]).view(rows, C)
    v *= L
    dstep = x * along + torch.einsum("tcn,cn->tc", v, A)
    ddt = dstep / (1 + torch.exp(-dt))
    out["dx"] = D * g + step * along
    out["ddt"] = ddt
    out["ddt_bias"] = ddt.sum(0)
    out["dA"] = torch.einsum("tcn,tc->cn", v, step)
    return out


def _exact_norm(s):
    S, C = s["x"].shape
    G = s["groups"]
    w, b = s["weight"].double(), s["bias"].double()
    x = s["x"].double().view(S, G, -1)
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    scale = torch.rsqrt(var + s["eps"])
    n = ((x - mean) * scale).view(S, C)
    v = n * w + b
    u = v if s["z"] is None else s["z"].double()
    sig = 1 / (1 + torch.exp(-u))
    if not s["train"]:
        return {"y": v * sig if s["z"] is None else v * u * sig}
    dy = s["dy"].double()
    slope = sig * (1 + u * (1 - sig))
    out = {"y": v * sig if s["z"] is None else v * u * sig}
    if s["z"] is not None:
        out["dz"] = dy * v * slope
    dv = dy * (slope if s["z"] is None else u * sig)
    out["dweight"], out["dbias"] = (dv * n).sum(0), dv.sum(0)
    q = (dv * w).view(S, G, -1)
    n = n.view(S, G, -1)
    out["dx"] = ((q - q.mean(-1, keepdim=True) - n * (q * n).mean(-1, keepdim=True)) * scale).view(S, C)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] in ("conv_step", "conv_prompt"):
        return _exact_conv(s)
    return _exact_norm(s) if s["kind"] == "norm" else _exact_scan(s)


# ------------------------------------------------------------------- work --

def work(case):
    kind, C = case["kind"], case["C"]
    pb = 2 if case["params"] == "bf16" else 4
    if kind in ("conv_step", "conv_prompt"):
        rows = case["batch"] if kind == "conv_step" else case["S"]
        seqs = case["batch"] if kind == "conv_step" else case["docs"]
        # half of a prompt batch's sequences read a state, all of them write one
        states = seqs * 3 * C * 2 * (2 if kind == "conv_step" else 1.5)
        return {"bytes": rows * C * 4 + states + 5 * C * pb, "flops": rows * C * 12}
    if kind == "norm":
        S, gate = case["S"], int(case["gate"])
        fwd = S * C * 2 * (2 + gate) + 2 * C * pb
        bwd = S * C * 2 * (3 + 2 * gate) + 4 * C * pb
        return {"bytes": fwd + (bwd if case["train"] else 0),
                "flops": S * C * (14 + (26 if case["train"] else 0))}
    N, G, gate = case["N"], case["groups"], int(case["gate"])
    rows = case["batch"] if kind == "state_step" else case["S"]
    params = (C * N + 2 * C) * pb
    fwd = rows * C * 2 * (3 + gate) + rows * G * N * 4 + params
    # a token and channel: the step size, N states (decay, its exponential, input,
    # update, output) and the gate
    flops = rows * C * (7 * N + 12 + 5 * gate)
    if kind == "scan_train":
        bwd = rows * C * 2 * (5 + 2 * gate) + rows * G * N * 8 + 2 * params
        return {"bytes": fwd + bwd, "flops": flops + rows * C * (22 * N + 20 + 10 * gate)}
    seqs = case["batch"] if kind == "state_step" else case["docs"]
    states = seqs * C * N * 4 * (2 if kind == "state_step" else 1.5)
    return {"bytes": fwd + states, "flops": flops}
