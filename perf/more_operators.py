"""The operators of a recurrent layer around the packed causal convolution,
measured: the gated linear recurrence (prompts, training, single tokens), the
layer norm on the residual stream, and carried states that are put aside in 8
bits and taken back.

``run`` computes them in plain torch operations, or, where ``own`` is true,
through this package's entry points.  ``exact`` computes the same outputs from
the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 64          # values of a state that share a scale
SCALE = 8.0         # the recurrence's decay at an open gate is exp(-SCALE softplus(decay))


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One sequence decoding one token: the latency of a single call.
        {"name": "recur_step_1", "kind": "recur_step", "batch": 1, "C": 2048, "gate": True,
         "params": "f32"},
        # A full serving batch, one token each, slots scattered over a cache.
        {"name": "recur_step_1000", "kind": "recur_step", "batch": 1000, "C": 4096, "gate": True,
         "params": "bf16"},
        # One short prompt: latency again, too few rows to fill the machine.
        {"name": "recur_prompt_short", "kind": "recur_prompt", "S": 77, "docs": 1, "C": 2048, "gate": True,
         "params": "f32"},
        # A long prefill batch at the convolution's headline width and documents.
        {"name": "recur_prompt_long", "kind": "recur_prompt", "S": 65536, "docs": 22, "C": 4096,
         "gate": True, "params": "f32"},
        # A small training batch: odd length, ragged documents, rows that are not a
        # multiple of a cache line, parameters kept in bfloat16, no gate.
        {"name": "recur_train_ragged", "kind": "recur_train", "S": 1543, "docs": 11, "C": 520,
         "gate": False, "params": "bf16"},
        # A training batch of packed documents.
        {"name": "recur_train_large", "kind": "recur_train", "S": 16384, "docs": 6, "C": 4096,
         "gate": True, "params": "f32"},
        # The norm before a layer in a decoding batch.
        {"name": "norm_serve", "kind": "norm", "S": 33, "C": 520, "residual": True, "train": False,
         "params": "f32"},
        # The norm of a prefill batch, wide rows.
        {"name": "norm_prompt", "kind": "norm", "S": 8192, "C": 8192, "residual": True, "train": False,
         "params": "bf16"},
        # An odd training batch: rows of no whole number of vectors, no residual.
        {"name": "norm_train_odd", "kind": "norm", "S": 1543, "C": 1001, "residual": False, "train": True,
         "params": "f32"},
        # A training batch: the residual stream's sum and norm, and their gradients.
        {"name": "norm_train", "kind": "norm", "S": 16384, "C": 4096, "residual": True, "train": True,
         "params": "f32"},
        # One sequence that is put aside and one that is taken back.
        {"name": "park_1", "kind": "park", "batch": 1, "state": "scan", "C": 2048, "N": 16, "code": "int8"},
        # A full serving batch of the selective scan's states that changes places.
        {"name": "park_512", "kind": "park", "batch": 512, "state": "scan", "C": 4096, "N": 16,
         "code": "e4m3"},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number spread over [lo, hi] by its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    kind = rng.choice(["recur_step", "recur_prompt", "recur_train", "recur_train", "norm", "norm", "park"])
    params, gate = rng.choice(["f32", "bf16"]), rng.random() < 0.5
    if kind == "recur_step":
        return {"kind": kind, "batch": _spread(rng, 1, 1000), "C": _spread(rng, 64, 8192), "gate": gate,
                "params": params}
    if kind.startswith("recur"):
        C = _spread(rng, 64, 8192, rng.choice([1, 2, 8, 64]))
        most = 65536 if kind == "recur_prompt" else 16384
        S = _spread(rng, 1, min(65536, most * 4096 // C))
        return {"kind": kind, "S": S, "docs": _spread(rng, 1, 64), "C": C, "gate": gate, "params": params}
    if kind == "norm":
        C = _spread(rng, 64, 8192, rng.choice([1, 8, 64]))
        return {"kind": kind, "S": _spread(rng, 1, min(65536, 16384 * 4096 // C)), "C": C,
                "residual": rng.random() < 0.5, "train": rng.random() < 0.5, "params": params}
    state = rng.choice(["scan", "recur", "conv"])
    N = rng.choice([8, 13, 16, 64]) if state == "scan" else 1 if state == "recur" else 3
    C = _spread(rng, 64, 8192, 8)
    return {"kind": kind, "batch": _spread(rng, 1, min(1000, 512 * 4096 * 16 // (C * N))), "state": state,
            "C": C, "N": N, "code": rng.choice(["int8", "e4m3"])}


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


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    m, host = _Maker(seed), random.Random(seed)
    kind, C = case["kind"], case["C"]
    bf = torch.bfloat16
    s = {"kind": kind}
    if kind == "park":
        # Sequences leave a cache for a pool, and come back into other slots.
        n, N = case["batch"], case["N"]
        tail = {"scan": (C, N), "recur": (C,), "conv": (3, C)}[case["state"]]
        slots, index = _slots(2 * n, host)
        # a channel's states are of about one size, sizes differ from channel to channel
        size = torch.exp(m.normal(C))
        state = m.normal(slots, *tail) * (size[:, None] if case["state"] == "scan" else size)
        s["state"] = state.to(bf if case["state"] == "conv" else torch.float32)
        s["leave"], s["enter"] = _ints(index[:n]), _ints(index[n:])
        pool, places = _slots(n, host)
        s["places"] = _ints(places)
        E = math.prod(tail)
        s["codes"] = torch.zeros(pool, E, dtype=torch.int8, device=DEVICE)
        if case["code"] == "e4m3":
            s["codes"] = s["codes"].view(torch.float8_e4m3fn)
        s["scales"] = torch.zeros(pool, (E + BLOCK - 1) // BLOCK, device=DEVICE)
        return s
    pt = bf if case["params"] == "bf16" else torch.float32
    if kind == "norm":
        S = case["S"]
        s["train"], s["eps"] = case["train"], 1e-5
        s["x"] = m.normal(S, C).to(bf)
        # the stream has grown over the layers before
        s["residual"] = m.normal(S, C, std=3.0, mean=0.3).to(bf) if case["residual"] else None
        if case["train"]:
            s["dy"] = m.normal(S, C).to(bf)
            s["dstream"] = m.normal(S, C).to(bf) if case["residual"] else None
        s["weight"] = m.uniform(C, lo=0.5, hi=1.5).to(pt)
        s["bias"] = m.normal(C, std=0.1).to(pt)
        return s
    # The recurrence: decays of 0.9 to 0.999 a token at an open gate; the two gates
    # are halves of one projection's result, as a layer has them.
    rows = case["batch"] if kind == "recur_step" else case["S"]
    s["x"] = m.normal(rows, C).to(bf)
    gates = m.normal(rows, 2 * C).to(bf)
    s["r"], s["i"] = gates[:, :C], gates[:, C:]
    s["z"] = m.normal(rows, C).to(bf) if case["gate"] else None
    soft = -torch.log(m.uniform(C, lo=0.9, hi=0.999)) / SCALE
    s["decay"] = (soft + torch.log(-torch.expm1(-soft))).to(pt)
    if kind != "recur_step":
        edges = [0]
        for n in _lengths(case):
            edges.append(edges[-1] + n)
        s["cu"] = _ints(edges)
        s["longest"] = max(_lengths(case))
    if kind == "recur_train":
        s["dy"] = m.normal(rows, C).to(bf)
        return s
    count = rows if kind == "recur_step" else case["docs"]
    slots, index = _slots(count, host)
    s["state"] = m.normal(slots, C)
    s["index"] = _ints(index)
    if kind == "recur_prompt":
        s["resume"] = torch.tensor([i % 2 for i in range(count)], dtype=torch.bool, device=DEVICE)
    return s


# --------------------------------------------- the framework's entry points --

def _run_own(s):
    import varlen_depthwise_causal_amd as vdc
    kind = s["kind"]
    if kind == "recur_step":
        y = vdc.gated_recurrence_update(s["x"], s["r"], s["i"], s["decay"], s["state"], z=s["z"], scale=SCALE,
                                        state_index=s["index"])
        return {"y": y, "state": s["state"]}
    if kind == "recur_prompt":
        y = vdc.gated_recurrence_fwd(s["x"], s["r"], s["i"], s["decay"], s["cu"], z=s["z"], scale=SCALE,
                                     state=s["state"], state_index=s["index"], resume=s["resume"])
        return {"y": y, "state": s["state"]}
    if kind == "recur_train":
        y, keep = vdc.gated_recurrence_fwd(s["x"], s["r"], s["i"], s["decay"], s["cu"], z=s["z"], scale=SCALE,
                                           keep=True)
        dx, dr, di, ddecay, dz = vdc.gated_recurrence_bwd(s["x"], s["r"], s["i"], s["decay"], s["cu"], s["dy"],
                                                          keep, z=s["z"], scale=SCALE)
        out = {"y": y, "dx": dx, "dr": dr, "di": di, "ddecay": ddecay}
        return out if s["z"] is None else {**out, "dz": dz}
    if kind == "park":
        vdc.state_quantize(s["state"], s["codes"], s["scales"], state_index=s["leave"],
                           pool_index=s["places"])
        vdc.state_dequantize(s["codes"], s["scales"], s["state"], pool_index=s["places"],
                             state_index=s["enter"])
        return {"state": s["state"], "scales": s["scales"]}
    y, stream = vdc.layer_norm_fwd(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], eps=s["eps"])
    out = {"y": y} if s["residual"] is None else {"y": y, "stream": stream}
    if not s["train"]:
        return out
    dx, dw, db = vdc.layer_norm_bwd(stream, s["weight"], s["dy"], bias=s["bias"], dstream=s["dstream"],
                                    eps=s["eps"])
    return {**out, "dx": dx, "dweight": dw, "dbias": db}


# ------------------------------------------------------------- plain forms --

def _silu(v):
    return v * torch.sigmoid(v)


def _doubling(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] over the first axis, by doubled steps; a is 0
    at the first token of a document, none of which is longer than `longest`."""
    k = 1
    while k < longest:
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _recur_terms(s):
    """Decays, the inputs' factors and the gated inputs."""
    decay = s["decay"].float()
    soft = torch.where(decay > 20, decay, torch.log1p(torch.exp(decay)))
    log_a = -SCALE * soft * torch.sigmoid(s["r"].float())
    a = torch.exp(log_a)
    m = torch.sqrt(-torch.expm1(2 * log_a))
    return log_a, a, m, torch.sigmoid(s["i"].float()) * s["x"].float()


def _gated(s, h):
    return (h if s["z"] is None else h * _silu(s["z"].float())).to(torch.bfloat16)


def _plain_recur_step(s):
    _, a, m, gx = _recur_terms(s)
    index = s["index"].long()
    h = a * s["state"][index] + m * gx
    s["state"][index] = h
    return {"y": _gated(s, h), "state": s["state"]}


def _plain_recur_prompt(s):
    _, a, m, gx = _recur_terms(s)
    b = m * gx
    cu, index = s["cu"].long(), s["index"].long()
    some = cu[1:] > cu[:-1]                                            # documents with tokens
    begin = s["state"][index] * s["resume"][:, None]
    first = cu[:-1][some]
    b[first] += a[first] * begin[some]
    a[first] = 0
    h = _doubling(a, b, s["longest"])
    begin[some] = h[cu[1:][some] - 1]
    s["state"][index] = begin
    return {"y": _gated(s, h), "state": s["state"]}


def _plain_recur_train(s):
    bf = torch.bfloat16
    log_a, a, m, gx = _recur_terms(s)
    cu, decay = s["cu"].long(), s["decay"].float()
    a[cu[:-1][cu[1:] > cu[:-1]]] = 0
    h = _doubling(a, m * gx, s["longest"])
    y = _gated(s, h)
    # backward
    g, dz = s["dy"].float(), None
    if s["z"] is not None:
        z = s["z"].float()
        k = torch.sigmoid(z)
        dz = (g * h * (k * (1 + z * (1 - k)))).to(bf)
        g = g * _silu(z)
    after = torch.cat([a[1:], torch.zeros_like(a[:1])])
    lam = _doubling(after.flip(0), g.flip(0), s["longest"]).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * a          # the decayed state of the token before
    # log a has the state's decay in it and the inputs' factor m = sqrt(1 - a^2)
    dlog = lam * (before - gx * torch.exp(2 * log_a) / m)
    rest = dlog * log_a
    dgx = lam * m
    gi = torch.sigmoid(s["i"].float())
    soft = torch.where(decay > 20, decay, torch.log1p(torch.exp(decay)))
    ddecay = rest.sum(0, dtype=torch.float64) * (torch.sigmoid(decay) / soft).double()
    out = {"y": y, "dx": (dgx * gi).to(bf), "dr": (rest * (1 - torch.sigmoid(s["r"].float()))).to(bf),
           "di": (dgx * gx * (1 - gi)).to(bf), "ddecay": ddecay.to(s["decay"].dtype)}
    return out if dz is None else {**out, "dz": dz}


def _plain_norm(s):
    bf = torch.bfloat16
    w, b = s["weight"].float(), s["bias"].float()
    stream = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(bf)
    x = stream.float()
    mid = x - x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((mid * mid).mean(-1, keepdim=True) + s["eps"])
    xhat = mid * rstd
    out = {"y": (xhat * w + b).to(bf)}
    if s["residual"] is not None:
        out["stream"] = stream
    if not s["train"]:
        return out
    dy = s["dy"].float()
    q = dy * w
    dx = rstd * (q - q.mean(-1, keepdim=True) - xhat * (q * xhat).mean(-1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["dstream"].float()
    return {**out, "dx": dx.to(bf), "dweight": (dy * xhat).sum(0, dtype=torch.float64).to(s["weight"].dtype),
            "dbias": dy.sum(0, dtype=torch.float64).to(s["bias"].dtype)}


def _plain_park(s):
    state, leave, enter, places = s["state"], s["leave"].long(), s["enter"].long(), s["places"].long()
    n, E = leave.numel(), s["codes"].shape[1]
    blocks = s["scales"].shape[1]
    v = torch.zeros(n, blocks * BLOCK, device=state.device)
    v[:, :E] = state[leave].float().reshape(n, E)
    v = v.view(n, blocks, BLOCK)
    e4m3 = s["codes"].dtype == torch.float8_e4m3fn
    # rounded once, and quotients next to the border of two codes; a block with
    # nothing of 2^-64 or more is zeros
    most = v.abs().amax(-1)
    scale = torch.where(most < 2.0 ** -64, 0.0, (most.double() / (448.0 if e4m3 else 127.0)).float())
    t = v.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[..., None]
    if e4m3:
        # three bits after the first one, none of them below 2^-9
        step = torch.exp2(torch.frexp(t)[1].clamp(min=-5).double() - 4)
        q = torch.round(t / step) * step
    else:
        q = torch.round(t)
    back = (q.float() * scale[..., None]).view(n, -1)[:, :E]
    q = q.view(n, -1)[:, :E].float()
    s["codes"].view(torch.int8)[places] = q.to(s["codes"].dtype).view(torch.int8)
    s["scales"][places] = scale
    state[enter] = back.to(state.dtype).view(n, *state.shape[1:])
    return {"state": state, "scales": s["scales"]}


_PLAIN = {"recur_step": _plain_recur_step, "recur_prompt": _plain_recur_prompt,
          "recur_train": _plain_recur_train, "norm": _plain_norm, "park": _plain_park}


def run(state):
    return _run_own(state) if own else _PLAIN[state["kind"]](state)


# -------------------------------------------------- the definitions, 64 bits --

def _open(v):
    return 1 / (1 + torch.exp(-v))


def _exact_recur(s):
    x, decay = s["x"].double(), s["decay"].double()
    r, i = _open(s["r"].double()), _open(s["i"].double())
    soft = torch.logaddexp(decay, torch.zeros_like(decay))
    u = 2 * SCALE * soft * r                                           # a^2 = exp(-u)
    a, m = torch.exp(-u / 2), (-torch.expm1(-u)).sqrt()
    H = m * i * x
    z = None if s["z"] is None else s["z"].double()
    gate = 1.0 if z is None else z * _open(z)
    after = s["state"].double() if "state" in s else None
    if s["kind"] == "recur_step":
        at = s["index"].long()
        after[at] = H = H + a * after[at]
        return {"y": H * gate, "state": after}
    e = s["cu"].tolist()
    docs = list(zip(e, e[1:]))
    zero = torch.zeros_like(x[:1])
    for d, (lo, hi) in enumerate(docs):
        h = zero[0]
        if after is not None and bool(s["resume"][d]):
            h = after[int(s["index"][d])].clone()
        for t in range(lo, hi):                                        # one token after another
            h = torch.addcmul(H[t], a[t], h, out=H[t])
        if after is not None:
            after[int(s["index"][d])] = h
    if after is not None:
        return {"y": H * gate, "state": after}
    dy = s["dy"].double()
    out = {"y": H * gate}
    if z is not None:
        k = _open(z)
        out["dz"] = dy * H * (k + z * k * (1 - k))
    L = dy * gate
    first = torch.zeros(x.shape[0], dtype=torch.bool, device=DEVICE)
    for lo, hi in docs:
        if hi > lo:
            first[lo] = True
        for t in range(hi - 2, lo - 1, -1):                            # and back
            L[t].addcmul_(a[t + 1], L[t + 1])
    past = torch.cat([zero, H[:-1]]).masked_fill(first[:, None], 0)
    # d/du of a = exp(-u / 2) is -a / 2, of m = sqrt(1 - exp(-u)) it is a^2 / (2 m)
    du = L * (i * x * a * a / m - a * past) / 2
    out["dx"], out["di"] = L * m * i, L * m * x * i * (1 - i)
    out["dr"] = du * u * (1 - r)
    out["ddecay"] = (du * 2 * SCALE * r).sum(0) * _open(decay)
    return out


def _exact_norm(s):
    x = s["x"].double()
    out = {}
    if s["residual"] is not None:
        out["stream"] = x + s["residual"].double()
        x = out["stream"].float().bfloat16().double()                  # what the stream holds
    w, b = s["weight"].double(), s["bias"].double()
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    scale = torch.rsqrt(var + s["eps"])
    n = (x - mean) * scale
    out["y"] = n * w + b
    if not s["train"]:
        return out
    dy = s["dy"].double()
    out["dweight"], out["dbias"] = (dy * n).sum(0), dy.sum(0)
    q = dy * w
    out["dx"] = (q - q.mean(-1, keepdim=True) - n * (q * n).mean(-1, keepdim=True)) * scale
    if s["residual"] is not None:
        out["dx"] = out["dx"] + s["dstream"].double()
    return out


def _exact_park(s):
    """Codes by the nearest of all that there are, ties to the even one."""
    state, scales = s["state"].double(), s["scales"].double()
    e4m3 = s["codes"].dtype == torch.float8_e4m3fn
    if e4m3:
        codes = torch.arange(127, dtype=torch.uint8, device=DEVICE).view(torch.float8_e4m3fn).double()
    else:
        codes = torch.arange(128, device=DEVICE).double()              # by magnitude: code k is entry k
    middle = (codes[1:] + codes[:-1]) / 2
    for a, b, p in zip(s["leave"].tolist(), s["enter"].tolist(), s["places"].tolist()):
        flat = state[a].reshape(-1)
        back = torch.empty_like(flat)
        for lo in range(0, flat.numel(), BLOCK * 65536):
            part = flat[lo:lo + BLOCK * 65536]
            n = (part.numel() + BLOCK - 1) // BLOCK
            v = torch.cat([part, part.new_zeros(n * BLOCK - part.numel())]).view(n, BLOCK)
            one = (v.abs().amax(1) / codes[-1]).float().double()       # a scale is held in 32 bits
            one[v.abs().amax(1) < 2.0 ** -64] = 0
            t = v.abs() / torch.where(one > 0, one, torch.ones_like(one))[:, None]
            k = torch.searchsorted(middle, t)                          # middles below t
            tie = (t == middle[k.clamp(max=middle.numel() - 1)]) & (k % 2 == 1)
            q = codes[k + tie] * torch.sign(v) * (one > 0)[:, None]
            back[lo:lo + part.numel()] = (q * one[:, None]).view(-1)[:part.numel()]
            scales[p, lo // BLOCK:lo // BLOCK + n] = one
        state[b] = back.view(state.shape[1:])
    return {"state": state, "scales": scales}


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "park":
        return _exact_park(s)
    return _exact_norm(s) if s["kind"] == "norm" else _exact_recur(s)


# ------------------------------------------------------------------- work --

def work(case):
    kind, C = case["kind"], case["C"]
    if kind == "park":
        # a state read and its codes and scales written, these read and a state written
        E = C * case["N"]
        held = E + (E + BLOCK - 1) // BLOCK * 4
        return {"bytes": case["batch"] * 2 * (E * (2 if case["state"] == "conv" else 4) + held),
                "flops": case["batch"] * E * 4}
    pb = 2 if case["params"] == "bf16" else 4
    if kind == "norm":
        S, res = case["S"], int(case["residual"])
        fwd = S * C * 2 * (2 + 2 * res) + 2 * C * pb
        bwd = S * C * 2 * (3 + res) + 3 * C * pb
        return {"bytes": fwd + (bwd if case["train"] else 0),
                "flops": S * C * (8 + res + (14 + res if case["train"] else 0))}
    gate = int(case["gate"])
    rows = case["batch"] if kind == "recur_step" else case["S"]
    fwd, flops = rows * C * 2 * (4 + gate) + C * pb, rows * C * (20 + 5 * gate)
    if kind == "recur_train":
        # the backward needs the inputs again
        bwd = rows * C * 2 * (7 + 2 * gate) + 2 * C * pb
        return {"bytes": fwd + bwd, "flops": flops + rows * C * (40 + 12 * gate)}
    seqs = rows if kind == "recur_step" else case["docs"]
    return {"bytes": fwd + seqs * C * 4 * (2 if kind == "recur_step" else 1.5), "flops": flops}
