"""Seeded inputs for the tests of the state space layer's operators."""
import math

import torch


def edges(lengths):
    e = [0]
    for n in lengths:
        e.append(e[-1] + n)
    return e


class Maker:
    def __init__(self, seed, device):
        self.g, self.device = torch.Generator().manual_seed(seed), device

    def normal(self, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=self.g) * std + mean).to(dtype).to(self.device)

    def uniform(self, *shape, lo, hi, dtype=torch.float32):
        return (torch.rand(*shape, generator=self.g) * (hi - lo) + lo).to(dtype).to(self.device)


def scan_inputs(seed, lengths, C, N, G=1, *, device, params=torch.float32, gate=True, D=True, bias=True,
                softplus=True, wide=False, rows=None):
    """x, dt, A, B, C, D, z, dt_bias and the documents.  wide: x, dt, z, B and C
    are cut out of wider rows, B and C at an odd column."""
    m = Maker(seed, device)
    e = edges(lengths)
    S = e[-1] if rows is None else rows

    def act(std=1.0, mean=0.0, lift=False):
        pad = 6 if wide else 0
        t = m.normal(S, C + pad, std=std, mean=mean)
        if lift:
            t = t.abs()
        return t[:, pad // 2:pad // 2 + C] if wide else t

    k = {"x": act(), "A": (-(torch.arange(1, N + 1, device=device)
                             * torch.exp(m.normal(C, N, std=0.1, dtype=torch.float32)))).to(params)}
    # step sizes around 0.001 to 0.3, some of them over 1
    k["dt"] = act(std=0.5) if softplus else act(std=0.1, lift=True)
    step = torch.exp(m.uniform(C, lo=math.log(1e-3), hi=math.log(0.3)))
    k["dt_bias"] = (step + torch.log(-torch.expm1(-step))).to(params) if bias and softplus else None
    if softplus and not bias:
        k["dt"] = act(std=1.0, mean=-3.0)
    k["D"] = m.normal(C, mean=1.0, std=0.2, dtype=params) if D else None
    k["z"] = act() if gate else None
    both = m.normal(S, 2 * G * N + (3 if wide else 0))
    off = 3 if wide else 0
    if wide:
        k["B"] = both[:, off:off + G * N].unflatten(1, (G, N))
        k["C"] = both[:, off + G * N:].unflatten(1, (G, N))
    else:
        k["B"] = both[:, :G * N].contiguous().unflatten(1, (G, N))
        k["C"] = both[:, G * N:].contiguous().unflatten(1, (G, N))
    return k, list(zip(e, e[1:])), torch.tensor(e, dtype=torch.int32, device=device)
