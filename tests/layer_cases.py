"""Seeded inputs for the tests of the recurrent layer's operators."""
import torch

from ssm_cases import Maker, edges


def recur_inputs(seed, lengths, C, *, device, params=torch.float32, gate=True, wide=False, rows=None, low=0.9,
                 high=0.999, scale=8.0):
    """x, r, i, decay, z and the documents; decays of `low` to `high` a token at an
    open gate.  wide: the activations are cut out of wider rows at an odd column."""
    m = Maker(seed, device)
    e = edges(lengths)
    S = e[-1] if rows is None else rows

    def act(**k):
        t = m.normal(S, C + (7 if wide else 0), **k)
        return t[:, 3:3 + C] if wide else t

    k = {"x": act(), "r": act(std=2.0), "i": act(std=2.0), "z": act() if gate else None}
    soft = (-torch.log(m.uniform(C, lo=low, hi=high)) / scale).double()
    k["decay"] = (soft + torch.log(-torch.expm1(-soft))).to(params)
    return k, list(zip(e, e[1:])), torch.tensor(e, dtype=torch.int32, device=device)


def norm_inputs(seed, S, C, *, device, params=torch.float32, bias=True, residual=True, wide=False, mean=0.3,
                std=3.0):
    m = Maker(seed, device)

    def act(**k):
        t = m.normal(S, C + (5 if wide else 0), **k)
        return t[:, 1:1 + C] if wide else t

    k = {"x": act(), "residual": act(std=std, mean=mean) if residual else None, "dy": act(),
         "dstream": act() if residual else None}
    k["weight"] = m.uniform(C, lo=0.5, hi=1.5, dtype=params)
    k["bias"] = m.normal(C, std=0.1, dtype=params) if bias else None
    return k
