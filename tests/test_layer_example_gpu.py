"""The example's layers: they run, train and serve; the gradients of their
parameters against a plain model in 64 bits; prompts in parts with single
tokens behind them against the whole sequences, also where the sequences were
put aside in between."""
import importlib.util
import os

import pytest
import torch
from torch.nn import functional as F

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_layer.py")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("recurrent_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain(model, p, u, docs):
    """The model's forward pass on the parameters p (64 bits, by their names)."""
    def norm(x, name):
        return F.layer_norm(x, x.shape[-1:], p[name + "norm_weight"], p[name + "norm_bias"], 1e-5)

    stream, branch = 0, u
    for n, layer in enumerate(model.layers):
        at = "layers.%d." % n
        stream = stream + branch
        x, z = (norm(stream, at) @ p[at + "proj_in.weight"].t()).split(layer.inner, dim=-1)
        past = [F.pad(x[lo:hi], (0, 0, 3, 0)) for lo, hi in docs]
        w = p[at + "conv_weight"]
        x = torch.cat([sum(w[:, k] * s[k:k + s.shape[0] - 3] for k in range(4)) for s in past])
        x = F.silu(x + p[at + "conv_bias"])
        r, i = (x @ p[at + "proj_gates.weight"].t() + p[at + "proj_gates.bias"]).split(layer.inner, dim=-1)
        u_ = 16 * F.softplus(p[at + "decay"]) * torch.sigmoid(r)
        a, b = torch.exp(-u_ / 2), (-torch.expm1(-u_)).sqrt() * torch.sigmoid(i) * x
        hs = []
        for lo, hi in docs:
            h = torch.zeros_like(b[0])
            for t in range(lo, hi):
                h = a[t] * h + b[t]
                hs.append(h)
        branch = (torch.stack(hs) * F.silu(z)) @ p[at + "proj_out.weight"].t()
    return norm(stream + branch, "")


def test_gradients_of_the_parameters(example):
    torch.manual_seed(3)
    lengths = [40, 1, 90, 70]
    model = example.RecurrentModel(64, 2, device=DEV)
    u = torch.randn(sum(lengths), 64, device=DEV).bfloat16()
    dy = torch.randn(sum(lengths), 64, device=DEV).bfloat16()
    e = [0, 40, 41, 131, 201]
    y = model(u, torch.tensor(e, dtype=torch.int32, device=DEV))
    y.backward(dy)
    p = {n: t.detach().double().requires_grad_() for n, t in model.named_parameters()}
    want = plain(model, p, u.double(), list(zip(e, e[1:])))
    want.backward(dy.double())
    # Two layers of five results in BF16 one after another (the norm, the
    # projections, the convolution, the recurrence) and as many gradients on the
    # way back, each off by half a step at most, 2^-8 of its values.
    allowed = 2 * 10 * 2.0 ** -8
    assert float((y.double() - want).norm() / want.norm()) <= allowed / 2
    for n, t in model.named_parameters():
        off = float((t.grad.double() - p[n].grad).norm() / p[n].grad.norm())
        print("%-28s %.2e" % (n, off))
        assert off <= allowed, n


@pytest.mark.parametrize("width,layers", [(128, 2), (80, 3)])
def test_model_trains_and_answers(example, width, layers):
    torch.manual_seed(1)
    model = example.RecurrentModel(width, layers, device=DEV)
    losses = example.train(model, width, [60, 1, 200, 123], 5, DEV)
    assert all(v == v and v < float("inf") for v in losses)
    got, want = example.answer(model, width, [150, 2, 37], 6, DEV)
    # as above, and whole steps where sums differ in their order
    off = float((got.float() - want.float()).norm() / want.float().norm())
    print("relative difference %.2e" % off)
    assert off <= layers * 5 * 2.0 ** -7


@pytest.mark.parametrize("code,half", [(torch.int8, 0.5 / 127), (torch.float8_e4m3fn, 16.0 / 448)])
def test_sequences_put_aside(example, code, half):
    """Each value comes back within half of a code's largest step, and the
    sequences go on."""
    torch.manual_seed(2)
    model = example.RecurrentModel(96, 2, device=DEV)
    caches = model.caches(7)
    cu = torch.tensor([0, 50, 90], dtype=torch.int32, device=DEV)
    slots = torch.tensor([5, 2], dtype=torch.int32, device=DEV)
    model.prefill(torch.randn(90, 96, device=DEV).bfloat16(), cu, caches, slots)
    pool, places = example.Pool(caches, 3, code), torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    before = [[c.clone() for c in layer] for layer in caches]
    pool.put(caches, slots, places)
    pool.take(caches, torch.tensor([0, 6], dtype=torch.int32, device=DEV), places)
    for was, now in zip(before, caches):
        for a, b in zip(was, now):
            assert torch.equal(a[[1, 2, 3, 4, 5]], b[[1, 2, 3, 4, 5]])
            for src, dst in ((5, 0), (2, 6)):
                x, y = a[src].double().flatten(), b[dst].double().flatten()
                n = (x.numel() + 63) // 64 * 64 - x.numel()
                top = F.pad(x, (0, n)).view(-1, 64).abs().amax(1).repeat_interleave(64)[:x.numel()]
                # the scale's rounding, and the value's own to the cache's type
                step = torch.finfo(a.dtype).eps / 2
                assert bool(((x - y).abs() <= top * half * (1 + 2.0 ** -22) + y.abs() * (step + 2.0 ** -23)).all())
    got, want = example.answer(model, 96, [150, 2, 37], 6, DEV, code)
    assert got.shape == want.shape and bool(torch.isfinite(got).all())
