"""The example's sequences go on from states that were put aside: their tokens are
those of states that stayed, within what the codes' steps allow, and those of
another sequence's states are not."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_layer.py")
DEV = "cuda:0"
WIDTH, LAYERS, TOKENS = 96, 2, 6


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("recurrent_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


# A layer's BF16 results, five of them, whole steps where sums differ in their order.
ROUNDED = LAYERS * 5 * 2.0 ** -7
# A value comes back within half a step: of int8, of its block's largest value, which
# is at most 4 times the root mean square of 64 values of a normal distribution; of
# e4m3, of the value.  The recurrence's states are linear in those before the tokens,
# with factors below 1, and contract those of the convolution (SiLU's slope is at most
# 1.1, the weights' row norm below 1): two caches a layer give twice the relative
# difference at most, each layer once more.  The outputs, in which the tokens' own
# stream is most, differ by less.
ALLOWED = {torch.int8: ROUNDED + LAYERS * 2 * 4 * 0.5 / 127, torch.float8_e4m3fn: ROUNDED + LAYERS * 2 * 2.0 ** -4}


@pytest.mark.parametrize("code", list(ALLOWED))
def test_tokens_after_states_put_aside(example, code):
    torch.manual_seed(4)
    model = example.RecurrentModel(WIDTH, LAYERS, device=DEV)
    lengths, n = [150, 9, 37], 3
    caches, slots = model.caches(6), ints([5, 1, 3])
    edges = ints([0, 150, 159, 196])
    model.prefill(torch.randn(sum(lengths), WIDTH, device=DEV).bfloat16(), edges, caches, slots)
    tokens = [torch.randn(n, WIDTH, device=DEV).bfloat16() for _ in range(TOKENS)]
    stayed = [[c.clone() for c in layer] for layer in caches]
    want = torch.stack([model.step(u, stayed, slots) for u in tokens], 1)
    pool, places = example.Pool(caches, 4, code), ints([3, 0, 1])
    pool.put(caches, slots, places)
    results, states = [], []
    for back in ([0, 2, 4], [2, 4, 0]):  # the second: each row has another sequence's states
        held = [[torch.full_like(c, 7.0) for c in layer] for layer in caches]
        pool.take(held, ints([0, 2, 4]), places)
        results.append(off(torch.stack([model.step(u, held, ints(back)) for u in tokens], 1), want))
        states.append([off(h[1][back], s[1][[5, 1, 3]]) for h, s in zip(held, stayed)])
    for right, wrong in [results, *zip(*states)]:
        print("%s: %.2e, of other sequences %.2e, allowed %.2e" % (code, right, wrong, ALLOWED[code]))
        assert right <= ALLOWED[code] and right < wrong
    for _, wrong in zip(*states):
        assert wrong > ALLOWED[code]


@pytest.mark.parametrize("code", list(ALLOWED))
def test_answers_after_states_put_aside(example, code):
    """The example's own answers against the whole sequences."""
    torch.manual_seed(5)
    model = example.RecurrentModel(WIDTH, LAYERS, device=DEV)
    got, want = example.answer(model, WIDTH, [150, 2, 37], TOKENS, DEV, code)
    assert off(got, want) <= ALLOWED[code] + ROUNDED < off(got, want[[1, 2, 0]])
