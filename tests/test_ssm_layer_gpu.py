"""The example layer: training lowers its loss, and prompts in parts with
single tokens behind them answer as the whole sequences do."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ssm_layer.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("ssm_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("width,states,groups", [(128, 16, 1), (96, 24, 2)])
def test_layer_trains_and_answers(example, width, states, groups):
    torch.manual_seed(1)
    layer = example.SsmLayer(width, states, groups, device="cuda:0")
    losses = example.train(layer, width, [60, 1, 200, 123], 20, "cuda:0")
    print(losses)
    assert losses[-1] < 0.9 * losses[0]
    got, want = example.answer(layer, width, [150, 2, 37], 6, "cuda:0")
    # Five roundings to BF16 stand one after another (the projections, the
    # convolution, the scan, the norm); each may differ by a whole step, 2^-7
    # of the value, where the products' or the chunks' sums differ in order.
    off = float((got.float() - want.float()).norm() / want.float().norm())
    print("relative difference %.2e" % off)
    assert off <= 5 * 2.0 ** -7
