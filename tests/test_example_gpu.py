"""The layer example, end to end: gradients through both operators train it, and
decoding token by token from the pool of states gives what whole sequences give.

Bars: logits are sums over layers of bf16 values, each rounded at a handful of places in
either path (2^-9 root-mean-square and less each): 2e-2 of the logits' norm; rows in
e4m3 (2^-4 at most, 2.6e-2 root-mean-square) through two layers: 0.15."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_delta_layer.py")
    spec = importlib.util.spec_from_file_location("gated_delta_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trains_and_decodes(example):
    torch.manual_seed(0)
    model = example.Model().cuda()
    assert example.decode_error(model) <= 2e-2
    losses = example.train(model, 200)
    assert all(x == x for x in losses)
    assert max(losses[-5:]) < 4.16 - 0.5  # half a nat below guessing one of 64
    assert example.decode_error(model) <= 2e-2
    assert example.decode_error(model, e4m3=True) <= 0.15
