"""The 4-bit feed-forward example: its pieces run together as a user would run
them, forward, backward, training and token by token."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location(
        "feed_forward_4bit", os.path.join(ROOT, "examples", "feed_forward_4bit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("size", [(256, 512, 300), (200, 328, 77)])
def test_forward_and_gradients_follow_fp32(ex, kind, size):
    """4-bit rounding of normal data leaves a relative error of about 0.11
    (MXFP4 0.13) per operand.  y is a product of a product: four operands and
    the activation, at most 0.3 in all, a cosine of 0.95; each gradient passes
    through at most six roundings, 0.35, 0.93."""
    hidden, ffn, tokens = size
    torch.manual_seed(3)
    layer = ex.FeedForward4Bit(hidden, ffn, kind)
    x = torch.randn((tokens, hidden), device="cuda").bfloat16()
    dy = (torch.randn((tokens, hidden), device="cuda") * 1e-3).bfloat16()
    y, saved = layer.forward(x)
    got = (y, *layer.backward(dy, saved))
    for a, b, least in zip(got, ex.reference(layer, x, dy), (0.95, 0.93, 0.93, 0.93)):
        assert a.shape == b.shape and ex.cosine(a, b) > least


@pytest.mark.parametrize("kind", [0, 1])
def test_training_reduces_the_loss(ex, kind):
    losses = ex.train(ex.FeedForward4Bit(256, 512, kind), steps=40, tokens=512)
    assert losses[-1] < 0.7 * losses[0]


@pytest.mark.parametrize("kind", [0, 1])
def test_tokens_one_by_one_are_the_batch(ex, kind):
    """The same operands and scales (calibrated, or per block): only the order
    of the sums and one rounding to bf16 between the products differ."""
    torch.manual_seed(4)
    layer = ex.FeedForward4Bit(256, 640, kind)
    x = torch.randn((200, 256), device="cuda").bfloat16()
    serve = layer.serving(x)
    whole = serve(x).float()
    one = torch.cat([serve(x[i:i + 1]) for i in range(0, 200, 20)]).float()
    want = whole[::20]
    assert (one - want).norm() <= 0.05 * want.norm()
