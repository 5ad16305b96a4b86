"""The gated MLP example: the MX operators together in a training step and for one token."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_mlp.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_mlp", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 128, 256), (100, 256, 384), (517, 512, 1408)])
def test_gradients_point_where_fp32_ones_do(example, tokens, hidden, inner):
    """E2M1 weights carry a relative error near 0.11 and E4M3 / E5M2 operands near 0.03 / 0.05, so the
    products' results stay within an angle of about 0.2 and the gradients behind three of them within
    0.4: cosines above 0.98 and 0.92."""
    mlp = example.GatedMLP(hidden, inner)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    dout = torch.randn(tokens, hidden, generator=gen, device="cuda").mul_(1e-3).bfloat16()
    out, kept = mlp.forward(x)
    dx, grads = mlp.backward(kept, dout)
    ref, ref_dx, ref_grads = example.reference(mlp, x, dout)
    assert example.cosine(out, ref) > 0.98 and example.cosine(dx, ref_dx) > 0.98
    for name in grads:
        assert grads[name].shape == ref_grads[name].shape
        assert example.cosine(grads[name], ref_grads[name]) > 0.92, name
    alone = mlp.forward(x[:1], keep=False)
    assert alone[1] is None and example.cosine(alone[0], out[:1]) > 0.9999


def test_training_lowers_the_loss(example):
    losses, _ = example.train(500, 256, 384, 20)
    assert losses[-1] < 0.7 * losses[0] and min(losses) == min(losses[10:])
