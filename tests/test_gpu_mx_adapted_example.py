"""The adapted MLP example: LayerNorm, adapted products, SwiGLU and the adapters' gradients together, in a
training step, for a batch of requests and for one."""
import importlib.util
import os

import pytest
import torch

import mx_block_scaled_x128_amd as mx

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_mlp.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("adapted_mlp", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def inputs(tokens, hidden):
    gen = torch.Generator(device="cuda").manual_seed(5)
    return (torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16(),
            torch.randn(tokens, hidden, generator=gen, device="cuda").mul_(1e-3).bfloat16())


@pytest.mark.parametrize("tokens,hidden,inner,adapters,rank", [(1, 128, 256, 1, 8), (100, 256, 384, 2, 24),
                                                              (517, 512, 1408, 3, 16)])
def test_gradients_point_where_fp32_ones_do(example, tokens, hidden, inner, adapters, rank):
    """E4M3 operands are off by at most 2^-4 of themselves (0.03 in the mean), E5M2 gradients by 2^-3 (0.06), the
    transposed weights' E2M1 codes, in other blocks than the forward ones', by about 0.11.  So the output stays
    within an angle of 0.1, gradients behind two data-gradient products within 0.4: cosines above 0.99 and 0.92."""
    mlp = example.AdaptedMLP(hidden, inner, adapters, rank)
    x, dout = inputs(tokens, hidden)
    ids = example.sequences(tokens, adapters) if tokens > 1 else torch.zeros(1, dtype=torch.int32, device="cuda")
    out, kept = mlp.forward(x, ids)
    dx, grads = mlp.backward(kept, dout)
    ref, ref_dx, ref_grads = example.reference(mlp, x, ids, dout)
    assert example.cosine(out, ref) > 0.99 and example.cosine(dx, ref_dx) > 0.98
    for name in grads:
        assert grads[name].shape == ref_grads[name].shape
        assert example.cosine(grads[name], ref_grads[name]) > 0.92, name


def test_requests_served_together_and_alone(example):
    """A batch over all adapters and none: each row is what its request gets alone, within bf16's rounding and the
    cast of an activation that the order of a sum moved across a tie."""
    mlp = example.AdaptedMLP(256, 384, 3, 16)
    x, _ = inputs(9, 256)
    ids = torch.tensor([2, -1, 0, 1, 1, 2, 0, -1, 2], dtype=torch.int32, device="cuda")
    together = mlp.forward(x, ids, keep=False)
    assert together[1] is None
    for i in range(9):
        alone = mlp.forward(x[i:i + 1], ids[i:i + 1], keep=False)[0]
        assert example.cosine(alone, together[0][i:i + 1]) > 0.9999
    plain = mlp.forward(x[1:2], torch.zeros(1, dtype=torch.int32, device="cuda"), keep=False)[0]
    assert example.cosine(plain, together[0][1:2]) < 0.9999  # an adapter does something


def test_a_captured_step(example):
    """Forward and backward captured once, replayed on other requests' ids and inputs with eager work between."""
    mlp = example.AdaptedMLP(128, 256, 2, 8)
    x, dout = inputs(200, 128)
    ids = example.sequences(200, 2)

    def step():
        out, kept = mlp.forward(x, ids)
        dx, grads = mlp.backward(kept, dout)
        return [out, dx] + [grads[k] for k in sorted(grads)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        ids.copy_(torch.roll(ids, 37))
        x.mul_(1.1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([t.clone() for t in held], step()):
            assert torch.equal(a, b)


def test_an_update_changes_what_is_served(example):
    mlp = example.AdaptedMLP(128, 256, 2, 8)
    x, dout = inputs(64, 128)
    ids = example.sequences(64, 2)
    out, kept = mlp.forward(x, ids)
    grads = mlp.backward(kept, dout)[1]
    assert all(torch.isfinite(g).all() and g.abs().max() > 0 for g in grads.values())
    mlp.update(grads, 1.0)
    assert not torch.equal(mlp.forward(x, ids, keep=False)[0], out)
    none = torch.full_like(ids, -1)
    other = example.AdaptedMLP(128, 256, 2, 8)
    other.w, other.b = mlp.w, mlp.b
    assert torch.equal(mlp.forward(x, none, keep=False)[0], other.forward(x, none, keep=False)[0])  # the weights are frozen
    assert mx.dequantize_mx(*mlp.up.q, mx.E2M1).shape == (512, 128)
