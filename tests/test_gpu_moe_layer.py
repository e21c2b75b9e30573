"""The example layer (examples/moe_layer.py): its serving step against the layer in plain torch,
its training step against automatic differentiation in 64 bits, and the serving step in a graph.

Bounds, in the 2-norm.  Served: the hidden rows and the experts' rows are rounded to bf16 (2^-9 of
each value, so at most 2^-9 of the norm) and so is the output: 3 * 2^-9.  Trained: rows, expert
rows and the output rounded once each, 3 * 2^-9 again; d_x the same; the losses are fp32 sums.
d_logits takes the rounding of the expert rows through <y, d_out>, 2^-9 of values that may cancel
against each other: 2^-6.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.moe.build()
    return module


@pytest.mark.parametrize("shape", [dict(), dict(T=1, H=1040, F=144, E=12, k=2, P=4, block_rows=2),
                                   dict(T=300, H=256, F=128, E=8, k=2, P=2, block_rows=300)])
def test_served(example, shape):
    assert example.check_served(**shape) <= 3 * 2.0 ** -9


@pytest.mark.parametrize("shape", [dict(), dict(S=1, T=513, H=72, E=20, k=5, P=5)])
def test_trained(example, shape):
    errors = example.check_trained(**shape)
    assert errors["out"] <= 3 * 2.0 ** -9 and errors["d_x"] <= 3 * 2.0 ** -9
    assert errors["losses"] <= 1e-5 and errors["d_logits"] <= 2.0 ** -6


def test_served_in_a_graph(example):
    """A captured step follows new logits and rows."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, F, E, k, P = 32, 256, 128, 16, 3, 4
    w1 = torch.randn(E, 2 * F, H, generator=g, device="cuda") / 16
    w2 = torch.randn(E, H, F, generator=g, device="cuda") / 11
    layer = example.ServedLayer(T, H, F, E, k, P, w1, w2, 32)
    logits = torch.randn(1, T, E, generator=g, device="cuda")
    x = torch.randn(1, T, H, generator=g, device="cuda").bfloat16()
    layer.step(logits, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(logits, x)
    for _ in range(3):
        logits.copy_(torch.randn(1, T, E, generator=g, device="cuda"))
        x.copy_(torch.randn(1, T, H, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = layer.path.out.clone()
        assert torch.equal(got, layer.step(logits, x))
