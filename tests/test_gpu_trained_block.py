"""The example block (examples/moe_layer.py): norm, router, experts and combine that train, against
automatic differentiation in 64 bits; and records that a norm has written, dispatched by a path.

Bounds, in the 2-norm, u = 2^-8 for each rounding to bf16.  out: the normed rows, the router's logits (of
size 1: u shifts a weight by at most u of itself, twice for the softmax's sum), hidden rows, expert rows,
out: 6 u.  h: u.  The gradients add those of d_y, d_pre, d_recv, the sum over a token's rows and d_x, and of
pre through the activation's second derivative: 12 u.  d_router comes from <y, d_out>, whose terms may
cancel, as in the tests of the trained layer: 2^-4.
"""
import importlib.util
import os

import pytest
import torch

import combine_moe_route_06_gb300 as m
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    m.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("shape", [dict(), dict(T=1, H=64, F=40, E=4, k=2, P=2),
                                   dict(T=777, H=256, F=136, E=24, k=4, P=8)])
def test_block(example, shape):
    u = 2.0 ** -8
    errors = example.check_block(**shape)
    assert errors["out"] <= 6 * u and errors["h"] <= u, errors
    assert max(errors[n] for n in ("d_x", "d_norm", "d_gate_up", "d_down")) <= 12 * u, errors
    assert errors["d_router"] <= 2.0 ** -4, errors


def test_block_in_a_graph(example):
    """A step, both ways, captured once and replayed on new rows."""
    T, H, F, E, k, P = 96, 256, 136, 8, 2, 4
    g = torch.Generator(device=DEV).manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    weights = [1 + 0.2 * randn(H)] + [(randn(*s) / s[-1] ** 0.5).bfloat16()
                                      for s in ((E, H), (E, 2 * F, H), (E, H, F))]
    block = example.TrainedBlock(T, H, F, E, k, P, *weights)
    x, residual, d_out, d_h = (randn(1, T, H).bfloat16() for _ in range(4))

    def step():
        return (*block.forward(x, residual), *block.backward(d_out, d_h))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        for t in (x, residual, d_out, d_h):
            t.copy_(randn(1, T, H))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("T,H,recv_part", [(1, 512, -1), (70, 5120, -1), (300, 1024, 2)])
def test_path_dispatches_records(T, H, recv_part):
    """dispatch_records of a norm's records receives what dispatch_fused makes of its rows, and the
    expert and the combine go on from there."""
    E, k, P = 16, 4, 4
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(1, T, H, generator=g, device=DEV).bfloat16()
    logits, weight = torch.randn(1, T, E, generator=g, device=DEV), torch.ones(H, device=DEV)
    scale = 0.5 + torch.rand(E, generator=g, device=DEV)
    y, record = torch.empty_like(x), torch.empty(1, T, m.mxfp8_record_bytes(H), dtype=torch.uint8, device=DEV)
    m.moe_rms_norm(x, weight, y=y, record=record)
    one, two = (m.MoePath(1, T, H, E, k, P, recv_part=recv_part, quant="mxfp8") for _ in range(2))
    one.dispatch_fused(logits, y)
    two.dispatch_records(logits, record)
    used = int(one.expert_offsets[-1])
    assert torch.equal(one.expert_offsets, two.expert_offsets) and torch.equal(one.recv[:used], two.recv[:used])
    for p in (one, two):
        p.expert(scale)
        p.combine()
    assert torch.equal(one.out, two.out) and int(two.dev_status.item()) == 0


def test_path_refuses_records():
    path = m.MoePath(1, 4, 512, 4, 2, 2)
    record = torch.empty(1, 4, 528, dtype=torch.uint8, device=DEV)
    logits = torch.zeros(1, 4, 4, device=DEV)
    with pytest.raises(ValueError, match="quant='mxfp8'"):
        path.dispatch_records(logits, record)
    path = m.MoePath(1, 4, 512, 4, 2, 2, quant="mxfp8")
    with pytest.raises(ValueError, match="record must be"):
        path.dispatch_records(logits, record[:, :3])
    with pytest.raises(TypeError, match="dtype"):
        path.dispatch_records(logits, record.view(torch.int8))
