"""The norm and the bf16 expert calls as programs make them: first of all calls inside a capture, on a
current stream of the program's own, traced, and with rows that move between calls."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
from gpu_util import DEV, i32_dev

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()


def randn(seed, *shape, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def step(x, weight, w, ends, ws, outs, stream=None):
    y, h, d_a, d_w, d_x, d_weight = outs
    m.moe_rms_norm(x, weight, y=y, stream=stream)
    m.moe_expert_product(y, w, h, ws, expert_offsets=ends, stream=stream)
    m.moe_expert_product_backward(h, y, w, ws, d_a=d_a, d_w=d_w, expert_offsets=ends, stream=stream)
    m.moe_rms_norm_backward(d_a, x, weight, d_x, ws, d_weight=d_weight, stream=stream)


def inputs(rows=90, H=136, E=3):
    x, weight, w = randn(1, rows, H), randn(2, H), randn(3, E, H, H)
    ends = i32_dev(np.array([0, rows // 2, rows // 2, rows]))
    ws = torch.empty(max(m.moe_expert_product_workspace_bytes(rows, E, H, H),
                         m.moe_rms_norm_backward_workspace_bytes(rows, H)), dtype=torch.uint8, device=DEV)
    outs = (torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(x),
            torch.empty(H, device=DEV))
    return x, weight, w, ends, ws, outs


def check(x, weight, w, ends, outs):
    """Each call's results from its own inputs, to the rounding of bf16 and a little more."""
    y, h, d_a, d_w, d_x, d_weight = (t.double() for t in outs)
    x, weight, w = x.double(), weight.double(), w.double()
    inv = 1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    near = lambda a, b: float((a - b).norm()) <= 2.0 ** -7 * float(b.norm())  # noqa: E731
    assert near(y, x * inv * weight)
    bounds = ends.tolist()
    for e in range(w.shape[0]):
        at = slice(bounds[e], bounds[e + 1])
        assert near(h[at], y[at] @ w[e].t()) and near(d_a[at], h[at] @ w[e]) and near(d_w[e], h[at].t() @ y[at])
    q = d_a * weight
    assert near(d_x, inv * (q - x * inv * inv * (q * x).mean(-1, keepdim=True)))
    assert near(d_weight, (d_a * x * inv).sum(0))


def first_calls_in_a_capture():
    args = inputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*args)
    for seed in range(2):
        args[0].copy_(randn(10 + seed, *args[0].shape))
        graph.replay()
        torch.cuda.synchronize()
        check(*args[:4], args[5])


def test_first_calls_in_a_capture():
    """A process whose first calls of the library are captured."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = f"import sys; sys.path[:0] = [{here!r}, {os.path.dirname(here)!r}]; " \
           "import test_gpu_norm_product_calls as t; t.first_calls_in_a_capture(); print('same')"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_current_stream():
    """Without a stream argument the calls follow the current stream."""
    args = inputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(*args)
    side.synchronize()
    check(*args[:4], args[5])
    got = [t.clone() for t in args[5]]
    torch.cuda.synchronize()
    step(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, args[5]))


def test_offsets_that_change_between_replays():
    """A captured product follows new offsets: the work is found out on the device."""
    rows, H, E = 700, 264, 5
    x, w = randn(4, rows, H), randn(5, E, H, H)
    ends = i32_dev(np.zeros(E + 1))
    ws = torch.empty(m.moe_expert_product_workspace_bytes(rows, E, H, H), dtype=torch.uint8, device=DEV)
    y, d_a, d_w = torch.empty_like(x), torch.empty_like(x), torch.empty(w.shape, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_expert_product(x, w, y, ws, expert_offsets=ends)
        m.moe_expert_product_backward(x, x, w, ws, d_a=d_a, d_w=d_w, expert_offsets=ends)
    for bounds in ([0, 700, 700, 700, 700, 700], [0, 1, 300, 300, 650, 700], [0, 0, 0, 0, 0, 0], [100, 200, 300, 400, 500, 600]):
        ends.copy_(i32_dev(np.array(bounds)))
        y.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        for e in range(E):
            at = slice(bounds[e], bounds[e + 1])
            want, grad = x[at].double() @ w[e].double().t(), x[at].double().t() @ x[at].double()
            assert float((y[at].double() - want).norm()) <= 2.0 ** -7 * float(want.norm())
            assert float((d_w[e].double() - grad).norm()) <= 1e-5 * float(grad.norm())
        assert bool((y[:bounds[0]] == -7).all()) and bool((y[bounds[-1]:] == -7).all())


def test_traced():
    """The calls' launches are among the traced kernels."""
    args = inputs(rows=1000)
    m.trace_enable(None, 64)
    try:
        step(*args)
        names = [name for name, ms in m.trace_records() if ms > 0]
    finally:
        m.trace_disable()
    for name in ("k_rms_norm", "k_expert_product", "k_expert_gradients", "k_rms_norm_backward", "k_sum_parts"):
        assert name in names, names


def test_status_word_is_optional_and_only_gains_bits():
    args = inputs()
    x, weight, w, ends, ws, outs = args
    st = torch.full((1,), 1 << 30, dtype=torch.int32, device=DEV)
    m.moe_expert_product(x, w, outs[0], ws, expert_offsets=ends, dev_status=st)
    assert int(st.item()) == 1 << 30
    m.moe_expert_product(x, w, outs[0], ws, expert_offsets=i32_dev(np.array([0, 5, 500, 500])), dev_status=st)
    assert int(st.item()) == (1 << 30) | (1 << m.MOE_ERR_INVALID_ARG)
    m.moe_expert_product(x, w, outs[0], ws, expert_offsets=i32_dev(np.array([0, 5, 500, 500])))
    torch.cuda.synchronize()
