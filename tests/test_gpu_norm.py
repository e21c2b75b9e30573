"""moe_rms_norm and moe_rms_norm_backward against their definitions in 64 bits.

Tolerance (u = 2^-24).  A thread adds at most 40 squares one after the other and the team's sums go
through two trees of five steps, so the mean square is off by at most 52 u of itself, and so is any sum
over a row against the sum of its terms' sizes; the root halves that, and the root, the division and
the two products round once each: y is within 32 u of itself (2^-19), and 2^-8 for its rounding to
bf16.  d_h = d_residual + inv (q - h inv along) takes the same for each of its terms: 2^-17 of their
sizes.  A column of d_weight is a sum of `rows` fp32 terms, each within 2^-17: (rows u + 2^-17) of the
sum of their sizes.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
from gpu_util import DEV

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()


def randn(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def guarded(*shape, dtype):
    """A tensor with a guard behind it, and a function that says whether the guard is untouched."""
    n = int(np.prod(shape))
    whole = torch.full((n + 4096,), 99, dtype=dtype, device=DEV)
    return whole[:n].view(shape), lambda: bool((whole[n:] == 99).all())


def definition(x, residual, weight, eps):
    h = x.double() + (0 if residual is None else residual.double())
    return h, h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def records_of(y):
    """MXFP8 records of bf16 rows: per 32 values an exponent, values in E4M3 (ties to even)."""
    blocks = y.float().cpu().view(y.shape[0], -1, 32)
    top = blocks.abs().amax(-1)
    power = torch.where(top > 0, torch.frexp(top).exponent - 9, -127).clamp(min=-127)
    codes = torch.ldexp(blocks.double(), -power.unsqueeze(-1).double()).clamp(-448, 448)
    codes = codes.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
    return torch.cat((codes, (power + 127).to(torch.uint8)), 1)


SIZES = [(1, 8), (1, 5120), (3, 32), (7, 264), (333, 1040), (9, 1024), (5, 1032), (2, 2048), (4, 2080),
         (65, 4096), (3, 4104), (130, 5120), (2, 5128), (5, 8192), (3, 8200), (2, 16384), (2, 32768),
         (2500, 72), (1300, 2048), (3001, 512)]


@pytest.mark.parametrize("rows,H", SIZES)
@pytest.mark.parametrize("kind,wkind", [(None, BF), (BF, BF), (F32, F32)])
def test_norm(rows, H, kind, wkind):
    x, weight = randn(1, rows, H), 1 + randn(2, H, dtype=wkind, scale=0.3)
    residual = None if kind is None else randn(3, rows, H, dtype=kind, scale=3)
    y, whole = guarded(rows, H, dtype=BF)
    record, whole_r = (guarded(rows, H + H // 32, dtype=torch.uint8) if H % 32 == 0 else (None, lambda: True))
    total, whole_t = (None, lambda: True) if kind is None else guarded(rows, H, dtype=kind)
    m.moe_rms_norm(x, weight, y=y, record=record, residual=residual, residual_out=total, eps=1e-5)
    h, want = definition(x, residual, weight, 1e-5)
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 1e-38).all())
    if kind is not None:
        assert bool(((total.double() - h).abs() <= (HALF[kind] + 2.0 ** -24) * h.abs() + 1e-38).all())
    if record is not None:
        assert torch.equal(record.cpu(), records_of(y))
    assert whole() and whole_r() and whole_t()


def test_record_alone_and_in_place():
    """Only the record; the residual updated in its own place; three dimensions."""
    x, residual = randn(4, 2, 33, 512), randn(5, 2, 33, 512, dtype=F32)
    weight = randn(6, 512)
    y, both = torch.empty_like(x), torch.empty(2, 33, 528, dtype=torch.uint8, device=DEV)
    total = torch.empty_like(residual)
    m.moe_rms_norm(x, weight, y=y, record=both, residual=residual, residual_out=total)
    alone = torch.empty_like(both)
    m.moe_rms_norm(x, weight, record=alone, residual=residual, residual_out=residual)
    assert torch.equal(alone, both) and torch.equal(residual, total)


@pytest.mark.parametrize("T,H", [(1, 512), (70, 5120)])
def test_records_are_those_of_the_quantized_pack(T, H):
    """Byte for byte, zero rows and large and small rows among them; and they dispatch as rows."""
    E, P, k = 16, 4, 3
    x, weight = randn(7, 1, T, H), randn(8, H)
    x[0, T // 2] = 0
    weight[: H // 4] *= 2.0 ** 60
    weight[H // 4: H // 2] *= 2.0 ** -100
    y, record = torch.empty_like(x), torch.empty(1, T, H + H // 32, dtype=torch.uint8, device=DEV)
    m.moe_rms_norm(x, weight, y=y, record=record)
    logits = randn(9, 1, T, E, dtype=F32)
    one = m.MoePath(1, T, H, E, k, P, quant="mxfp8")
    one.dispatch_fused(logits, y)
    two = m.MoePath(1, T, (H + H // 32) // 2, E, k, P)
    two.dispatch_fused(logits, record.view(BF))
    used = int(one.expert_offsets[-1])
    assert used == T * k and torch.equal(one.recv[:used], two.recv[:used].view(torch.uint8))
    one.expert(None)
    other = torch.empty_like(one.y)
    m.moe_expert_scale_mxfp8(two.recv.view(torch.uint8), two.expert_offsets, one.unit_scale, other)
    assert torch.equal(one.y[:used].view(torch.int16), other[:used].view(torch.int16))


def test_rows_that_are_not_finite_or_zero():
    """A NaN or infinity stays in its row; a row of zeros is zero."""
    x, weight = randn(10, 6, 1280), randn(11, 1280)
    x[1, 7], x[3, 1279], x[5] = float("nan"), float("inf"), 0
    y = torch.empty_like(x)
    m.moe_rms_norm(x, weight, y=y)
    clean = x.clone()
    clean[1], clean[3] = 0, 0
    want = torch.empty_like(x)
    m.moe_rms_norm(clean, weight, y=want)
    for r in (0, 2, 4, 5):
        assert torch.equal(y[r], want[r])
    assert bool((y[5] == 0).all()) and bool(y[1].isnan().all()) and bool(y[3, 1279].isnan())


@pytest.mark.parametrize("rows,H", SIZES)
@pytest.mark.parametrize("kind,wkind,add", [(BF, F32, False), (BF, BF, True), (F32, BF, True)])
def test_norm_backward(rows, H, kind, wkind, add):
    d_y, weight = randn(12, rows, H, scale=0.1), 1 + randn(13, H, dtype=wkind, scale=0.3)
    h = randn(14, rows, H, dtype=kind, scale=3)
    d_res = randn(15, rows, H, dtype=kind, scale=0.1) if add else None
    d_h, whole = guarded(rows, H, dtype=kind)
    d_x = torch.empty(rows, H, dtype=BF, device=DEV)
    d_w, whole_w = guarded(H, dtype=F32)
    need = m.moe_rms_norm_backward_workspace_bytes(rows, H)
    ws, whole_ws = guarded(need, dtype=torch.uint8)
    m.moe_rms_norm_backward(d_y, h, weight, d_h, ws, d_weight=d_w, d_residual=d_res, d_x=d_x, eps=1e-5)
    h64, q = h.double(), d_y.double() * weight.double()
    inv = 1 / (h64.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    want = inv * (q - h64 * inv * inv * (q * h64).mean(-1, keepdim=True))
    size = inv * (q.abs() + h64.abs() * inv * inv * (q * h64).abs().mean(-1, keepdim=True))
    if add:
        want, size = want + d_res.double(), size + d_res.double().abs()
    bound = 2.0 ** -17 * size + HALF[kind] * want.abs() + 1e-38
    assert bool(((d_h.double() - want).abs() <= bound).all())
    assert bool(((d_x.double() - want).abs() <= 2.0 ** -17 * size + 2.0 ** -8 * want.abs() + 1e-38).all())
    terms = d_y.double() * h64 * inv
    bound = (rows * 2.0 ** -24 + 2.0 ** -17) * terms.abs().sum(0) + 1e-38
    assert bool(((d_w.double() - terms.sum(0)).abs() <= bound).all())
    assert whole() and whole_w() and whole_ws()
    again = torch.empty_like(d_h)
    m.moe_rms_norm_backward(d_y, h, weight, again, d_residual=d_res, eps=1e-5)   # rows alone
    assert torch.equal(again, d_h)


def test_gradient_is_that_of_differences():
    """<d_h, v> against (f(h + t v) - f(h - t v)) / 2t in 64 bits, f = <d_y, norm(h)>; and the
    residual's gradient in its own place."""
    rows, H = 5, 264
    d_y, weight, h = randn(16, rows, H), randn(17, H, dtype=F32), randn(18, rows, H, dtype=F32)
    d_h, ws = torch.zeros_like(h), torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    d_w = torch.empty_like(weight)
    m.moe_rms_norm_backward(d_y, h, weight, d_h, ws, d_weight=d_w, d_residual=d_h, eps=1e-3)

    def f(h64, w64):
        return float((d_y.double() * h64 / (h64.square().mean(-1, keepdim=True) + 1e-3).sqrt() * w64).sum())

    t = 1e-4
    for seed in range(3):
        v, vw = randn(20 + seed, rows, H, dtype=F32).double(), randn(30 + seed, H, dtype=F32).double()
        h64, w64 = h.double(), weight.double()
        by_h = (f(h64 + t * v, w64) - f(h64 - t * v, w64)) / (2 * t)
        by_w = (f(h64, w64 + t * vw) - f(h64, w64 - t * vw)) / (2 * t)
        # f's third derivative along v times t^2 / 6, and 64-bit noise over 2t: both below 1e-4
        assert abs(by_h - float((d_h.double() * v).sum())) <= 1e-3 * (1 + abs(by_h))
        assert abs(by_w - float((d_w.double() * vw).sum())) <= 1e-3 * (1 + abs(by_w))


def test_no_rows():
    empty, weight = torch.empty(0, 64, dtype=BF, device=DEV), randn(40, 64)
    m.moe_rms_norm(empty, weight, y=empty, record=torch.empty(0, 66, dtype=torch.uint8, device=DEV))
    d_w = torch.full((64,), 7.0, device=DEV)
    ws = torch.empty(m.moe_rms_norm_backward_workspace_bytes(0, 64), dtype=torch.uint8, device=DEV)
    m.moe_rms_norm_backward(empty, empty, weight, empty, ws, d_weight=d_w)
    assert bool((d_w == 0).all())


def test_in_a_graph_and_on_another_stream():
    """A captured chain, norm then gradient, follows new rows, on a stream of its own."""
    rows, H = 77, 1536
    x, weight, d_y = randn(41, rows, H), randn(42, H), randn(43, rows, H)
    y, d_h = torch.empty_like(x), torch.empty_like(x)
    d_w = torch.empty(H, dtype=F32, device=DEV)
    ws = torch.empty(m.moe_rms_norm_backward_workspace_bytes(rows, H), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        m.moe_rms_norm(x, weight, y=y, stream=stream)
        m.moe_rms_norm_backward(d_y, x, weight, d_h, ws, d_weight=d_w, stream=stream)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(randn(50 + seed, rows, H))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        got = [t.clone() for t in (y, d_h, d_w)]
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, d_h, d_w)))
