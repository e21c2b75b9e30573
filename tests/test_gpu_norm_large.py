"""moe_rms_norm and moe_rms_norm_backward on rows whose sum of squares leaves fp32 while their mean square
does not, on both sides of that bound.  Tolerances as in test_gpu_norm.py: a power of two before the
squares is exact, and none of them that counts falls below fp32's normal range."""
import pytest
import torch

import combine_moe_route_06_gb300 as m
from gpu_util import DEV
from test_gpu_norm import BF, F32, HALF, definition, randn

pytestmark = pytest.mark.gpu

SIZES = [(3, 8), (5, 264), (9, 512), (4, 1040), (3, 2048), (7, 4096), (300, 5120), (2, 8192), (3, 8200),
         (2, 16384), (2, 32768)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()


def large_rows(rows, H, kind):
    """Rows of ordinary size, of RMS 2^58, 2^60 and 2^62 in turn, and one of 1.8e19 throughout, whose mean
    square is 0.95 of fp32's largest value (a bf16 row's x is the whole of them, an fp32 one's residual)."""
    h = randn(1, rows, H, dtype=F32)
    h *= torch.tensor([2.0 ** 58, 2.0 ** 60, 1.0, 2.0 ** 62], device=DEV).repeat(rows)[:rows, None]
    h[-1] = 1.8e19
    return h.to(kind)


@pytest.mark.parametrize("rows,H", SIZES)
@pytest.mark.parametrize("kind", [None, BF, F32])
def test_norm(rows, H, kind):
    h, weight = large_rows(rows, H, kind or BF), 1 + randn(2, H, dtype=kind or F32, scale=0.3)
    x, residual = (h, None) if kind is None else (randn(3, rows, H), h)
    y = torch.empty(rows, H, dtype=BF, device=DEV)
    record = torch.empty(rows, H + H // 32, dtype=torch.uint8, device=DEV) if H % 32 == 0 else None
    m.moe_rms_norm(x, weight, y=y, record=record, residual=residual, eps=1e-5)
    _, want = definition(x, residual, weight, 1e-5)
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 1e-38).all())
    if record is not None:
        again = torch.empty_like(record)
        m.moe_rms_norm(x, weight, record=again, residual=residual, eps=1e-5)
        assert torch.equal(record, again) and bool((record[:, :H] != 0).any(1).all())


@pytest.mark.parametrize("rows,H", SIZES)
@pytest.mark.parametrize("kind,wkind,add", [(BF, F32, False), (BF, BF, True), (F32, BF, True)])
def test_norm_backward(rows, H, kind, wkind, add):
    h, weight = large_rows(rows, H, kind), 1 + randn(4, H, dtype=wkind, scale=0.3)
    d_y = randn(5, rows, H, scale=0.1)
    d_res = randn(6, rows, H, dtype=kind, scale=2.0 ** -64) if add else None
    d_h, d_w = torch.empty_like(h), torch.empty(H, dtype=F32, device=DEV)
    ws = torch.empty(m.moe_rms_norm_backward_workspace_bytes(rows, H), dtype=torch.uint8, device=DEV)
    m.moe_rms_norm_backward(d_y, h, weight, d_h, ws, d_weight=d_w, d_residual=d_res, eps=1e-5)
    h64, q = h.double(), d_y.double() * weight.double()
    inv = 1 / (h64.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    want = inv * (q - h64 * inv * inv * (q * h64).mean(-1, keepdim=True))
    size = inv * (q.abs() + h64.abs() * inv * inv * (q * h64).abs().mean(-1, keepdim=True))
    if add:
        want, size = want + d_res.double(), size + d_res.double().abs()
    assert bool(((d_h.double() - want).abs() <= 2.0 ** -17 * size + HALF[kind] * want.abs() + 1e-38).all())
    terms = d_y.double() * h64 * inv
    bound = (rows * 2.0 ** -24 + 2.0 ** -17) * terms.abs().sum(0) + 1e-38
    assert bool(((d_w.double() - terms.sum(0)).abs() <= bound).all())


@pytest.mark.parametrize("H", [8, 512, 5120, 32768])
@pytest.mark.parametrize("kind", [BF, F32])
def test_rows_past_the_bound(H, kind):
    """A mean square of 1e40 is past fp32: such a row is 0, and its gradient is what comes from elsewhere;
    the rows beside it are as without it."""
    residual, x = randn(7, 5, H, dtype=kind), torch.zeros(5, H, dtype=BF, device=DEV)
    weight, d_y, d_res = randn(8, H, dtype=F32), randn(9, 5, H), randn(10, 5, H, dtype=kind)
    ws = torch.empty(m.moe_rms_norm_backward_workspace_bytes(5, H), dtype=torch.uint8, device=DEV)
    clean = []
    for value in (0.0, 1e20):
        residual[1], residual[4] = value, -value
        y, d_h, d_w = torch.empty_like(x), torch.empty_like(residual), torch.empty(H, dtype=F32, device=DEV)
        m.moe_rms_norm(x, weight, y=y, residual=residual)
        m.moe_rms_norm_backward(d_y, residual, weight, d_h, ws, d_weight=d_w, d_residual=d_res)
        clean.append((y, d_h, d_w))
    (y0, d_h0, d_w0), (y, d_h, d_w) = clean
    for r in (1, 4):
        assert bool((y[r] == 0).all()) and torch.equal(d_h[r], d_res[r])
    for r in (0, 2, 3):
        assert torch.equal(y[r], y0[r]) and torch.equal(d_h[r], d_h0[r])
    assert torch.equal(d_w, d_w0)
