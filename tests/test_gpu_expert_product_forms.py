"""The experts' bf16 products at sizes where their tiles are taken in turn, cut, or both, and the
weights' gradient over long sums.  Tolerances as in test_gpu_expert_product.py."""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
from gpu_util import DEV
from test_gpu_expert_product import (BF, F32, Rows, backward, check_backward, check_forward, forward, randn,
                                     workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()


FORWARD = [  # N, K, counts, gated
    (5120, 4096, [700, 800, 500], False),       # a turn of whole tiles, then tiles cut between pairs
    (2560, 4160, [700, 800, 500], True),
    (2048, 640, [700, 0, 3000], False),         # several turns of whole tiles
    (768, 1024, [2, 5000, 0, 300, 31], True),
    (264, 7168, [600], True),                   # few tiles, each cut into many parts
    (8, 20000, [40, 3], False), (136, 3200, [1] * 40, True)]


@pytest.mark.parametrize("N,K,counts,gated", FORWARD)
def test_forward(N, K, counts, gated):
    rows = Rows(counts, first=3)
    a, w = rows.fill(randn(1, rows.total, K)), randn(2, len(counts), 2 * N if gated else N, K, scale=K ** -0.5)
    y, pre = forward(rows, a, w, gated, gated)
    check_forward(rows, a, w, gated, y, pre)


BACKWARD = [  # N, K, counts, gate
    (4096, 5120, [700, 800, 500], False), (2688, 2816, [700, 800, 500, 33], True),
    (2560, 2304, [5000, 5100], False),          # weights: a turn of whole tiles, then cut ones
    (512, 768, [6000, 3, 0, 2, 1, 64], True),   # one expert has nearly all steps: its tiles are cut
    (8, 16, [20001], False), (72, 136, [64, 128, 4000, 1], True), (3200, 8, [300, 20], False)]


@pytest.mark.parametrize("N,K,counts,gate", BACKWARD)
@pytest.mark.parametrize("d_w_type", [F32, BF])
def test_backward(N, K, counts, gate, d_w_type):
    rows = Rows(counts, first=3)
    a, d_y = rows.fill(randn(3, rows.total, K)), rows.fill(randn(4, rows.total, N, scale=0.1))
    w, pre = randn(5, len(counts), N, K, scale=K ** -0.5), rows.fill(randn(6, rows.total, 2 * K)) if gate else None
    d_a, d_w = backward(rows, d_y, a, w, pre, d_w_type)
    check_backward(rows, d_y, a, w, pre, d_a, d_w)


@pytest.mark.parametrize("counts", [[16384], [3000, 9, 13001]])
def test_long_sums_keep_fp32(counts):
    """Sums of positive terms, where what an adder cuts off adds up.  It is at most 2^-23 of the sum for
    each 16 rows, over 768 rows at a time (48 * 2^-23), 16 * 2^-24 within 16 rows, and 2^-24 for each of the
    additions of those sums (22): 8.1e-6 in all, whatever the number of rows.  (One sum in the tensor core
    would be off by some 3e-5 over 16,384 rows.)"""
    N, K = 136, 264
    rows = Rows(counts, spare=0)
    a, d_y = randn(7, rows.total, K).abs(), randn(8, rows.total, N).abs()
    w = randn(9, len(counts), N, K)
    _, d_w = backward(rows, d_y, a, w, None, F32, want_a=False)
    for e, at in rows.each():
        want = d_y[at].double().t() @ a[at].double()
        assert float(((d_w[e].double() - want).abs() / want).max()) <= 8.1e-6


def test_the_same_bytes_with_cut_tiles():
    """Parts are added in an order of their own, not in that of their arrival: ten runs give the
    same bytes."""
    N, K, counts = 2560, 4160, [700, 3, 500]
    rows = Rows(counts)
    a, w = rows.fill(randn(10, rows.total, K)), randn(11, 3, 2 * N, K, scale=K ** -0.5)
    d_y, w2 = rows.fill(randn(12, rows.total, N)), randn(13, 3, N, K, scale=K ** -0.5)
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(rows.total, 3, N, K, True))
    y, pre = forward(rows, a, w, True, True, ws=ws)
    d_a, d_w = backward(rows, d_y, a, w2, None, F32, ws=ws)
    for _ in range(9):
        y2, pre2 = forward(rows, a, w, True, True, ws=ws)
        d_a2, d_w2 = backward(rows, d_y, a, w2, None, F32, ws=ws)
        used = rows.used
        assert torch.equal(y[used], y2[used]) and torch.equal(pre[used], pre2[used])
        assert torch.equal(d_a[used], d_a2[used]) and torch.equal(d_w, d_w2)


def test_zeros_have_the_same_sign_every_time():
    """Rows of zeros times negative weights, in tiles that are cut in two: whichever part is done last, the
    sign bits of the results are the same."""
    N, K, rows = 2560, 4160, Rows([700, 500], spare=0)
    a, w = torch.zeros(rows.total, K, dtype=BF, device=DEV), -randn(20, 2, N, K).abs()
    want = None
    for _ in range(10):
        y, _ = forward(rows, a, w, False, False)
        assert bool((y == 0).all())
        bits = y.view(torch.int16)
        assert want is None or torch.equal(bits, want)
        want = bits


def test_calls_on_two_streams_at_once():
    """Two calls with workspaces of their own, enqueued on two streams without a wait between."""
    N, K, counts = 512, 4096, [300, 40]
    rows = Rows(counts)
    a, w = rows.fill(randn(14, rows.total, K)), randn(15, 2, N, K, scale=K ** -0.5)
    want, _ = forward(rows, a, w, False, False)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(want, -7.0) for _ in range(8)]
    ws = [workspace(m.moe_expert_product_workspace_bytes(rows.total, 2, N, K))[0] for _ in range(2)]
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        m.moe_expert_product(a, w, y, ws[i % 2], stream=streams[i % 2], **rows.by)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in outs)


def test_a_call_after_one_that_makes_its_rows():
    """Product after product on one stream: each takes what the one before has just written."""
    H, counts = 512, [200, 0, 57]
    rows = Rows(counts, spare=0)
    x, w = randn(16, rows.total, H), randn(17, 3, H, H, scale=H ** -0.5)
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(rows.total, 3, H, H))
    bufs = [x] + [torch.empty_like(x) for _ in range(6)]
    for i in range(6):
        m.moe_expert_product(bufs[i], w, bufs[i + 1], ws, **rows.by)
    torch.cuda.synchronize()
    for i in range(6):
        check_forward(rows, bufs[i], w, False, bufs[i + 1], None)


def test_offsets_past_32_bits():
    """Rows, weights and gradients whose element offsets pass 2^32: the last rows of a buffer of 600,000
    rows of 7,200 values, and experts behind 2^32 weights."""
    K, N, total = 7200, 64, 600_000
    a = torch.empty(total, K, dtype=BF, device=DEV)
    last = randn(18, 70, K)
    a[-70:] = last
    E, K2 = 300, 7200                     # 300 x 2,048 x 7,200 = 4.4e9 weights
    w = torch.zeros(E, 2048, K2, dtype=BF, device=DEV)
    w[-1] = randn(19, 2048, K2, scale=K2 ** -0.5)
    ends = torch.full((E + 1,), total - 70, dtype=torch.int32, device=DEV)
    ends[-1] = total
    y = torch.zeros(total, 2048, dtype=BF, device=DEV)
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(total, E, 2048, K2))
    m.moe_expert_product(a, w, y, ws, expert_offsets=ends)
    want = last.double() @ w[-1].double().t()
    err = 2 * K * 2.0 ** -24 * (last.double().abs() @ w[-1].double().abs().t()) + 2.0 ** -8 * want.abs()
    assert bool(((y[-70:].double() - want).abs() <= err).all()) and bool((y[:-70] == 0).all())
    del y
    d_y, d_w = torch.empty(total, N, dtype=BF, device=DEV), torch.empty(E, N, K, dtype=F32, device=DEV)
    d_y[-70:] = randn(20, 70, N)
    d_a = a                               # (not read: d_w alone, then d_a alone)
    m.moe_expert_product_backward(d_y, a, w[:, :N].contiguous(), ws, d_w=d_w, expert_offsets=ends)
    dw = d_y[-70:].double().t() @ last.double()
    err = 140 * 2.0 ** -24 * (d_y[-70:].double().abs().t() @ last.double().abs()) + 2.0 ** -24 * dw.abs()
    assert bool(((d_w[-1].double() - dw).abs() <= err).all()) and not bool(d_w[:-1].any())
    w64 = w[:, :N].contiguous()
    m.moe_expert_product_backward(d_y, None, w64, ws, d_a=d_a, expert_offsets=ends)
    want = d_y[-70:].double() @ w64[-1].double()
    err = 2 * N * 2.0 ** -24 * (d_y[-70:].double().abs() @ w64[-1].double().abs()) + 2.0 ** -8 * want.abs()
    assert bool(((d_a[-70:].double() - want).abs() <= err).all())
