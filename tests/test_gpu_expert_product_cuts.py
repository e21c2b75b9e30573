"""The experts' bf16 products where tiles are cut between pairs and joined from their parts.

Which calls cut is worked out here from the rule that the kernel follows, so that the cases below are known
to cut on 148 and 152 SMs, and then seen on the GPU: the last 1,280 bytes of the workspace are the counters
of parts that have arrived, cleared at the start of a call that may cut, one for each CTA of the pair at each
cut tile's first part.  Tolerances as in test_gpu_expert_product.py."""
import os
import re

import pytest
import torch

import combine_moe_route_06_gb300 as m
from conftest import ROOT
from gpu_util import DEV
from test_gpu_expert_product import (BF, F32, Rows, backward, check_backward, check_forward, forward, randn,
                                     workspace)

gpu = pytest.mark.gpu
SOURCE = open(os.path.join(ROOT, "combine_moe_route_06_gb300", "csrc", "expert_product.cu")).read()


def constant(name):
    return int(re.search(rf"\b{name} = (\d+)[,;]", SOURCE).group(1))


STEP, TILE, CUT = constant("kStep"), constant("kTileRows"), constant("kCutSteps")
MIN_PART, MIN_WIDE = constant("kMinPart"), constant("kMinPartWide")


@pytest.fixture(scope="module")
def lib():
    m.build()


def up(a, b):
    return -(-a // b)


def tile_rows(pairs, tiles_a, rows, experts):
    most = TILE
    while most > 64 and tiles_a * (2 * rows // most + experts) <= pairs:
        most //= 2
    return most


def plan(pairs, tiles, steps, widest):
    """Tiles that pairs take whole in turn, and parts of every tile: tiles[e] of steps[e] for each expert."""
    tasks, total, longest = sum(tiles), sum(t * s for t, s in zip(tiles, steps)), max(steps)
    turns = up(tasks, pairs)
    if longest <= CUT:
        waves = turns
    elif longest * tasks > 2 * total:           # a few experts have most of the steps
        waves = 0
    elif (turns * pairs - tasks) * longest <= CUT * pairs:
        waves = turns
    else:
        waves = max(0, tasks // pairs - 1)
    whole = min(tasks, waves * pairs)
    starts = [0]
    for t, s in zip(tiles, steps):
        for _ in range(t):
            starts.append(starts[-1] + s)
    rest = total - starts[whole]
    parts = min(pairs, max(tasks - whole, rest // (MIN_PART if widest <= 64 else MIN_WIDE)))
    ends = [starts[whole] + i * (rest // parts) + min(i, rest % parts) for i in range(1, parts)] if parts else []
    return whole, [1 + sum(starts[i] < end < starts[i + 1] for end in ends) for i in range(tasks)]


def by_rows(pairs, tile_pairs, rows, outputs, length):
    """plan() of a product over the experts' rows: `outputs` a row, sums of `length`."""
    tiles = up(outputs, TILE)
    most = tile_rows(tile_pairs, tiles, rows.total, min(rows.total, len(rows.counts)))
    each = [up(c, most) for c in rows.counts]
    return plan(pairs, [tiles * n for n in each], [up(length, STEP)] * len(each), min(most, max(rows.counts)))


def by_weights(pairs, tile_pairs, rows, N, K):
    """plan() of the weights' gradient."""
    E, tiles = len(rows.counts), up(N, TILE)
    most = tile_rows(tile_pairs, E * tiles, K, 1)
    return plan(pairs, [tiles * up(K, most)] * E, [max(1, up(c, STEP)) for c in rows.counts], most)


class Counts:
    """The experts' rows without a GPU, as Rows(counts, first=3) has them."""

    def __init__(self, counts):
        self.counts, self.total = counts, 3 + sum(counts) + 3


def cut(parts):
    return sum(n > 1 for n in parts)


def device_pairs():
    return min(torch.cuda.get_device_properties(0).multi_processor_count, 160) // 2


def arrived(ws):
    return ws[-1280:].view(torch.int32)


FORWARD = [  # N, K, counts, gated, whether tiles are taken whole before the cut ones, most parts of a tile
    (264, 7168, [600], True, False, 3), (8, 20000, [40, 3], False, False, 9), (136, 3200, [1] * 40, True, False, 2),
    (2560, 5120, [700, 800, 900], False, False, 2), (2560, 3200, [2000, 1900], False, True, 2)]
ROWS = [  # N, K, counts, gate, whether ..., most parts
    (5120, 264, [600, 40], True, False, 3), (5120, 264, [600, 40], False, False, 3),
    (5120, 2048, [700, 800, 900], True, False, 2), (3200, 2560, [2000, 1900], True, True, 2),
    (3200, 2560, [2000, 1900], False, True, 2)]
WEIGHTS = [  # N, K, counts, whether ..., most parts
    (2560, 2048, [5000, 5000], True, 2), (2560, 2048, [5000, 5000, 0], True, 3),
    (512, 768, [6000, 3, 0, 2, 1, 64], False, 3), (8, 16, [20001], False, 9)]


def plan_forward(pairs, rows, N, K, gated):
    return by_rows(pairs, pairs, rows, 2 * N if gated else N, K)


@pytest.mark.parametrize("pairs", [74, 76])
def test_the_cases_cut(pairs):
    for N, K, counts, gated, turn, most in FORWARD:
        whole, parts = plan_forward(pairs, Counts(counts), N, K, gated)
        assert cut(parts) and max(parts) >= most and (whole > 0) == turn, (N, K)
    for N, K, counts, _, turn, most in ROWS:
        whole, parts = by_rows(pairs, pairs, Counts(counts), K, N)
        assert cut(parts) and max(parts) >= most and (whole > 0) == turn, (N, K)
    for N, K, counts, turn, most in WEIGHTS:
        whole, parts = by_weights(pairs, pairs, Counts(counts), N, K)
        assert cut(parts) and max(parts) >= most and (whole > 0) == turn, (N, K)


def assert_cut(ws, parts):
    """The counters of a call with one product: at each cut tile's first pair both CTAs of it have
    counted all of its parts, or all but the one that found the others there."""
    assert cut(parts)
    got = sorted(v for v in arrived(ws).tolist() if v)
    want = sorted(n for n in parts if n > 1 for _ in range(2))
    assert len(got) == len(want) and all(w - 1 <= g <= w for g, w in zip(got, want))


@gpu
@pytest.mark.parametrize("N,K,counts,gated,turn,most", FORWARD)
def test_forward(lib, N, K, counts, gated, turn, most):
    rows = Rows(counts, first=3)
    a, w = rows.fill(randn(1, rows.total, K)), randn(2, len(counts), 2 * N if gated else N, K, scale=K ** -0.5)
    ws, past = workspace(m.moe_expert_product_workspace_bytes(rows.total, len(counts), N, K, gated))
    y, pre = forward(rows, a, w, gated, gated, ws=ws)
    check_forward(rows, a, w, gated, y, pre)
    assert_cut(ws, plan_forward(device_pairs(), rows, N, K, gated)[1])
    assert bool((past == 0xff).all())


@gpu
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("N,K,counts,gate,turn,most", ROWS)
def test_rows_gradient(lib, N, K, counts, gate, turn, most, both):
    """Alone, and beside the weights' gradient on pairs of its own."""
    rows = Rows(counts, first=3)
    E = len(counts)
    d_y, a = rows.fill(randn(3, rows.total, N, scale=0.1)), rows.fill(randn(4, rows.total, K))
    w, pre = randn(5, E, N, K, scale=N ** -0.5), rows.fill(randn(6, rows.total, 2 * K)) if gate else None
    ws, past = workspace(m.moe_expert_product_backward_workspace_bytes(rows.total, E, N, K))
    d_a, d_w = backward(rows, d_y, a, w, pre, F32 if both else None, ws=ws)
    check_backward(rows, d_y, a, w, pre, d_a, d_w)
    if both:
        assert N != 5120 or K != 264 or bool(arrived(ws)[:160].any())    # (rows' counters, then the weights')
    else:
        assert_cut(ws, by_rows(device_pairs(), device_pairs(), rows, K, N)[1])
    assert bool((past == 0xff).all())


@gpu
@pytest.mark.parametrize("d_w_type", [F32, BF])
@pytest.mark.parametrize("N,K,counts,turn,most", WEIGHTS)
def test_weights_gradient(lib, N, K, counts, turn, most, d_w_type):
    rows = Rows(counts, first=3)
    E = len(counts)
    d_y, a = rows.fill(randn(7, rows.total, N, scale=0.1)), rows.fill(randn(8, rows.total, K))
    w = randn(9, E, N, K)
    ws, past = workspace(m.moe_expert_product_backward_workspace_bytes(rows.total, E, N, K))
    _, d_w = backward(rows, d_y, a, w, None, d_w_type, want_a=False, ws=ws)
    check_backward(rows, d_y, a, w, None, None, d_w)
    assert_cut(ws, by_weights(device_pairs(), device_pairs(), rows, N, K)[1])
    assert bool((past == 0xff).all())


def repeated(make, ws, times=10):
    """The bytes of `make()` are the same every time, with the workspace as it was left or overwritten."""
    want = make()
    for i in range(times - 1):
        if i % 3 == 1:
            ws.fill_(0xff)
        for got, first in zip(make(), want):
            assert torch.equal(got.view(torch.uint8), first.view(torch.uint8))


@gpu
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,counts,gated,turn,most", FORWARD)
def test_the_same_bytes_forward(lib, N, K, counts, gated, turn, most, zero):
    """Parts are added in an order of their own, not in that of their arrival.  Also with rows of
    zeros and negative weights, whose sums are zeros with a sign."""
    rows, E = Rows(counts, first=3, spare=3), len(counts)
    a, w = randn(10, rows.total, K), randn(11, E, 2 * N if gated else N, K, scale=K ** -0.5)
    if zero:
        a, w = torch.zeros_like(a), -w.abs()
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(rows.total, E, N, K, gated))
    repeated(lambda: [t for t in forward(rows, a, w, gated, gated, ws=ws) if t is not None], ws)
    assert bool(arrived(ws).any())


@gpu
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,counts,gate,turn,most", ROWS)
def test_the_same_bytes_rows(lib, N, K, counts, gate, turn, most, zero):
    rows, E = Rows(counts, first=3), len(counts)
    d_y, w = randn(12, rows.total, N, scale=0.1), randn(13, E, N, K, scale=N ** -0.5)
    pre = randn(14, rows.total, 2 * K) if gate else None
    if zero:
        d_y, w = torch.zeros_like(d_y), -w.abs()
    ws, _ = workspace(m.moe_expert_product_backward_workspace_bytes(rows.total, E, N, K))
    repeated(lambda: [backward(rows, d_y, None, w, pre, None, ws=ws)[0]], ws)
    assert bool(arrived(ws).any())


@gpu
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,counts,turn,most", WEIGHTS)
def test_the_same_bytes_weights(lib, N, K, counts, turn, most, zero):
    rows, E = Rows(counts, first=3), len(counts)
    d_y, a, w = randn(15, rows.total, N, scale=0.1), randn(16, rows.total, K), randn(17, E, N, K)
    if zero:
        d_y, a = torch.zeros_like(d_y), -a.abs()
    ws, _ = workspace(m.moe_expert_product_backward_workspace_bytes(rows.total, E, N, K))
    repeated(lambda: [backward(rows, d_y, a, w, None, F32, want_a=False, ws=ws)[1]], ws)
    assert bool(arrived(ws).any())


@gpu
def test_two_graphs_share_a_workspace(lib):
    """Two captured calls that both cut tiles, replayed in turn over one workspace, whatever it holds:
    each clears the counters and reads no part that the other has left."""
    E, rows = 2, Rows([600, 40], first=3)
    a, w = rows.fill(randn(18, rows.total, 7168)), randn(19, E, 528, 7168, scale=7168 ** -0.5)
    d_y, w2 = rows.fill(randn(20, rows.total, 5120, scale=0.1)), randn(21, E, 5120, 264, scale=5120 ** -0.5)
    act, pre2 = rows.fill(randn(22, rows.total, 264)), rows.fill(randn(23, rows.total, 528))
    ws, _ = workspace(max(m.moe_expert_product_workspace_bytes(rows.total, E, 264, 7168, True),
                          m.moe_expert_product_backward_workspace_bytes(rows.total, E, 5120, 264)))
    y, pre = forward(rows, a, w, True, True, ws=ws)
    check_forward(rows, a, w, True, y, pre)
    assert bool(arrived(ws)[:160].any())
    d_a, d_w = backward(rows, d_y, act, w2, pre2, F32, ws=ws)
    check_backward(rows, d_y, act, w2, pre2, d_a, d_w)
    assert bool(arrived(ws)[:160].any())
    out = [torch.full_like(t, -7.0) for t in (y, pre, d_a, d_w)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        m.moe_expert_product(a, w, out[0], ws, gated=True, pre=out[1], **rows.by)
    with torch.cuda.graph(graphs[1]):
        m.moe_expert_product_backward(d_y, act, w2, ws, d_a=out[2], d_w=out[3], pre=pre2, **rows.by)
    for turn in range(4):
        for t in out:
            t.fill_(-7)
        ws.fill_((0xff, 0, 1, 0x7f)[turn])
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(out, (y, pre, d_a, d_w)))
