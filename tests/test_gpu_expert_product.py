"""moe_expert_product and moe_expert_product_backward against their definitions in 64 bits.

Tolerance (u = 2^-24).  A sum of L products in fp32, in any order and with truncating adders, is off
by at most 2 L u of the sum of their sizes; what follows in fp32 (exp, division, products) takes at most
2^-18 of its result (gates up to 16 or so; 2^-15 beyond), and a result is rounded once, 2^-8 in bf16 and 2^-24 in fp32.  Gated:
d(silu(g) v) <= 1.1 |v| dg + |silu(g)| dv, |silu'| < 1.1.  The gradient in gate and up is d v f and d g s
with f = s (1 + g (1 - s)), |f| < 1.1, s < 1, whose terms are at most |g| s (1 - s) + s < 1.3.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
from gpu_util import DEV, host, i32_dev

gpu = pytest.mark.gpu
pytestmark = gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()


def randn(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def within(got, want, bound):
    """|got - want| <= bound; past bf16's largest value, (2 - 2^-7) 2^127, either that or infinity."""
    got, top = got.double(), (2 - 2.0 ** -7) * 2.0 ** 127
    past = want.abs() + bound > top
    fine = torch.where(past, got * want.sign() >= torch.minimum(want.abs() - bound, torch.full_like(want, top)),
                       (got - want).abs() <= bound)
    return bool(fine.all())


class Rows:
    """The experts' rows of a buffer: runs with `spare` rows behind them, or blocks."""

    def __init__(self, counts, block_rows=0, first=0, spare=3, pad=1):
        self.counts, self.block_rows = list(counts), block_rows
        if block_rows:
            self.starts = [e * block_rows for e in range(len(counts))]
            self.total = len(counts) * block_rows + spare
            self.by = {"masked_counts": i32_dev(np.array(counts)), "block_rows": block_rows}
        else:
            ends = first + np.cumsum([0] + [-(-c // pad) * pad for c in counts])
            self.starts, self.total = [int(v) for v in ends[:-1]], int(ends[-1]) + spare
            self.counts = [int(v) for v in np.diff(ends)]
            self.by = {"expert_offsets": i32_dev(ends)}
        self.used = torch.zeros(self.total, dtype=torch.bool, device=DEV)
        for s, c in zip(self.starts, self.counts):
            self.used[s:s + c] = True

    def fill(self, t):
        """Garbage where no expert has rows: nothing of it may reach a result."""
        t[~self.used] = float("nan")
        return t

    def each(self):
        return [(e, slice(s, s + c)) for e, (s, c) in enumerate(zip(self.starts, self.counts)) if c]


def workspace(need):
    whole = torch.full((need + (1 << 16),), 0xff, dtype=torch.uint8, device=DEV)
    return whole[:need], whole[need:]


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def forward(rows, a, w, gated, keep, stream=None, ws=None):
    E, n, K = w.shape
    N = n // 2 if gated else n
    y = torch.full((rows.total, N), -7.0, dtype=BF, device=DEV)
    pre = torch.full((rows.total, 2 * N), -7.0, dtype=BF, device=DEV) if keep else None
    past = None
    if ws is None:
        ws, past = workspace(m.moe_expert_product_workspace_bytes(rows.total, E, N, K, gated))
    st = status()
    m.moe_expert_product(a, w, y, ws, gated=gated, pre=pre, dev_status=st, stream=stream, **rows.by)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (past is None or bool((past == 0xff).all()))
    return y, pre


def check_forward(rows, a, w, gated, y, pre):
    N, K = y.shape[1], a.shape[1]
    for e, at in rows.each():
        x, we = a[at].double(), w[e].double()
        out, err = x @ we.t(), 2 * K * U * (x.abs() @ we.abs().t())
        fp32 = 2.0 ** -18
        if gated:
            if pre is not None:
                assert bool(((pre[at].double() - out).abs() <= err + 2.0 ** -8 * out.abs()).all()), e
            g, up = out[:, :N], out[:, N:]
            silu = g * torch.sigmoid(g)
            eg, eu = err[:, :N], err[:, N:]
            fp32 = torch.where(g.abs() <= 16, 2.0 ** -18, 2.0 ** -15)
            out, err = silu * up, 1.1 * up.abs() * eg + silu.abs() * eu + 1.1 * eg * eu
        bound = err + (2.0 ** -8 + fp32) * out.abs() + 1e-38
        assert within(y[at], out, bound), e
    assert bool((y[~rows.used] == -7).all())
    assert pre is None or bool((pre[~rows.used] == -7).all())


def backward(rows, d_y, a, w, pre, d_w_type, want_a=True, stream=None, ws=None):
    E, N, K = w.shape
    d_a = torch.full((rows.total, 2 * K if pre is not None else K), -7.0, dtype=BF, device=DEV) if want_a else None
    d_w = None if d_w_type is None else torch.full((E, N, K), -7.0, dtype=d_w_type, device=DEV)
    past = None
    if ws is None:
        ws, past = workspace(m.moe_expert_product_backward_workspace_bytes(rows.total, E, N, K))
    st = status()
    m.moe_expert_product_backward(d_y, a, w, ws, d_a=d_a, d_w=d_w, pre=pre, dev_status=st, stream=stream, **rows.by)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (past is None or bool((past == 0xff).all()))
    return d_a, d_w


def check_backward(rows, d_y, a, w, pre, d_a, d_w):
    E, N, K = w.shape
    for e in range(E):
        at = slice(rows.starts[e], rows.starts[e] + rows.counts[e])
        dy, we = d_y[at].double(), w[e].double()
        if d_w is not None:
            x = a[at].double()
            out = dy.t() @ x
            half = U if d_w.dtype == F32 else 2.0 ** -8
            bound = 2 * max(1, rows.counts[e]) * U * (dy.abs().t() @ x.abs()) + half * out.abs()
            assert bool(((d_w[e].double() - out).abs() <= bound).all()), e
        if d_a is None or rows.counts[e] == 0:
            continue
        d, err, fp32 = dy @ we, 2 * N * U * (dy.abs() @ we.abs()), 2.0 ** -18
        if pre is not None:
            g, up = pre[at, :K].double(), pre[at, K:].double()
            s = torch.sigmoid(g)
            f = s * (1 + g * (1 - s))
            fp32 = torch.where(g.abs() <= 16, 2.0 ** -18, 2.0 ** -15)
            terms = s + (g * s * (1 - s)).abs()      # of f, which may cancel
            err = torch.cat((1.1 * up.abs() * err + fp32 * terms * (d * up).abs(), (g * s).abs() * err), 1)
            fp32 = torch.cat((fp32, fp32), 1)
            d = torch.cat((d * up * f, d * g * s), 1)
        bound = err + (2.0 ** -8 + fp32) * d.abs() + 1e-38
        assert within(d_a[at], d, bound), e
    assert d_a is None or bool((d_a[~rows.used] == -7).all())


CASES = [  # N, K, counts
    (8, 8, [1]), (8, 16, [1, 0, 2]), (64, 64, [64]), (128, 64, [16]), (72, 136, [0, 5, 1]),
    (256, 128, [33, 0, 0, 64]), (136, 400, [2, 0, 17, 0, 9]), (328, 1048, [16, 15, 0, 33]),
    (256, 2048, [1, 1]), (640, 5120, [1]), (96, 264, [129, 64]), (200, 512, [300, 1, 128]),
    (520, 96, [513, 127]), (40, 64, [3, 0] * 32), (1000, 3600, [7]), (24, 7168, [1, 0, 0, 2, 8, 1]),
    (1600, 256, [260, 90]), (40, 96, [2100, 0, 2400]), (512, 512, [256, 255, 257]), (264, 328, [31, 32, 33, 65])]


@pytest.mark.parametrize("N,K,counts", CASES)
@pytest.mark.parametrize("gated,keep", [(False, False), (True, True)])
def test_forward_runs(N, K, counts, gated, keep):
    rows = Rows(counts, first=5)
    a = rows.fill(randn(1, rows.total, K))
    w = randn(2, len(counts), 2 * N if gated else N, K, scale=K ** -0.5)
    y, pre = forward(rows, a, w, gated, keep)
    check_forward(rows, a, w, gated, y, pre)


@pytest.mark.parametrize("N,K,counts", CASES[::2])
@pytest.mark.parametrize("gated", [False, True])
def test_forward_blocks(N, K, counts, gated):
    rows = Rows(counts, block_rows=max(counts) + 3)
    a = rows.fill(randn(3, rows.total, K))
    w = randn(4, len(counts), 2 * N if gated else N, K, scale=K ** -0.5)
    y, _ = forward(rows, a, w, gated, False)
    check_forward(rows, a, w, gated, y, None)


@pytest.mark.parametrize("N,K,counts", CASES)
@pytest.mark.parametrize("gate,d_w_type", [(False, F32), (True, BF)])
def test_backward_runs(N, K, counts, gate, d_w_type):
    rows = Rows(counts, first=5)
    a, d_y = rows.fill(randn(5, rows.total, K)), rows.fill(randn(6, rows.total, N, scale=0.1))
    w = randn(7, len(counts), N, K, scale=K ** -0.5)
    pre = rows.fill(randn(8, rows.total, 2 * K)) if gate else None
    d_a, d_w = backward(rows, d_y, a, w, pre, d_w_type)
    check_backward(rows, d_y, a, w, pre, d_a, d_w)


@pytest.mark.parametrize("N,K,counts", CASES[1::2])
def test_backward_blocks(N, K, counts):
    rows = Rows(counts, block_rows=max(counts) + 1, spare=0)
    a, d_y = rows.fill(randn(9, rows.total, K)), rows.fill(randn(10, rows.total, N, scale=0.1))
    w = randn(11, len(counts), N, K, scale=K ** -0.5)
    d_a, d_w = backward(rows, d_y, a, w, None, F32)
    check_backward(rows, d_y, a, w, None, d_a, d_w)
    only_a, none = backward(rows, d_y, None, w, None, None)
    assert none is None and torch.equal(only_a, d_a)
    none, only_w = backward(rows, d_y, a, w, None, F32, want_a=False)
    assert none is None and torch.equal(only_w, d_w)


def test_gate_values_far_from_zero():
    """Gates where exp overflows or underflows: no NaN, silu and its gradient at their limits.  (2^-18
    is for gates up to 16; |gate| 2^-24 and 2^-21 more cover the others, below 2^-15 up to 120.)"""
    K = 64
    rows = Rows([40], spare=0)
    a = torch.zeros(40, K, dtype=BF, device=DEV)
    gates = torch.tensor([0, 1, -1, 30, -30, 80, -80, 88, -88, 89, -89, 95, -95, 104, -104, 127, -127, 400,
                          -400, 3e4, -3e4, 1e30, -1e30, 3e38, -3e38, -1.25], device=DEV).to(BF)
    a[: len(gates), 0] = gates
    a[:, 1] = 1
    w = torch.zeros(1, 16, K, dtype=BF, device=DEV)
    w[0, :8, 0] = 1                     # gate = the row's first value
    w[0, 8:, 1] = 2                     # up = 2
    y, pre = forward(rows, a, w, True, True)
    check_forward(rows, a, w, True, y, pre)
    d_y, w2 = torch.ones(40, 8, dtype=BF, device=DEV), torch.ones(1, 8, 8, dtype=BF, device=DEV)
    d_pre, _ = backward(rows, d_y, y, w2, pre, None)
    check_backward(rows, d_y, None, w2, pre, d_pre, None)
    assert not bool(d_pre.isnan().any())


def test_what_is_not_finite_stays_in_its_row():
    N, K = 136, 200
    rows = Rows([20, 70, 3])
    a, w = rows.fill(randn(12, rows.total, K)), randn(13, 3, 2 * N, K, scale=K ** -0.5)
    y, _ = forward(rows, a, w, True, False)
    a[7, 3], a[25, K - 1] = float("nan"), float("inf")
    z, _ = forward(rows, a, w, True, False)
    same = torch.ones(rows.total, dtype=torch.bool, device=DEV)
    same[7] = same[25] = False
    assert torch.equal(y[same], z[same]) and bool(z[7].isnan().all()) and not bool(z[25].isfinite().any())
    # in the weights' gradient it stays with its expert
    d_y, w = rows.fill(randn(14, rows.total, N)), w[:, :N].contiguous()
    d_y[7, 0] = float("nan")
    a[7, 3], a[25, K - 1] = 1, 1
    _, d_w = backward(rows, d_y, a, w, None, F32)
    assert bool(d_w[0, 0].isnan().all()) and bool(d_w[0, 1:].isfinite().all()) and bool(d_w[1:].isfinite().all())


@pytest.mark.parametrize("E,counts", [(1024, [1] * 1024), (1024, [0] * 1023 + [5]), (777, [2, 0, 0] * 259)])
def test_many_experts(E, counts):
    N, K = 24, 72
    rows = Rows(counts)
    a, w = rows.fill(randn(15, rows.total, K)), randn(16, E, N, K, scale=K ** -0.5)
    y, _ = forward(rows, a, w, False, False)
    check_forward(rows, a, w, False, y, None)
    d_y = rows.fill(randn(17, rows.total, N))
    d_a, d_w = backward(rows, d_y, a, w, None, BF)
    check_backward(rows, d_y, a, w, None, d_a, d_w)


def test_no_rows():
    w = randn(18, 2, 16, 24)
    for total, by in ((0, {"expert_offsets": i32_dev(np.zeros(3))}),
                      (9, {"expert_offsets": i32_dev(np.full(3, 4))}),
                      (8, {"masked_counts": i32_dev(np.zeros(2)), "block_rows": 4})):
        a, d_y = torch.full((total, 24), float("nan"), dtype=BF, device=DEV), torch.empty(total, 16, dtype=BF, device=DEV)
        y, d_a = torch.full_like(d_y, 3), torch.full_like(a, 3)
        ws, _ = workspace(m.moe_expert_product_workspace_bytes(total, 2, 16, 24))
        st = status()
        m.moe_expert_product(a, w, y, ws, dev_status=st, **by)
        d_w = torch.full((2, 16, 24), 7.0, device=DEV)
        m.moe_expert_product_backward(d_y, a, w, ws, d_a=d_a, d_w=d_w, dev_status=st, **by)
        assert bool((y == 3).all()) and bool((d_a == 3).all()) and bool((d_w == 0).all())
        assert int(st.item()) == 0


BAD = 1 << m.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("ends,flag,cut", [
    ([0, 4, 30], BAD, [(0, 4), (4, 10)]), ([-3, 4, 10], BAD, [(0, 0), (4, 10)]),
    ([0, 20, 30], BAD, [(0, 10), (0, 0)]), ([2, 9, 5], BAD, None), ([0, 10, 10], 0, [(0, 10), (0, 0)]),
    ([10, 10, 10], 0, [(0, 0), (0, 0)]), ([2 ** 31 - 1] * 3, BAD, [(0, 0), (0, 0)])])
def test_ranges_that_leave_the_buffer(ends, flag, cut):
    N, K = 16, 72
    a, w, d_y = randn(19, 10, K), randn(20, 2, N, K), randn(21, 10, N)
    tail = torch.full((64, N), 9.0, dtype=BF, device=DEV)
    y, after = tail[:10], tail[10:]
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(10, 2, N, K))
    st = status()
    y.fill_(-7)
    m.moe_expert_product(a, w, y, ws, expert_offsets=i32_dev(np.array(ends)), dev_status=st)
    d_a, d_w = torch.full((10, K), -7.0, dtype=BF, device=DEV), torch.empty(2, N, K, device=DEV)
    st2 = status()
    m.moe_expert_product_backward(d_y, a, w, ws, d_a=d_a, d_w=d_w, expert_offsets=i32_dev(np.array(ends)),
                                  dev_status=st2)
    assert int(st.item()) == flag and int(st2.item()) == flag and bool((after == 9).all())
    if cut is None:
        return
    rows = Rows([0, 0])
    rows.starts, rows.counts = [s for s, _ in cut], [t - s for s, t in cut]
    rows.used = torch.zeros(10, dtype=torch.bool, device=DEV)
    for s, t in cut:
        rows.used[s:t] = True
    check_forward(rows, a, w, False, y, None)
    check_backward(rows, d_y, a, w, None, d_a, d_w)


def test_a_count_past_its_block():
    N, K = 24, 40
    a, w, y = randn(22, 12, K), randn(23, 3, N, K), torch.full((12, N), -7.0, dtype=BF, device=DEV)
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(12, 3, N, K))
    st = status()
    m.moe_expert_product(a, w, y, ws, masked_counts=i32_dev(np.array([2, 9, -1])), block_rows=4, dev_status=st)
    rows = Rows([2, 4, 0], block_rows=4, spare=0)
    check_forward(rows, a, w, False, y, None)
    assert int(st.item()) == BAD


def test_determinism_and_a_shared_workspace():
    """The same bytes every time, whatever the workspace held before, and with two captured graphs
    that share it, replayed in turn."""
    N, K, counts = 264, 1024, [40, 0, 300, 7]
    rows = Rows(counts)
    a, w = rows.fill(randn(24, rows.total, K)), randn(25, 4, 2 * N, K, scale=K ** -0.5)
    d_y, w2 = rows.fill(randn(26, rows.total, N)), randn(27, 4, N, K, scale=K ** -0.5)
    ws, _ = workspace(max(m.moe_expert_product_workspace_bytes(rows.total, 4, N, K, True),
                          m.moe_expert_product_backward_workspace_bytes(rows.total, 4, N, K)))
    y, pre = forward(rows, a, w, True, True, ws=ws)
    d_a, d_w = backward(rows, d_y, a, w2, None, F32, ws=ws)
    out = [torch.full_like(t, -7.0) for t in (y, pre, d_a, d_w)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        m.moe_expert_product(a, w, out[0], ws, gated=True, pre=out[1], **rows.by)
    with torch.cuda.graph(graphs[1]):
        m.moe_expert_product_backward(d_y, a, w2, ws, d_a=out[2], d_w=out[3], **rows.by)
    for turn in range(3):
        for t in out:
            t.fill_(-7)
        ws.fill_(0xff if turn % 2 else 0)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(out, (y, pre, d_a, d_w)))


def test_on_another_stream():
    N, K = 136, 520
    rows = Rows([30, 9])
    a, w = rows.fill(randn(28, rows.total, K)), randn(29, 2, N, K)
    y, _ = forward(rows, a, w, False, False)
    side = torch.cuda.Stream()
    z, _ = forward(rows, a, w, False, False, stream=side)
    assert torch.equal(y, z)


def test_refusals():
    a, w, y = randn(30, 4, 16), randn(31, 2, 8, 16), torch.empty(4, 8, dtype=BF, device=DEV)
    ws, _ = workspace(m.moe_expert_product_workspace_bytes(4, 2, 8, 16))
    ends = i32_dev(np.array([0, 2, 4]))
    ok = dict(expert_offsets=ends)
    with pytest.raises(ValueError, match="y: expected shape"):
        m.moe_expert_product(a, w, y[:3], ws, **ok)
    with pytest.raises(ValueError, match="a: expected shape"):
        m.moe_expert_product(randn(32, 4, 24), w, y, ws, **ok)
    with pytest.raises(ValueError, match="even number"):
        m.moe_expert_product(a, randn(33, 2, 9, 16), y, ws, gated=True, **ok)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_expert_product(a, w.transpose(1, 2), y, ws, **ok)
    with pytest.raises(TypeError, match="dtype"):
        m.moe_expert_product(a.float(), w, y, ws, **ok)
    with pytest.raises(ValueError, match="expert_offsets: expected shape"):
        m.moe_expert_product(a, w, y, ws, expert_offsets=ends[:2])
    with pytest.raises(m.MoeError, match="ws_bytes"):
        m.moe_expert_product(a, w, y, ws[:8], **ok)
    with pytest.raises(m.MoeError, match="not both"):
        m.moe_expert_product(a, w, y, ws)
    with pytest.raises(m.MoeError, match="`pre` is of gated"):
        m.moe_expert_product(a, w, y, ws, pre=torch.empty(4, 16, dtype=BF, device=DEV), **ok)
    with pytest.raises(ValueError, match="neither is wanted"):
        m.moe_expert_product_backward(y, a, w, ws, **ok)
    with pytest.raises(ValueError, match="a: needed"):
        m.moe_expert_product_backward(y, None, w, ws, d_w=torch.empty_like(w), **ok)
    with pytest.raises(ValueError, match="d_a: needed"):
        m.moe_expert_product_backward(y, a, w, ws, d_w=torch.empty_like(w), pre=torch.empty(4, 32, dtype=BF, device=DEV), **ok)
    with pytest.raises(ValueError, match="d_a: expected shape"):
        m.moe_expert_product_backward(y, a, w, ws, d_a=torch.empty_like(a), pre=torch.empty(4, 32, dtype=BF, device=DEV), **ok)
    with pytest.raises(m.MoeError, match="16-byte"):
        shifted = torch.empty(4 * 16 + 1, dtype=BF, device=DEV)[1:].view(4, 16)
        m.moe_expert_product(shifted, w, y, ws, **ok)


def test_an_expert_as_it_is_trained():
    """Gate and up, silu, down and the way back, against automatic differentiation in 64 bits.

    In the 2-norm: h, y, pre and the gradients are rounded to bf16 (2^-8 of each value at most, so of the
    norm); y takes h's and its own, d_w2 the rounding of h, d_x and d_w13 those of pre (twice, through
    the activation's derivative and its factor), of d_pre and their own: 5 * 2^-8 at most."""
    H, F, counts = 264, 136, [40, 0, 77]
    rows = Rows(counts, pad=8)
    x, w13 = randn(40, rows.total, H), randn(41, 3, 2 * F, H, scale=H ** -0.5)
    w2, d_y = randn(42, 3, H, F, scale=F ** -0.5), randn(43, rows.total, H)
    h, pre = forward(rows, x, w13, True, True)
    y, _ = forward(rows, h, w2, False, False)
    d_pre, d_w2 = backward(rows, d_y, h, w2, pre, F32)
    d_x, d_w13 = backward(rows, d_pre, x, w13, None, F32)
    leaves = [t.double().requires_grad_() for t in (x, w13, w2)]
    total = 0
    want = torch.zeros(rows.total, H, dtype=torch.float64, device=DEV)
    for e, at in rows.each():
        both = leaves[0][at] @ leaves[1][e].t()
        out = (torch.nn.functional.silu(both[:, :F]) * both[:, F:]) @ leaves[2][e].t()
        want[at] = out.detach()
        total = total + (out * d_y[at].double()).sum()
    total.backward()
    used = rows.used
    for got, ref in ((y[used], want[used]), (d_x[used], leaves[0].grad[used]), (d_w13, leaves[1].grad),
                     (d_w2, leaves[2].grad)):
        assert float((got.double() - ref).norm() / ref.norm()) <= 5 * 2.0 ** -8


def test_gradient_is_that_of_differences():
    """<d_w, V> and <d_a, V> against differences of f = <d_y, product> in 64 bits (f is linear in
    each, so a difference is exact but for rounding); and of the gated rows through gate and up."""
    N, K, rows = 24, 40, Rows([9, 0, 5], spare=0)
    a, w, d_y = randn(44, 14, K), randn(45, 3, N, K), randn(46, 14, N)
    pre = randn(47, 14, 2 * K)
    d_a, d_w = backward(rows, d_y, a, w, None, F32)
    d_pre, _ = backward(rows, d_y, a, w, pre, None)

    def f(x, weights):
        return float(sum((x[at] @ weights[e].t() * d_y[at].double()).sum() for e, at in rows.each()))

    def gate(p):
        return torch.nn.functional.silu(p[:, :K]) * p[:, K:]

    t = 1e-4
    a64, w64, p64 = a.double(), w.double(), pre.double()
    v, vw, vp = (randn(48 + i, *s.shape, dtype=F32).double() for i, s in enumerate((a, w, pre)))
    for got, along, plus, minus in ((d_a, v, f(a64 + t * v, w64), f(a64 - t * v, w64)),
                                    (d_w, vw, f(a64, w64 + t * vw), f(a64, w64 - t * vw)),
                                    (d_pre, vp, f(gate(p64 + t * vp), w64), f(gate(p64 - t * vp), w64))):
        # each product's gradient is rounded to bf16 at most (2^-8); the difference takes t^2 and 1e-16 f / t
        bound = 2.0 ** -8 * float((got.double() * along).abs().sum()) + 1e-3
        assert abs((plus - minus) / (2 * t) - float((got.double() * along).sum())) <= bound
