"""Training direction: moe_balance_loss, moe_route_backward and moe_combine_backward against
their definitions in 64 bits, and the gradients against differences of the definitions.

Tolerances.  The kernels compute in fp32 (unit u = 2^-24).  With |l - max| <= 40 the argument of
exp is off by at most 40 u, exp itself by 2 units, a sum of n terms by (n/32 + 8) u relative to the
sum of magnitudes (32 lanes, then trees), so a probability is off by less than (50 + E/16) u
relative and a mean over T tokens by another (T/64 + 16) u.  REL below covers E <= 1024 and
T <= 4096 with a factor of two: 2 * (50 + 64 + 64 + 16) u < 2.4e-5.  A bf16 gradient adds half a
unit of 8 bits, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
import moe_synth as ms
from gpu_util import DEV, bf16_dev, bf16_host, f32_dev, host, i32_dev

pytestmark = pytest.mark.gpu
REL = 2.4e-5
RNG = np.random.default_rng


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()


# ------------------------------------------------------------------ definitions in 64 bits

def losses64(l, ids, mask):
    """(losses, counts, prob_mean, lse, n_valid) of logits l [S,T,E]."""
    S, T, E = l.shape
    k = ids.shape[2]
    counts, n_valid = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    prob, lse, losses = np.zeros((S, E)), np.zeros((S, T)), np.zeros(2)
    for s in range(S):
        ts = [t for t in range(T) if mask is None or mask[s, t]]
        n_valid[s] = len(ts)
        for t in ts:
            for e in ids[s, t]:
                if 0 <= e < E:
                    counts[s, e] += 1
            top = l[s, t].max()
            if top == -np.inf:
                lse[s, t] = -np.inf
                continue
            ex = np.exp(l[s, t] - top)
            lse[s, t] = top + np.log(ex.sum())
            prob[s] += ex / ex.sum()
            losses[1] += lse[s, t] ** 2 / (S * len(ts))
        if ts:
            prob[s] /= len(ts)
            losses[0] += E / (k * len(ts)) * (counts[s] * prob[s]).sum() / S
    return losses, counts, prob, lse, n_valid


def route_grad64(l, ids, w, dw, counts, n_valid, lse, d, mask):
    S, T, E = l.shape
    k = ids.shape[2]
    out = np.zeros((S, T, E))
    size = np.zeros((S, T, E))          # sum of the magnitudes of the terms, for the bound
    for s in range(S):
        for t in range(T):
            if mask is not None and not mask[s, t]:
                continue
            if d is not None and lse[s, t] != -np.inf:
                p = np.exp(l[s, t] - l[s, t].max())
                p /= p.sum()
                A = d[0] * E * counts[s] / (k * S * n_valid[s] ** 2)
                z = 2 * d[1] * lse[s, t] / (S * n_valid[s])
                out[s, t] += p * (A - (A * p).sum() + z)
                size[s, t] += p * (np.abs(A) + np.abs(A * p).sum() + abs(z))
            if w is not None:
                ok = (ids[s, t] >= 0) & (ids[s, t] < E)
                wj, gj = np.where(ok, w[s, t], 0), np.where(ok, dw[s, t], 0)
                g = wj * (gj - (wj * gj).sum())
                mag = np.abs(wj) * (np.abs(gj) + np.abs(wj * gj).sum())
                for j in range(k):
                    if ok[j]:
                        out[s, t, ids[s, t, j]] += g[j]
                        size[s, t, ids[s, t, j]] += mag[j]
    return out, size


def to_logits(l, dtype):
    t = torch.from_numpy(np.ascontiguousarray(l, np.float32)).to(DEV)
    t = t if dtype == "f32" else t.bfloat16()
    return t, t.double().cpu().numpy()


def run_losses(lt, ids, mask, stream=None):
    S, T, E = lt.shape
    o = {"counts": torch.full((S, E), -7, dtype=torch.int32, device=DEV),
         "prob_mean": torch.full((S, E), -7.0, device=DEV),
         "lse": torch.full((S, T), -7.0, device=DEV),
         "n_valid": torch.full((S,), -7, dtype=torch.int32, device=DEV),
         "losses": torch.full((2,), -7.0, device=DEV)}
    ws = torch.full((m.moe_balance_loss_workspace_bytes(S, T, E),), 0xff, dtype=torch.uint8,
                    device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    mk = None if mask is None else torch.from_numpy(mask.astype(np.uint8)).to(DEV)
    m.moe_balance_loss(lt, i32_dev(ids), o["counts"], o["prob_mean"], o["lse"], o["n_valid"],
                       o["losses"], ws, token_mask=mk, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return o, int(st.item())


def make(S, T, E, k, seed, mask=None, spread=1.0):
    r = RNG(seed)
    l = r.standard_normal((S, T, E)) * spread
    ids = np.stack([r.permutation(E)[:k] for _ in range(S * T)]).reshape(S, T, k) if T else \
        np.zeros((S, 0, k), int)
    mk = None
    if mask == "random":
        mk = r.random((S, T)) < 0.7
    elif mask == "tail":
        mk = np.arange(T)[None, :] < r.integers(0, T + 1, (S, 1))
    elif mask == "one_source_empty":
        mk = np.ones((S, T), bool)
        mk[S // 2] = False
    elif mask == "none_valid":
        mk = np.zeros((S, T), bool)
    return l, ids.astype(np.int32), mk


SHAPES = [(1, 1, 1, 1), (1, 128, 16, 2), (3, 33, 33, 5), (2, 65, 64, 8), (1, 700, 384, 6),
          (5, 17, 127, 3), (2, 40, 513, 32), (1, 90, 1024, 10), (70, 5, 20, 4), (310, 3, 8, 2),
          (2, 301, 128, 8), (3, 50, 100, 7), (1, 61, 36, 9),
          (4, 256, 48, 4), (3, 1024, 33, 2), (32, 16, 64, 3), (8, 128, 384, 6), (33, 16, 8, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [None, "random", "tail", "one_source_empty", "none_valid"])
@pytest.mark.parametrize("shape", SHAPES)
def test_losses_and_gradient(shape, mask, dtype):
    S, T, E, k = shape
    l, ids, mk = make(S, T, E, k, seed=S * 1000 + T, mask=mask, spread=2.0)
    lt, l = to_logits(l, dtype)
    o, status = run_losses(lt, ids, mk)
    losses, counts, prob, lse, n_valid = losses64(l, ids, mk)
    assert status == 0
    assert np.array_equal(host(o["counts"]), counts)
    assert np.array_equal(host(o["n_valid"]), n_valid)
    assert np.all(np.abs(host(o["prob_mean"]) - prob) <= REL * prob)
    assert np.all(np.abs(host(o["lse"]) - lse) <= REL * np.maximum(np.abs(lse), 1))
    # z: squares of lse, so twice its error, plus the mean's; lse may cross zero
    assert np.abs(host(o["losses"]) - losses)[0] <= REL * losses[0]
    assert np.abs(host(o["losses"]) - losses)[1] <= 3 * REL * max(losses[1], np.abs(lse).mean())

    r = RNG(7)
    w = r.random((S, T, k)).astype(np.float32)
    dw = r.standard_normal((S, T, k)).astype(np.float32)
    d = np.array([0.7, -0.3], np.float32)
    out = torch.full((S, T, E), -7.0, device=DEV, dtype=lt.dtype)
    mt = None if mk is None else torch.from_numpy(mk.astype(np.uint8)).to(DEV)
    for use_w, use_d in ((True, True), (True, False), (False, True)):
        m.moe_route_backward(lt, i32_dev(ids), f32_dev(w) if use_w else None,
                             f32_dev(dw) if use_w else None, o["lse"], o["counts"], o["n_valid"],
                             f32_dev(d) if use_d else None, out, token_mask=mt)
        got = out.double().cpu().numpy()
        want, size = route_grad64(l, ids, w if use_w else None, dw, counts, n_valid, lse,
                                  d if use_d else None, mk)
        bound = 3 * REL * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
        assert np.all(np.abs(got - want) <= bound + 1e-30), (use_w, use_d)
        if mk is not None:
            assert np.all(got[~mk] == 0)


@pytest.mark.parametrize("shape,mask", [((2, 6, 24, 3), None), ((3, 5, 40, 4), "random")])
def test_gradient_against_differences(shape, mask):
    """d_logits against central differences of losses64 and of the routing softmax."""
    S, T, E, k = shape
    l, _, mk = make(S, T, E, k, seed=3, mask=mask)
    lt, l = to_logits(l, "f32")
    ids = np.argsort(-l, axis=-1, kind="stable")[..., :k].astype(np.int32)
    r = RNG(5)
    dw = r.standard_normal((S, T, k)).astype(np.float32)
    d = np.array([0.9, 0.2], np.float32)

    def objective(x):
        total = float((losses64(x, ids, mk)[0] * d).sum())
        picked = np.take_along_axis(x, ids.astype(int), -1)
        ex = np.exp(picked - picked.max(-1, keepdims=True))
        w = ex / ex.sum(-1, keepdims=True)
        live = 1.0 if mk is None else mk[..., None]
        return total + float((w * dw * live).sum())

    o, _ = run_losses(lt, ids, mk)
    ids_t, w_t = i32_dev(ids), torch.empty((S, T, k), device=DEV)
    got_ids = torch.empty_like(ids_t)
    m.moe_route_topk(lt, got_ids, w_t)
    assert torch.equal(got_ids, ids_t)
    out = torch.empty_like(lt)
    m.moe_route_backward(lt, ids_t, w_t, f32_dev(dw), o["lse"], o["counts"], o["n_valid"],
                         f32_dev(d), out,
                         token_mask=None if mk is None else torch.from_numpy(mk.astype(np.uint8)).to(DEV))
    got = host(out)
    h = 1e-5   # central difference: error ~ h^2 |f'''| / 6 < 1e-9 plus 1e-16 / h of rounding
    for _ in range(60):
        at = (r.integers(S), r.integers(T), r.integers(E))
        up, down = l.copy(), l.copy()
        up[at] += h
        down[at] -= h
        want = (objective(up) - objective(down)) / (2 * h)
        assert abs(got[at] - want) <= 1e-6 + 1e-4 * abs(want), at


def test_infinities_and_masked_garbage():
    """-inf logits are probabilities of 0, a row of -inf adds only itself to n_valid, and what
    masked tokens hold (NaN, inf, ids past E) is never read."""
    S, T, E, k = 2, 40, 48, 4
    l, ids, _ = make(S, T, E, k, seed=11)
    r = RNG(2)
    l[r.random(l.shape) < 0.3] = -np.inf
    l[0, 5] = -np.inf
    l[1, 0] = -np.inf
    l[0, 7, 1:] = -np.finfo(np.float32).max
    mk = r.random((S, T)) < 0.8
    mk[0, 5] = mk[1, 0] = mk[0, 7] = True
    dirty = l.copy()
    dirty[~mk] = np.nan
    bad_ids = ids.copy()
    bad_ids[~mk] = E + 1000
    w = r.random((S, T, k)).astype(np.float32)
    dw = r.standard_normal((S, T, k)).astype(np.float32)
    dirty_w, dirty_dw = w.copy(), dw.copy()
    dirty_w[~mk] = np.nan
    dirty_dw[~mk] = np.inf
    lt, _ = to_logits(dirty, "f32")
    l = l.astype(np.float32).astype(np.float64)
    o, status = run_losses(lt, bad_ids, mk)
    assert status == 0
    with np.errstate(over="ignore"):
        losses, counts, prob, lse, n_valid = losses64(l, ids, mk)
    assert np.array_equal(host(o["counts"]), counts) and np.array_equal(host(o["n_valid"]), n_valid)
    assert np.all(np.abs(host(o["prob_mean"]) - prob) <= REL * prob)
    got = host(o["lse"]).astype(np.float64)
    assert got[0, 5] == -np.inf and got[1, 0] == -np.inf
    fin = np.isfinite(lse)
    assert np.all(np.abs(got[fin] - lse[fin]) <= REL * np.maximum(np.abs(lse[fin]), 1))
    # where the row of lowest values has no other, its lse^2 is past fp32: the loss is inf
    got = host(o["losses"])
    with np.errstate(over="ignore", invalid="ignore"):
        assert np.all((got == losses.astype(np.float32)) |
                      (np.abs(got - losses) <= 3 * REL * np.abs(losses)))
    out = torch.full((S, T, E), -7.0, device=DEV)
    d = np.array([1.0, 0.5], np.float32)
    m.moe_route_backward(lt, i32_dev(bad_ids), f32_dev(dirty_w), f32_dev(dirty_dw), o["lse"],
                         o["counts"], o["n_valid"], f32_dev(d), out,
                         token_mask=torch.from_numpy(mk.astype(np.uint8)).to(DEV))
    want, size = route_grad64(l, ids, w, dw, counts, n_valid, lse, d, mk)
    assert np.all(np.abs(host(out) - want) <= 3 * REL * size + 1e-30)


def test_ids_out_of_range_and_repeated():
    """ids < 0 are not routed, ids >= E flag the status word, repeated picks of a token add up."""
    S, T, E, k = 1, 30, 12, 5
    l, ids, _ = make(S, T, E, k, seed=4)
    ids[0, 3, 2] = -1
    ids[0, 8] = -1
    ids[0, 9] = 6
    lt, l64 = to_logits(l, "f32")
    o, status = run_losses(lt, ids, None)
    losses, counts, prob, lse, n_valid = losses64(l64, ids, None)
    assert status == 0 and np.array_equal(host(o["counts"]), counts)
    w, dw = (RNG(i).random((S, T, k)).astype(np.float32) for i in (1, 2))
    out = torch.empty_like(lt)
    d = np.array([0.5, 0.5], np.float32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_route_backward(lt, i32_dev(ids), f32_dev(w), f32_dev(dw), o["lse"], o["counts"],
                         o["n_valid"], f32_dev(d), out, dev_status=st)
    want, size = route_grad64(l64, ids, w, dw, counts, n_valid, lse, d, None)
    assert int(st.item()) == 0 and np.all(np.abs(host(out) - want) <= 3 * REL * size + 1e-30)
    ids[0, 20, 1] = E
    o, status = run_losses(lt, ids, None)
    assert status == m.status_bit(m.MOE_ERR_BAD_EXPERT_ID)
    m.moe_route_backward(lt, i32_dev(ids), f32_dev(w), f32_dev(dw), o["lse"], o["counts"],
                         o["n_valid"], f32_dev(d), out, dev_status=st)
    counts = losses64(l64, ids, None)[1]
    want, size = route_grad64(l64, ids, w, dw, counts, n_valid, lse, d, None)
    assert int(st.item()) == m.status_bit(m.MOE_ERR_BAD_EXPERT_ID)
    assert np.all(np.abs(host(out) - want) <= 3 * REL * size + 1e-30)


def test_empty_batch_and_repeats():
    lt = torch.empty((2, 0, 16), device=DEV)
    o, status = run_losses(lt, np.zeros((2, 0, 3), np.int32), None)
    assert status == 0 and not host(o["counts"]).any() and not host(o["prob_mean"]).any()
    assert not host(o["n_valid"]).any() and not host(o["losses"]).any()
    l, ids, mk = make(2, 3000, 96, 6, seed=9, mask="random")
    lt, _ = to_logits(l, "f32")
    first, _ = run_losses(lt, ids, mk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        again, _ = run_losses(lt, ids, mk, stream=stream)
        for key in first:
            assert torch.equal(first[key], again[key]), key


# ------------------------------------------------------------------ combine

def combine_case(N, k, H, share, spare, seed):
    r = RNG(seed)
    pairs = r.permutation(N * k)[:round(share * N * k)]
    rows = len(pairs) + spare
    places = r.permutation(rows)[:len(pairs)]
    pair_row = np.full(N * k, -1, np.int32)
    recv_pair = np.full(rows, -1, np.int32)
    pair_row[pairs] = places
    recv_pair[places] = pairs
    y = ms.bf16_bits_from_f32(r.standard_normal((rows, H)).astype(np.float32))
    g = ms.bf16_bits_from_f32(r.standard_normal((N, H)).astype(np.float32))
    w = r.random((N, k)).astype(np.float32)
    return y, g, w, pair_row.reshape(N, k), recv_pair


def check_combine(y, g, w, pair_row, recv_pair, S=1, use_recv=True, stream=None):
    (rows, H), (N, k) = y.shape, w.shape
    d_y = torch.full((rows, H), -7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((S, N // S, k), -7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_combine_backward(bf16_dev(g).view(S, N // S, H), bf16_dev(y), i32_dev(pair_row).view(S, N // S, k),
                           f32_dev(w).view(S, N // S, k), d_y, dw,
                           recv_pair=i32_dev(recv_pair) if use_recv else None, dev_status=st,
                           stream=stream)
    torch.cuda.synchronize()
    yf, gf = (ms.f32_from_bf16_bits(a) for a in (y, g))
    want = np.full((rows, H), 0 if use_recv else ms.bf16_bits_from_f32(np.float32([-7]))[0], np.uint16)
    dot, mag = np.zeros((N, k)), np.zeros((N, k))
    for n in range(N):
        for j in range(k):
            row = pair_row[n, j]
            if 0 <= row < rows:
                want[row] = ms.bf16_bits_from_f32(w[n, j] * gf[n])
                prod = yf[row].astype(np.float64) * gf[n]
                dot[n, j], mag[n, j] = prod.sum(), np.abs(prod).sum()
    assert np.array_equal(bf16_host(d_y), want)
    # H fp32 multiply-adds, each within 2^-24 of the partial sum's magnitude
    assert np.all(np.abs(host(dw).reshape(N, k) - dot) <= H * 2.0 ** -24 * mag)
    return int(st.item())


@pytest.mark.parametrize("N,k,H,share,spare", [
    (1, 1, 8, 1.0, 0), (128, 2, 256, 1.0, 0), (37, 6, 5120, 1.0, 3), (9, 32, 264, 1.0, 40),
    (50, 8, 1288, 0.4, 70), (20, 9, 2048, 0.125, 500), (5, 3, 16, 0.0, 10), (300, 1, 72, 1.0, 0)])
def test_combine_backward(N, k, H, share, spare):
    case = combine_case(N, k, H, share, spare, seed=N + H)
    assert check_combine(*case) == 0
    assert check_combine(*case, use_recv=False) == 0


def test_combine_backward_sources_streams_and_bad_rows():
    y, g, w, pair_row, recv_pair = combine_case(60, 4, 512, 1.0, 5, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert check_combine(y, g, w, pair_row, recv_pair, S=3, stream=None) == 0
    recv_pair[pair_row[7, 2]] = -1
    pair_row[7, 2] = len(y) + 3           # past the rows: skipped, its weight's gradient 0
    assert check_combine(y, g, w, pair_row, recv_pair) == m.status_bit(m.MOE_ERR_INVALID_ARG)


def test_combine_backward_is_the_gradient_of_combine():
    """<d_out, combine(y + h v) - combine(y - h v)> / 2h against <d_y, v> and the same for w, with
    the combine's definition in 64 bits (linear in each: the difference is exact)."""
    y, g, w, pair_row, recv_pair = combine_case(40, 6, 320, 0.8, 7, seed=2)
    d_y = torch.empty((len(y), 320), dtype=torch.bfloat16, device=DEV)
    dw = torch.empty((1, 40, 6), device=DEV)
    m.moe_combine_backward(bf16_dev(g).view(1, 40, 320), bf16_dev(y), i32_dev(pair_row).view(1, 40, 6),
                           f32_dev(w).view(1, 40, 6), d_y, dw, recv_pair=i32_dev(recv_pair))
    yf, gf = (ms.f32_from_bf16_bits(a).astype(np.float64) for a in (y, g))

    def objective(yy, ww):
        out = np.zeros_like(gf)
        for n in range(40):
            for j in range(6):
                if pair_row[n, j] >= 0:
                    out[n] += ww[n, j] * yy[pair_row[n, j]]
        return (out * gf).sum()

    r = RNG(8)
    vy, vw = r.standard_normal(yf.shape), r.standard_normal(w.shape)
    dy64 = ms.f32_from_bf16_bits(bf16_host(d_y)).astype(np.float64)
    slope = (objective(yf + vy, w) - objective(yf - vy, w)) / 2
    # each d_y is within 2^-9 of w * d_out, so the inner product within 2^-9 of its magnitudes
    assert abs((dy64 * vy).sum() - slope) <= 2.0 ** -9 * np.abs(dy64 * vy).sum()
    slope = (objective(yf, w + vw) - objective(yf, w - vw)) / 2
    got = host(dw)[0].astype(np.float64)
    assert abs((got * vw).sum() - slope) <= 1e-5 * np.abs(got * vw).sum()


def test_combine_backward_empty_batch():
    d_y = torch.full((5, 16), 3.0, dtype=torch.bfloat16, device=DEV)
    e = torch.empty
    m.moe_combine_backward(e((1, 0, 16), dtype=torch.bfloat16, device=DEV), d_y.clone(),
                           e((1, 0, 2), dtype=torch.int32, device=DEV), e((1, 0, 2), device=DEV),
                           d_y, e((1, 0, 2), device=DEV),
                           recv_pair=torch.full((5,), -1, dtype=torch.int32, device=DEV))
    assert not d_y.any()


# ------------------------------------------------------------------ refusals with GPU tensors

def test_binding_refuses_types_shapes_and_strides():
    S, T, E, k = 2, 8, 16, 2
    f = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = torch.empty(m.moe_balance_loss_workspace_bytes(S, T, E), dtype=torch.uint8, device=DEV)
    good = [f(S, T, E), i(S, T, k), i(S, E), f(S, E), f(S, T), i(S), f(2), ws]

    def refused(error, match, at, value, **kw):
        args = list(good)
        args[at] = value
        with pytest.raises(error, match=match):
            m.moe_balance_loss(*args, **kw)

    refused(TypeError, "logits: dtype", 0, f(S, T, E).double())
    refused(ValueError, "logits: expected 3 dims", 0, f(T, E))
    refused(ValueError, "logits: must be contiguous", 0, f(S, E, T).transpose(1, 2))
    refused(TypeError, "topk_ids: dtype", 1, i(S, T, k).long())
    refused(ValueError, r"topk_ids: expected shape \(2, 8, 2\), got \(2, 7, 2\)", 1, i(S, T - 1, k))
    refused(ValueError, "counts: expected shape", 2, i(S, E + 1))
    refused(ValueError, "losses: expected shape", 6, f(3))
    refused(TypeError, "ws: expected a torch.Tensor", 7, None)
    refused(ValueError, "token_mask: expected shape", 0, good[0],
            token_mask=torch.ones(S, T + 1, dtype=torch.uint8, device=DEV))
    refused(m.MoeError, "ws_bytes", 7, ws[:256])
    refused(AttributeError, "cuda_stream", 0, good[0], stream=object())
    m.moe_balance_loss(*good)
    with pytest.raises(ValueError, match="logits: needed with d_losses"):
        m.moe_route_backward(None, i(S, T, k), None, None, f(S, T), i(S, E), i(S), f(2), f(S, T, E))
    with pytest.raises(TypeError, match="logits: dtype"):      # d_logits of another type
        m.moe_route_backward(f(S, T, E), i(S, T, k), None, None, f(S, T), i(S, E), i(S), f(2),
                             f(S, T, E).bfloat16())
    with pytest.raises(m.MoeError, match="no gradient comes in"):
        m.moe_route_backward(None, i(S, T, k), None, None, None, None, None, None, f(S, T, E))
    y = torch.zeros(5, 16, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="y: expected shape"):
        m.moe_combine_backward(f(1, 3, 24).bfloat16(), y, i(1, 3, 2), f(1, 3, 2), y.clone(), f(1, 3, 2))
    with pytest.raises(ValueError, match="recv_pair: expected shape"):
        m.moe_combine_backward(f(1, 3, 16).bfloat16(), y, i(1, 3, 2), f(1, 3, 2), y.clone(), f(1, 3, 2),
                               recv_pair=i(4))
    w4 = torch.empty(m.moe_w4_bytes(2, 16, 32), dtype=torch.uint8, device=DEV)
    a = f(4, 32).bfloat16()
    out = f(4, 16).bfloat16()
    big = torch.empty(m.moe_expert_product_w4_workspace_bytes(4, 2, 16, 32), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="are not the packed weights"):
        m.moe_expert_product_w4(a, w4[:-1], f(2), out, big, expert_offsets=i(3))
    with pytest.raises(ValueError, match="expert_offsets: expected shape"):
        m.moe_expert_product_w4(a, w4, f(2), out, big, expert_offsets=i(2))
    with pytest.raises(m.MoeError, match="not both"):
        m.moe_expert_product_w4(a, w4, f(2), out, big)
