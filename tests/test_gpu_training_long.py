"""The training calls at lengths where their kernels go round their loops: several rows a warp,
several tokens a CTA, more rows than the resident CTAs take at once.  Definitions in 64 bits,
vectorised.

Tolerances, in units u = 2^-24.  With D the largest distance of a logit from its row's maximum, a
term exp(l - max) is off by D (the rounded argument) plus 2 (2 + 1.18 D) (CUDA's bound of the fast
exp, 2 + floor(1.173 D) units of 2^-23); a row's sum by that and E/32 + 5 additions; a probability
by both and 4 for the reciprocal and the product.  A mean over n tokens adds the longest chain of
additions: a lane's rows, its CTA's warps, a warp's parts, the last eight.  All terms are positive,
so these are relative.  lse is off by u |lse|, 2 u |log sum| and the sum's relative error."""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
import moe_synth as ms
from gpu_util import bf16_dev, bf16_host, f32_dev, host, i32_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()


def error_units(l):
    E = l.shape[-1]
    D = float((l.max(-1, keepdims=True) - l).max())
    term = D + 2 * (2 + 1.18 * D)
    row = term + E / 32 + 5
    return term, row, term + row + 4


def chain_units(S, T):
    """Additions behind a mean: at least 8 warps a CTA and two rows a warp or 304 CTAs in all."""
    parts = max(1, min((T + 15) // 16, 304 // S))
    return -(-T // (8 * parts)) + 16 + -(-parts // 8) + 8 + 4


LONG = [(4, 5000, 40, 4, True), (1, 20000, 24, 2, True), (8, 4096, 384, 6, True), (1, 4096, 128, 8, False),
        (1, 100003, 24, 2, True), (1, 20011, 33, 3, False), (2, 9001, 200, 32, True)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,T,E,k,masked", LONG)
def test_losses_and_gradient(S, T, E, k, masked, dtype):
    r = np.random.default_rng(T + E)
    lt = torch.from_numpy(r.standard_normal((S, T, E), np.float32)).to(DEV)
    lt = lt if dtype == "f32" else lt.bfloat16()
    l = lt.double().cpu().numpy()
    ids = r.integers(0, E, (S, T, k)).astype(np.int32)
    mask = r.random((S, T)) < 0.6 if masked else np.ones((S, T), bool)
    mt = torch.from_numpy(mask.astype(np.uint8)).to(DEV) if masked else None
    o = {"counts": torch.full((S, E), -7, dtype=torch.int32, device=DEV),
         "prob": torch.full((S, E), -7.0, device=DEV), "lse": torch.full((S, T), -7.0, device=DEV),
         "n": torch.full((S,), -7, dtype=torch.int32, device=DEV),
         "losses": torch.full((2,), -7.0, device=DEV)}
    ws = torch.full((m.moe_balance_loss_workspace_bytes(S, T, E),), 0xff, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids_t = i32_dev(ids)
    m.moe_balance_loss(lt, ids_t, o["counts"], o["prob"], o["lse"], o["n"], o["losses"], ws,
                       token_mask=mt, dev_status=st)
    # the definition
    valid = mask[..., None].astype(np.float64)
    n = mask.sum(1)
    top = l.max(-1, keepdims=True)
    ex = np.exp(l - top)
    sums = ex.sum(-1, keepdims=True)
    p = ex / sums
    lse = np.where(mask, (top + np.log(sums))[..., 0], 0)
    prob = (p * valid).sum(1) / n[:, None]
    counts = np.stack([np.bincount(ids[s][mask[s]].ravel(), minlength=E) for s in range(S)])
    balance = np.mean([E / (k * n[s]) * (counts[s] * prob[s]).sum() for s in range(S)])
    z = np.mean((lse ** 2).sum(1) / n)
    assert int(st.item()) == 0
    assert np.array_equal(host(o["counts"]), counts) and np.array_equal(host(o["n"]), n)
    term, row, one = error_units(l)
    chain = chain_units(S, T)
    mean = (one + chain) * U
    assert np.all(np.abs(host(o["prob"]) - prob) <= mean * prob)
    e_lse = U * (np.abs(lse) + 2 * np.abs(np.log(sums[..., 0])) + row + 2)
    assert np.all(np.abs(host(o["lse"]) - lse)[mask] <= e_lse[mask])
    assert np.all(host(o["lse"])[~mask] == 0)
    got = host(o["losses"]).astype(np.float64)
    # counts times means, summed over E, then over S: E/32 + 10 + S/32 + 5 additions and 6 products
    assert abs(got[0] - balance) <= (mean + (E / 32 + S / 32 + 21) * U) * balance
    e_z = np.mean(((2 * np.abs(lse) * e_lse + e_lse ** 2) * mask).sum(1) / n)
    assert abs(got[1] - z) <= e_z + (chain + 10 + S / 32) * U * z

    w, dw = r.random((S, T, k)).astype(np.float32), r.standard_normal((S, T, k)).astype(np.float32)
    d_t = f32_dev([0.7, -0.3])
    d = d_t.double().cpu().numpy()
    out = torch.full((S, T, E), -7.0, device=DEV, dtype=lt.dtype)
    A = (d[0] * E * counts / (k * S * n[:, None].astype(np.float64) ** 2))[:, None, :]
    zc = (2 * d[1] * lse / (S * n[:, None]))[..., None]
    loss = p * (A - (A * p).sum(-1, keepdims=True) + zc)
    # every term of the bracket to E/32 + 12 roundings and the error of its probabilities
    loss_err = U * p * ((2 * one + E / 32 + 12) * (np.abs(A) + (A * p).sum(-1, keepdims=True)) +
                        (one + 12) * np.abs(zc)) \
        + p * np.abs(2 * d[1] / (S * n[:, None]) * e_lse)[..., None]
    dot = (w.astype(np.float64) * dw).sum(-1, keepdims=True)
    g, mag = w * (dw - dot), np.abs(w) * (np.abs(dw) + (np.abs(w.astype(np.float64) * dw)).sum(-1, keepdims=True))
    at = (np.arange(S)[:, None, None], np.arange(T)[None, :, None], ids)
    part, part_err = np.zeros_like(l), np.zeros_like(l)
    np.add.at(part, at, g)
    np.add.at(part_err, at, (k + 12) * U * mag)
    for use_w, use_d in ((True, True), (True, False), (False, True)):
        m.moe_route_backward(lt, ids_t, f32_dev(w) if use_w else None, f32_dev(dw) if use_w else None,
                             o["lse"], o["counts"], o["n"], d_t if use_d else None, out,
                             token_mask=mt, dev_status=st)
        got = out.double().cpu().numpy()
        want = (loss if use_d else 0) + (part if use_w else 0)
        err = (loss_err if use_d else 0) + (part_err if use_w else 0) + 2 * U * np.abs(want)
        want = want * valid
        if dtype == "bf16":
            err = err + 2.0 ** -8 * (np.abs(want) + err)
        assert np.all(np.abs(got - want)[mask] <= (err + 1e-38)[mask]), (use_w, use_d)
        assert np.all(got[~mask] == 0)
    assert int(st.item()) == 0


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("N,k,H,share,spare", [
    # one warp a token, tokens handed out as warps come free
    (5000, 2, 64, 1.0, 100), (20003, 8, 24, 0.125, 1000), (20003, 2, 40, 1.0, 7), (5000, 8, 136, 1.0, 3),
    (30011, 32, 8, 0.2, 0),
    # a CTA a token, several tokens a CTA; two rows at a time where tokens have few
    (400, 6, 2048, 1.0, 9), (1200, 8, 2056, 0.9, 40), (37, 2, 2048, 1.0, 5), (1100, 2, 2304, 1.0, 0),
    (700, 8, 2048, 0.125, 300), (64, 1, 5120, 1.0, 2000),
    # far more rows than tokens have: padding
    (64, 2, 256, 1.0, 4000), (0, 2, 64, 1.0, 5000)])
def test_combine_backward(N, k, H, share, spare):
    r = np.random.default_rng(N + H)
    pairs = r.permutation(N * k)[:round(share * N * k)]
    rows = len(pairs) + spare
    places = r.permutation(rows)[:len(pairs)]
    pair_row, recv_pair = np.full(N * k, -1, np.int32), np.full(rows, -1, np.int32)
    pair_row[pairs], recv_pair[places] = places, pairs
    y = ms.bf16_bits_from_f32(r.standard_normal((rows, H), np.float32))
    g = ms.bf16_bits_from_f32(r.standard_normal((N, H), np.float32))
    w = r.random((N, k)).astype(np.float32)
    # the definition; one rounding of w * d_out, H fp32 multiply-adds
    gf = ms.f32_from_bf16_bits(g)
    token, weight = recv_pair[places] // k, w.reshape(-1)[recv_pair[places]]
    want = np.zeros((rows, H), np.uint16)
    want[places] = ms.bf16_bits_from_f32(weight[:, None] * gf[token])
    prod = ms.f32_from_bf16_bits(y[places]).astype(np.float64) * gf[token]
    dot, mag = np.zeros(N * k), np.zeros(N * k)
    dot[pairs], mag[pairs] = prod.sum(1), np.abs(prod).sum(1)
    args = (bf16_dev(g).view(1, N, H), bf16_dev(y), i32_dev(pair_row).view(1, N, k),
            f32_dev(w).view(1, N, k))
    for use_recv in (True, False):
        d_y = torch.full((rows, H), -7.0, dtype=torch.bfloat16, device=DEV)
        dw = torch.full((1, N, k), -7.0, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        m.moe_combine_backward(*args, d_y, dw, recv_pair=i32_dev(recv_pair) if use_recv else None,
                               dev_status=st)
        if not use_recv:
            want[recv_pair < 0] = ms.bf16_bits_from_f32(np.float32([-7]))[0]
        assert np.array_equal(bf16_host(d_y), want)
        assert np.all(np.abs(host(dw).reshape(-1) - dot) <= H * U * mag)
        assert int(st.item()) == 0


def test_gradients_on_another_stream():
    """The same bytes on a stream that is not the current one."""
    r = np.random.default_rng(1)
    S, T, E, k, H = 2, 700, 48, 4, 256
    N = S * T
    lt = f32_dev(r.standard_normal((S, T, E), np.float32))
    ids, w = i32_dev(r.integers(0, E, (S, T, k))), f32_dev(r.random((S, T, k), np.float32))
    dw_in, lse = f32_dev(r.standard_normal((S, T, k), np.float32)), torch.logsumexp(lt, -1)
    counts, n, d = i32_dev(r.integers(0, 99, (S, E))), i32_dev([T, T]), f32_dev([0.7, -0.3])
    y, g = (torch.randn(rows, H, device=DEV).bfloat16() for rows in (N * k, N))
    pair_row = torch.randperm(N * k, device=DEV).int().view(S, T, k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = []
    for stream in (None, side):
        out, d_y, dw = torch.full_like(lt, -7), torch.full_like(y, -7), torch.full_like(w, -7)
        torch.cuda.synchronize()
        m.moe_route_backward(lt, ids, w, dw_in, lse, counts, n, d, out, stream=stream)
        m.moe_combine_backward(g.view(S, T, H), y, pair_row, w, d_y, dw, stream=stream)
        torch.cuda.synchronize()
        results.append((out, d_y, dw))
    for one, other in zip(*results):
        assert torch.equal(one, other) and not bool((one == -7).all())
