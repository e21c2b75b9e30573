"""moe_w4_pack and moe_expert_product_w4 against the product in 64 bits.

Tolerance.  Codes times scales are exact; a row of `a` is held with a power-of-two scale and a
step of at most 2^-38 of its largest value; a sum of K products in fp32, in any order and with
truncating adders, is off by at most 2 K u sum |a w| (u = 2^-24).  The result is rounded once to
8 bits (2^-8 covers it and the fp32 factor, exp and division of the epilogue, a few u).  For gated
weights d(silu(g) u) <= 1.1 |u| dg + |silu(g)| du, |silu'| < 1.1.
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
import moe_synth as ms
from gpu_util import DEV, bf16_dev, bf16_host, f32_dev, host, i32_dev

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b):
    b = np.asarray(b).astype(int)
    sign, ex, man = np.where(b >> 7, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (1 + man / 8) * 2.0 ** (ex - 7.0))
    return sign * np.where((b & 127) == 127, np.nan, v)


def make_weights(E, rows, K, seed):
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (E, rows, K // 2), dtype=np.uint8)
    scales = r.integers(0x28, 0x48, (E, rows, K // 16), dtype=np.uint8)
    edge = np.array([0x00, 0x01, 0x07, 0x08, 0x7e, 0xb8], np.uint8)   # 0, subnormal, 448, negative
    at = r.random(scales.shape) < 0.01
    scales[at] = r.choice(edge, at.sum())
    factor = (r.random(E) + 0.5).astype(np.float32) / 16
    return codes, scales, factor


def dense(codes, scales, factor):
    E, rows, half = codes.shape
    w = np.empty((E, rows, 2 * half))
    w[..., 0::2] = E2M1[codes & 15]
    w[..., 1::2] = E2M1[codes >> 4]
    return w * np.repeat(e4m3(scales), 16, axis=-1) * factor[:, None, None].astype(np.float64)


def pack(codes, scales, gated):
    E, rows, half = codes.shape
    N = rows // 2 if gated else rows
    w4 = torch.full((m.moe_w4_bytes(E, N, 2 * half, gated),), 0xAB, dtype=torch.uint8, device=DEV)
    m.moe_w4_pack(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), w4, gated=gated)
    return w4


def product(a_bits, w4, factor, N, gated, offsets=None, counts=None, block_rows=0, stream=None,
            ws=None):
    rows, K = a_bits.shape
    E = len(factor)
    y = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device=DEV)
    past = None
    if ws is None:   # a workspace of just the size asked for, with a mebibyte behind it to watch
        need = m.moe_expert_product_w4_workspace_bytes(rows, E, N, K)
        whole = torch.full((need + (1 << 20),), 0xff, dtype=torch.uint8, device=DEV)
        ws, past = whole[:need], whole[need:]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_expert_product_w4(bf16_dev(a_bits), w4, f32_dev(factor), y, ws, gated=gated,
                            expert_offsets=None if offsets is None else i32_dev(offsets),
                            masked_counts=None if counts is None else i32_dev(counts),
                            block_rows=block_rows, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert past is None or bool((past == 0xff).all())
    return bf16_host(y), int(st.item())


def want_and_bound(a, w, gated):
    K = a.shape[1]
    out, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    step = 2.0 ** -38 * np.abs(a).max(1, keepdims=True) * np.abs(w).sum(1)[None, :]
    err = 2 * K * 2.0 ** -24 * mag + step
    if gated:
        n = out.shape[1] // 2
        g, u = out[:, :n], out[:, n:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        err = 1.1 * np.abs(u) * err[:, :n] + np.abs(silu) * err[:, n:] + 1.1 * err[:, :n] * err[:, n:]
        out = silu * u
    return out, err + 2.0 ** -8 * np.abs(out)


def check(y_bits, a_bits, codes, scales, factor, gated, ranges):
    """Every expert's rows against the definition; every other row untouched."""
    a = ms.f32_from_bf16_bits(a_bits).astype(np.float64)
    y = ms.f32_from_bf16_bits(y_bits).astype(np.float64)
    w = dense(codes, scales, factor)
    rest = np.ones(len(a), bool)
    for e, (s, c) in enumerate(ranges):
        if c == 0:
            continue
        rest[s:s + c] = False
        want, bound = want_and_bound(a[s:s + c], w[e], gated)
        worst = np.max(np.abs(y[s:s + c] - want) - bound)
        assert worst <= 0, (e, s, c, worst)
    assert np.all(y[rest] == -7)


def rows_of(seed, rows, K, scale=1.0):
    r = np.random.default_rng(seed)
    return ms.bf16_bits_from_f32((r.standard_normal((rows, K)) * scale).astype(np.float32))


gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()


CASES = [  # E, N, K, gated, counts
    (1, 8, 16, False, [1]), (1, 8, 16, True, [1]), (1, 128, 128, False, [1]), (1, 64, 128, True, [3]),
    (3, 72, 144, True, [0, 5, 1]), (5, 136, 400, False, [2, 0, 17, 0, 9]), (2, 256, 2048, True, [1, 1]),
    (4, 328, 1040, True, [16, 15, 0, 33]), (1, 640, 5120, False, [1]), (2, 96, 272, False, [129, 64]),
    (3, 200, 512, True, [300, 1, 128]), (2, 520, 96, False, [513, 127]), (64, 40, 64, True, [3, 0] * 32),
    (1, 1000, 3600, True, [7]), (6, 24, 7168, False, [1, 0, 0, 2, 8, 1]), (2, 1600, 256, True, [260, 90]),
    (3, 40, 96, False, [2100, 0, 2400]), (2, 24, 2320, True, [2060, 2050])]


@gpu
@pytest.mark.parametrize("E,N,K,gated,counts", CASES)
@pytest.mark.parametrize("layout", ["runs", "padded", "blocks"])
def test_product(E, N, K, gated, counts, layout):
    codes, scales, factor = make_weights(E, N * (2 if gated else 1), K, seed=E + N + K)
    if layout == "blocks":
        block = max(counts) + 3
        rows, ranges = E * block + 5, [(e * block, c) for e, c in enumerate(counts)]
    else:   # runs of the counts, or of counts rounded up to 8 after 3 rows of others
        runs = counts if layout == "runs" else [-(-c // 8) * 8 for c in counts]
        starts = np.concatenate([[0], np.cumsum(runs)]) + (0 if layout == "runs" else 3)
        rows, ranges = int(starts[-1]) + 6, [(int(s), c) for s, c in zip(starts, runs)]
    a = rows_of(N + K, rows, K)
    w4 = pack(codes, scales, gated)
    if layout == "blocks":
        y, status = product(a, w4, factor, N, gated, counts=counts, block_rows=block)
    else:
        y, status = product(a, w4, factor, N, gated, offsets=starts)
    assert status == 0
    check(y, a, codes, scales, factor, gated, ranges)


@gpu
def test_many_experts():
    E, N, K = 1024, 16, 48
    r = np.random.default_rng(0)
    counts = r.integers(0, 3, E)
    counts[1023] = 150
    codes, scales, factor = make_weights(E, N, K, seed=1)
    starts = np.concatenate([[0], np.cumsum(counts)])
    a = rows_of(2, int(starts[-1]), K)
    y, status = product(a, pack(codes, scales, False), factor, N, False, offsets=starts)
    assert status == 0
    check(y, a, codes, scales, factor, False, [(int(s), int(c)) for s, c in zip(starts, counts)])


@gpu
@pytest.mark.parametrize("gated", [False, True])
def test_row_magnitudes_and_nan(gated):
    """Rows of every magnitude keep their own precision, zero rows give zeros, and a row with a NaN
    or an infinity spoils no other."""
    E, N, K = 2, 136, 320
    codes, scales, factor = make_weights(E, N * (2 if gated else 1), K, seed=5)
    scales[scales == 0x7e] = 0x38
    counts = [14, 9]
    a = rows_of(6, 23, K)
    # the largest outputs stay finite: |y| <= ~1e2 * size (gated: its square)
    sizes = np.array([1, 1e15, 1e-15, 3e-39, 0, 1e-30, 1e12, 1] if gated else
                     [1, 1e30, 1e-30, 3e-39, 0, 1e-36, 1e20, 1])
    f = ms.f32_from_bf16_bits(a).astype(np.float64) * np.resize(sizes, 23)[:, None]
    f[12, 7] *= 2.0 ** 20                    # one value far above the rest of its row
    a = ms.bf16_bits_from_f32(f.astype(np.float32))
    a[3 + 8, 100] = ms.bf16_bits_from_f32(np.float32([np.nan]))[0]
    a[16, 33] = ms.bf16_bits_from_f32(np.float32([np.inf]))[0]
    starts = np.concatenate([[0], np.cumsum(counts)])
    y, status = product(a, pack(codes, scales, gated), factor, N, gated, offsets=starts)
    assert status == 0
    af, yf = (ms.f32_from_bf16_bits(v).astype(np.float64) for v in (a, y))
    w = dense(codes, scales, factor)
    for r in range(23):
        e = int(r >= 14)
        if r in (11, 16):
            assert not np.isfinite(yf[r]).any() if r == 11 else not np.isfinite(yf[r]).all()
            continue
        want, bound = want_and_bound(af[r:r + 1], w[e], gated)
        # below the normal range of bf16 a result has a step of 2^-133
        assert np.all(np.abs(yf[r] - want[0]) <= bound[0] + 2.0 ** -133), r


@gpu
@pytest.mark.parametrize("size,factor", [(1e36, 1e-5), (1e-33, 1e4)])
def test_sums_past_the_range_of_their_factors(size, factor):
    """Sums that would leave fp32 before the expert's factor brings them back."""
    E, N, K = 1, 24, 256
    codes, scales, _ = make_weights(E, N, K, seed=21)
    scales[:] = 0x7e if size > 1 else 0x08      # 448 and 2^-6
    factor = np.array([factor], np.float32)
    a = rows_of(22, 5, K, size)
    y, status = product(a, pack(codes, scales, False), factor, N, False, offsets=[0, 5])
    assert status == 0
    check(y, a, codes, scales, factor, False, [(0, 5)])


@gpu
def test_bad_row_ranges_are_cut_and_flagged():
    E, N, K = 3, 32, 64
    codes, scales, factor = make_weights(E, N, K, seed=8)
    w4 = pack(codes, scales, False)
    a = rows_of(9, 20, K)
    flag = m.status_bit(m.MOE_ERR_INVALID_ARG)
    for offsets, ranges in (([0, 5, 5, 40], [(0, 5), (5, 0), (5, 15)]),
                            ([0, 8, 4, 20], [(0, 8), (0, 0), (4, 16)]),
                            ([-3, 2, 6, 30], [(0, 0), (2, 4), (6, 14)]),
                            ([50, 60, 60, 60], [(0, 0)] * 3)):
        y, status = product(a, w4, factor, N, False, offsets=offsets)
        assert status == flag
        # expert 1 of the second list ends before it starts; its rows are the others' or none
        if offsets[1] <= offsets[2]:
            check(y, a, codes, scales, factor, False, ranges)
    y, status = product(a, w4, factor, N, False, counts=[7, 2, 6], block_rows=6)
    assert status == flag
    check(y, a, codes, scales, factor, False, [(0, 6), (6, 2), (12, 6)])
    y, status = product(a, w4, factor, N, False, counts=[-1, 2, 0], block_rows=6)
    assert status == flag
    check(y, a, codes, scales, factor, False, [(0, 0), (6, 2), (12, 0)])


@gpu
@pytest.mark.parametrize("spare", [0, 700])
def test_falling_offsets(spare):
    """Offsets that fall are flagged; what is in no run of theirs is not written."""
    E, N, K = 4, 40, 96
    codes, scales, factor = make_weights(E, N, K, seed=12)
    a = rows_of(13, 60 + spare, K)
    y, status = product(a, pack(codes, scales, False), factor, N, False, offsets=[2, 20, 50, 4, 30])
    assert status == m.status_bit(m.MOE_ERR_INVALID_ARG)
    y = ms.f32_from_bf16_bits(y)
    assert np.all(y[:2] == -7) and np.all(y[50:] == -7)


@gpu
def test_empty_calls():
    codes, scales, factor = make_weights(2, 32, 64, seed=8)
    w4 = pack(codes, scales, False)
    y, status = product(rows_of(1, 6, 64), w4, factor, 32, False, offsets=[0, 0, 0])
    assert status == 0 and np.all(ms.f32_from_bf16_bits(y) == -7)
    y, status = product(np.zeros((0, 64), np.uint16), w4, factor, 32, False, offsets=[0, 0, 0])
    assert status == 0 and y.size == 0


@gpu
def test_repeats_streams_and_one_workspace():
    """The same bytes on every run, on another stream, and with one workspace for calls of several
    shapes in a row."""
    ws = torch.full((m.moe_expert_product_w4_workspace_bytes(700, 4, 1000, 2048),), 0xff,
                    dtype=torch.uint8, device=DEV)
    runs = []
    for N, K, gated, counts in ((1000, 2048, True, [3, 0, 1, 0]), (264, 1040, False, [1, 2, 300, 3]),
                                (40, 64, False, [1, 0, 0, 0])):
        codes, scales, factor = make_weights(4, N * (2 if gated else 1), K, seed=N)
        starts = np.concatenate([[0], np.cumsum(counts)])
        a = rows_of(3, int(starts[-1]), K)
        need = m.moe_expert_product_w4_workspace_bytes(len(a), 4, N, K)
        assert need <= ws.numel()
        w4 = pack(codes, scales, gated)
        first, _ = product(a, w4, factor, N, gated, offsets=starts)
        check(first, a, codes, scales, factor, gated, [(int(s), c) for s, c in zip(starts, counts)])
        runs.append((a, w4, factor, N, gated, starts, first))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, None):
        for a, w4, factor, N, gated, starts, first in runs:
            y, status = product(a, w4, factor, N, gated, offsets=starts, ws=ws, stream=stream)
            assert status == 0 and np.array_equal(y, first)


@gpu
def test_graph_capture_follows_new_counts():
    """A captured call reads the counts of each replay."""
    E, N, K, block = 3, 136, 256, 40
    codes, scales, factor = make_weights(E, 2 * N, K, seed=4)
    w4, a = pack(codes, scales, True), rows_of(5, E * block, K)
    at, ft = bf16_dev(a), f32_dev(factor)
    y = torch.full((E * block, N), -7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(m.moe_expert_product_w4_workspace_bytes(E * block, E, N, K), dtype=torch.uint8,
                     device=DEV)
    counts = i32_dev([1, 1, 1])
    call = lambda: m.moe_expert_product_w4(at, w4, ft, y, ws, masked_counts=counts,  # noqa: E731
                                           block_rows=block, gated=True)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for now in ([1, 0, 2], [40, 17, 0], [0, 0, 0], [5, 33, 40]):
        counts.copy_(i32_dev(now))
        y.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        check(bf16_host(y), a, codes, scales, factor, True, [(e * block, c) for e, c in enumerate(now)])


# ------------------------------------------------------------------ refusals (no GPU)

FAKE = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 2)
NULL = ST = ctypes.c_void_p(0)
BIG = 1 << 40


def refused(fn, good, changes, needle):
    lib = m.load_library()
    bad = list(good)
    for at, value in changes.items():
        bad[at] = value
    assert getattr(lib, fn)(*bad) == m.MOE_ERR_INVALID_ARG
    assert needle in lib.moe_last_error_message().decode()


PACK = [FAKE, FAKE, 4, 64, 128, 0, FAKE, BIG, ST]


@pytest.mark.parametrize("changes,needle", [
    ({0: NULL}, "`codes`"), ({0: ctypes.c_void_p((1 << 20) + 4)}, "8-byte"), ({1: NULL}, "`scales`"),
    ({2: 0}, "E=0"), ({2: 1025}, "E=1025"), ({3: 12}, "N=12"), ({3: 0}, "N=0"), ({4: 24}, "K=24"),
    ({4: 0}, "K=0"), ({5: 2}, "gated=2"), ({6: NULL}, "`w4`"),
    ({6: ctypes.c_void_p((1 << 20) + 8)}, "16-byte"), ({7: 100}, "w4_size=100")])
def test_pack_refuses(changes, needle):
    refused("moe_w4_pack", PACK, changes, needle)


PRODUCT = [FAKE, 64, FAKE, NULL, 0, FAKE, FAKE, 4, 64, 128, 0, FAKE, FAKE, BIG, NULL, ST]


@pytest.mark.parametrize("changes,needle", [
    ({0: NULL}, "`a`"), ({0: ctypes.c_void_p((1 << 20) + 8)}, "16-byte"), ({1: -1}, "a_rows=-1"),
    ({2: NULL}, "not both"), ({3: FAKE, 4: 8}, "not both"), ({2: MIS}, "`expert_offsets`"),
    ({2: NULL, 3: FAKE}, "block_rows=0"), ({2: NULL, 3: FAKE, 4: 17}, "E * block_rows=68"),
    ({2: NULL, 3: MIS, 4: 16}, "`masked_counts`"), ({5: NULL}, "`w4`"), ({6: NULL}, "`w_factor`"),
    ({7: 2000}, "E=2000"), ({8: 4}, "N=4"), ({9: 8}, "K=8"), ({10: -1}, "gated=-1"),
    ({11: NULL}, "`y`"), ({12: NULL}, "`ws`"), ({13: 0}, "ws_bytes=0"), ({14: MIS}, "dev_status")])
def test_product_refuses(changes, needle):
    refused("moe_expert_product_w4", PRODUCT, changes, needle)


def test_sizes():
    assert m.moe_w4_bytes(1, 128, 128) == 9216
    assert m.moe_w4_bytes(2, 136, 144) == 2 * 2 * 2 * 9216
    assert m.moe_w4_bytes(1, 64, 128, True) == 2 * 9216
    assert m.moe_w4_bytes(1, 136, 128, True) == 4 * 9216
    with pytest.raises(m.MoeError, match="K=24"):
        m.moe_w4_bytes(1, 64, 24)
    assert m.moe_expert_product_w4_workspace_bytes(64, 4, 64, 128) > 0
    assert m.moe_expert_product_w4_workspace_bytes(-1, 4, 64, 128) == 0
    with pytest.raises(ValueError, match="CUDA tensor"):
        x = torch.zeros(4, 64, dtype=torch.uint8)
        m.moe_w4_pack(x[None], x[None], x)
