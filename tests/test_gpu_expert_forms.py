"""The forms of moe_expert_product_w4 that many or uneven rows take, against the product in 64 bits.

Large tiles (two weight blocks, more than 64 rows) in greater number than the SMs, so that a CTA
goes from one to the next; tiles cut between CTAs with few and many rows; parts from every CTA;
experts of one row beside one of 65; a row per CTA with more rows than CTAs.  Tolerances as in
test_gpu_expert_w4."""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
import moe_synth as ms
from test_gpu_expert_w4 import dense, make_weights, pack, product, rows_of, want_and_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()


def check(y_bits, a_bits, codes, scales, factor, gated, ranges):
    a = ms.f32_from_bf16_bits(a_bits).astype(np.float64)
    y = ms.f32_from_bf16_bits(y_bits).astype(np.float64)
    rest = np.ones(len(a), bool)
    for e, (s, c) in enumerate(ranges):
        rest[s:s + c] = False
        if c == 0:
            continue
        w = dense(codes[e:e + 1], scales[e:e + 1], factor[e:e + 1])[0]
        want, bound = want_and_bound(a[s:s + c], w, gated)
        worst = np.max(np.abs(y[s:s + c] - want) - bound)
        assert worst <= 0, (e, s, c, worst)
    assert np.all(y[rest] == -7)


FORMS = {
    # 253 and 240 large tiles, cut into shares that end inside a tile
    "large_gated": (3, 1400, 400, True, [900, 910, 890]),
    "large_plain": (3, 2560, 400, False, [900, 1024, 897]),
    # tiles of one and two chunks: the decode of the next tile runs across all of it
    "one_chunk": (2, 1408, 128, True, [1000, 1030]),
    "two_chunks": (2, 2560, 208, False, [1100, 1000]),
    # few tiles over long columns, cut in two, of 9-64 and of 65-128 rows
    "cut_64": (2, 256, 3600, True, [40, 64]),
    "cut_128": (2, 256, 3600, True, [100, 128]),
    "cut_plain": (2, 512, 3600, False, [9, 120]),
    "cut_one_block": (2, 640, 3600, False, [127, 33]),
    # a share of some 15 of 25 chunks: every CTA writes a part of a tile
    "all_parts": (8, 1280, 3152, True, [100, 70, 3, 33, 65, 9, 128, 17]),
    "all_parts_plain": (8, 2560, 3152, False, [64, 1, 128, 33, 65, 2, 97, 17]),
    "all_parts_small": (8, 1280, 3152, True, [64, 1, 40, 9, 17, 33, 48, 60]),
    # one expert of 65 rows decides the form of all
    "one_of_65": (6, 1024, 3152, True, [1, 65, 1, 0, 2, 1]),
    # about 64 rows an expert, some above
    "about_64": (24, 1000, 1040, True, [64 + (7 * e) % 23 - 11 for e in range(24)]),
    # more rows in use than CTAs that convert them, a row each
    "rows_by_cta": (2, 24, 160, False, [1500, 1900]),
    "rows_by_cta_long": (1, 16, 5136, True, [2400]),
}


@pytest.mark.parametrize("layout", ["runs", "blocks"])
@pytest.mark.parametrize("form", FORMS)
def test_forms(form, layout):
    E, N, K, gated, counts = FORMS[form]
    codes, scales, factor = make_weights(E, N * (2 if gated else 1), K, seed=len(form) + K)
    if layout == "blocks":
        block = max(counts) + 3
        rows, ranges = E * block + 5, [(e * block, c) for e, c in enumerate(counts)]
        by = dict(counts=counts, block_rows=block)
    else:
        starts = np.concatenate([[0], np.cumsum(counts)]) + 3
        rows, ranges = int(starts[-1]) + 6, [(int(s), c) for s, c in zip(starts, counts)]
        by = dict(offsets=starts)
    a, w4 = rows_of(N + K, rows, K), pack(codes, scales, gated)
    y, status = product(a, w4, factor, N, gated, **by)
    assert status == 0
    check(y, a, codes, scales, factor, gated, ranges)
    again, _ = product(a, w4, factor, N, gated, **by)
    assert np.array_equal(y, again)          # whichever part of a cut tile was last
