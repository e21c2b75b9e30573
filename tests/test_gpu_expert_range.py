"""moe_expert_product_w4 where parts of a result leave fp32 though the result does not: exp(-gate)
of low gates, and large factors.

Low gates: the sums are exact (one product each), so what is left is the epilogue: the exp of half the
gate, which enters squared, is off by the rounding of its argument, |gate| 2^-24, and by a fast
exp's few 2^-23, the rest by a fast reciprocal and four products: together below 2^-14 for
|gate| <= 120.  The rounding to bf16 is 2^-9, so 2^-8 covers both.  Results below bf16's normal
range have a step of 2^-133.  Factors: tolerances as in test_gpu_expert_w4."""
import numpy as np
import pytest
import torch

import combine_moe_route_06_gb300 as m
import moe_synth as ms
from test_gpu_expert_w4 import check, make_weights, pack, product, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()


def test_low_gates_keep_their_precision():
    gates = np.array([-120, -100, -95, -89, -88.5, -88, -87.5, -87, -86, -60, -1, 0, 1, 60, 88, 120.])
    ups = np.array([1., -3, 2.0 ** 10, 2.0 ** 20])
    N, K = 8, 16
    codes = np.zeros((1, 2 * N, K // 2), np.uint8)
    codes[0, :N, 0] = 0x02                       # gate: 1.0 times column 0
    codes[0, N:, 0] = 0x20                       # up: 1.0 times column 1
    scales = np.full((1, 2 * N, 1), 0x38, np.uint8)
    a = np.zeros((len(gates) * len(ups), K), np.float32)
    a[:, 0], a[:, 1] = np.repeat(gates, len(ups)), np.tile(ups, len(gates))
    bits = ms.bf16_bits_from_f32(a)
    assert np.array_equal(ms.f32_from_bf16_bits(bits), a)
    y, status = product(bits, pack(codes, scales, True), np.ones(1, np.float32), N, True,
                        offsets=[0, len(a)])
    assert status == 0
    g, u = a[:, :1].astype(np.float64), a[:, 1:2].astype(np.float64)
    want = g / (1 + np.exp(-g)) * u
    got = ms.f32_from_bf16_bits(y).astype(np.float64)
    worst = np.abs(got - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -133
    assert np.all(worst <= 0), (g[(worst > 0).any(1), 0], got[(worst > 0).any(1), 0])


@pytest.mark.parametrize("size,factor", [(1e-37, 1e35), (1e-35, -3e37), (1e-30, 1e34), (2e-38, 3e38),
                                         (1e35, 1e-30), (1e37, 1e-38)])
@pytest.mark.parametrize("rows", [5, 150])
def test_factors_of_any_size(size, factor, rows):
    """Results in range whatever the factor's share of them."""
    E, N, K = 1, 24, 256
    codes, scales, _ = make_weights(E, N, K, seed=31)
    factor = np.array([factor], np.float32)
    a = rows_of(32, rows, K, size)
    y, status = product(a, pack(codes, scales, False), factor, N, False, offsets=[0, rows])
    assert status == 0
    check(y, a, codes, scales, factor, False, [(0, rows)])
