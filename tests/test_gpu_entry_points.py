"""The compiled entry points: arguments that do not fit are refused before anything is enqueued,
and other Python threads run while a call enqueues."""
import sys
import threading

import pytest
import torch

import combine_moe_route_06_gb300 as m

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()


def product_args(E=2, N=16, K=32, block=4):
    """Zero rows and weights, big enough in either layout of the weights."""
    rows = E * block
    zeros = lambda *s, **kw: torch.zeros(s, device="cuda", **kw)  # noqa: E731
    ws = torch.empty(m.moe_expert_product_w4_workspace_bytes(rows, E, N, K), dtype=torch.uint8,
                     device="cuda")
    y = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device="cuda")
    w4 = zeros(m.moe_w4_bytes(E, N, K, True), dtype=torch.uint8)
    return (zeros(rows, K, dtype=torch.bfloat16), w4, torch.ones(E, device="cuda"), y, ws), \
        dict(masked_counts=torch.full((E,), block, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("block", [2 ** 32 + 4, 4 - 2 ** 32, 2 ** 31, -2 ** 31 - 1, 2 ** 70, -2 ** 70])
def test_block_rows_past_32_bits_are_refused(block):
    args, kw = product_args()
    with pytest.raises(ValueError, match="block_rows"):
        m.moe_expert_product_w4(*args, block_rows=block, **kw)
    torch.cuda.synchronize()
    assert bool((args[3] == 3).all())
    m.moe_expert_product_w4(*args, block_rows=4, **kw)
    assert not args[3].any()


class Unclear:
    """Neither true nor false."""

    def __bool__(self):
        raise RuntimeError("unclear")


def test_an_error_of_the_gated_argument_is_passed_on():
    args, kw = product_args()
    with pytest.raises(RuntimeError, match="unclear"):
        m.moe_expert_product_w4(*args, block_rows=4, gated=Unclear(), **kw)
    codes = torch.zeros((2, 32, 16), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 32, 2), dtype=torch.uint8, device="cuda")
    w4 = torch.full((m.moe_w4_bytes(2, 32, 32),), 7, dtype=torch.uint8, device="cuda")
    with pytest.raises(RuntimeError, match="unclear"):
        m.moe_w4_pack(codes, scales, w4, gated=Unclear())
    torch.cuda.synchronize()
    assert bool((args[3] == 3).all()) and bool((w4 == 7).all())


def test_other_threads_run_while_a_call_enqueues():
    """With a switch interval longer than the test a thread gets the interpreter only from one that
    gives it up, which the loop below does nowhere but inside the call."""
    S, T, E, k = 2, 256, 64, 4
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(m.moe_balance_loss_workspace_bytes(S, T, E), dtype=torch.uint8, device="cuda")
    args = [f(S, T, E), i(S, T, k), i(S, E), f(S, E), f(S, T), i(S), f(2), ws]
    m.moe_balance_loss(*args)
    torch.cuda.synchronize()
    go, ready, ran = threading.Lock(), threading.Event(), []

    def other():
        ready.set()
        go.acquire()
        ran.append(True)

    go.acquire()
    thread = threading.Thread(target=other, daemon=True)
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1000)
    try:
        thread.start()
        ready.wait()
        go.release()
        for _ in range(6000):
            m.moe_balance_loss(*args)
            if ran:
                break
        there = bool(ran)
    finally:
        sys.setswitchinterval(interval)
    thread.join(10)
    torch.cuda.synchronize()
    assert there
