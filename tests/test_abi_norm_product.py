"""Refusals of the norm and of the experts' bf16 products: bad sizes, types, pointers and alignments
are rejected before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

import combine_moe_route_06_gb300 as m

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced: the calls are rejected first
MIS = ctypes.c_void_p((1 << 20) + 2)
MIS8 = ctypes.c_void_p((1 << 20) + 8)
NULL = ST = ctypes.c_void_p(0)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.load_library()


def refused(lib, fn, good, changes, needle):
    bad = list(good)
    for at, value in changes.items():
        bad[at] = value
    assert getattr(lib, fn)(*bad) == m.MOE_ERR_INVALID_ARG
    assert needle in lib.moe_last_error_message().decode()


#           a, rows, offsets, counts, block, w, E, N, K, gated, y, pre, ws, bytes, status, stream
FORWARD = [FAKE, 64, FAKE, NULL, 0, FAKE, 4, 32, 64, 1, FAKE, NULL, FAKE, BIG, NULL, ST]


@pytest.mark.parametrize("changes,needle", [
    ({1: -1}, "a_rows=-1"), ({6: 0}, "E=0"), ({6: 1025}, "E=1025"), ({7: 12}, "N=12"), ({7: 0}, "N=0"),
    ({8: 4}, "K=4"), ({8: 12}, "K=12"), ({8: (1 << 20) + 8}, "K=1048584"), ({9: 2}, "gated=2"),
    ({7: 1 << 20, 8: 1 << 20}, "too many"), ({1: 2 ** 31 - 1, 7: 1 << 16, 8: 1 << 12}, "too many"),
    ({2: NULL}, "not both"), ({3: FAKE}, "not both"), ({2: MIS}, "`expert_offsets`"),
    ({2: NULL, 3: FAKE}, "block_rows=0"), ({2: NULL, 3: FAKE, 4: 17}, "E * block_rows=68"),
    ({2: NULL, 3: MIS, 4: 1}, "`masked_counts`"), ({0: NULL}, "`a`"), ({0: MIS8}, "`a` is not 16-byte"),
    ({5: NULL}, "`w`"), ({5: MIS8}, "`w` is not 16-byte"), ({10: NULL}, "`y`"), ({11: MIS8}, "`pre`"),
    ({9: 0, 11: FAKE}, "`pre` is of gated"), ({12: NULL}, "`ws`"),
    ({12: ctypes.c_void_p((1 << 20) + 64)}, "256-byte"), ({13: 16}, "ws_bytes=16"), ({14: MIS}, "dev_status")])
def test_product_refuses(lib, changes, needle):
    refused(lib, "moe_expert_product", FORWARD, changes, needle)


#           d_y, a, rows, offsets, counts, block, w, pre, E, N, K, d_a, d_w, type, ws, bytes, status, stream
BACK = [FAKE, FAKE, 64, FAKE, NULL, 0, FAKE, NULL, 4, 32, 64, FAKE, FAKE, 0, FAKE, BIG, NULL, ST]


@pytest.mark.parametrize("changes,needle", [
    ({2: -1}, "a_rows=-1"), ({8: 0}, "E=0"), ({9: 4}, "N=4"), ({10: 20}, "K=20"), ({13: 2}, "d_w_type=2"),
    ({3: NULL}, "not both"), ({11: NULL, 12: NULL}, "neither"), ({7: FAKE, 11: NULL}, "without `d_a`"),
    ({0: NULL}, "`d_y`"), ({1: NULL}, "`a`"), ({6: NULL}, "`w`"), ({7: MIS8}, "`pre`"), ({11: MIS8}, "`d_a`"),
    ({12: MIS8}, "`d_w`"), ({14: NULL}, "`ws`"), ({15: 0}, "ws_bytes=0"), ({16: MIS}, "dev_status")])
def test_product_backward_refuses(lib, changes, needle):
    refused(lib, "moe_expert_product_backward", BACK, changes, needle)


#       x, residual, type, weight, type, rows, H, eps, residual_out, y, record, stream
NORM = [FAKE, FAKE, 1, FAKE, 0, 8, 64, 1e-6, FAKE, FAKE, FAKE, ST]


@pytest.mark.parametrize("changes,needle", [
    ({2: 3}, "residual_type=3"), ({4: -1}, "weight_type=-1"), ({5: -1}, "rows=-1"), ({5: 1 << 31}, "rows="),
    ({6: 0}, "H=0"), ({6: 20}, "H=20"), ({6: 32776}, "H=32776"), ({6: 72}, "multiple of 32"),
    ({7: 0.0}, "eps"), ({7: -1.0}, "eps"), ({7: float("nan")}, "eps"), ({7: float("inf")}, "eps"),
    ({0: NULL}, "`x`"), ({0: MIS8}, "`x` is not 16-byte"), ({1: NULL}, "without `residual`"),
    ({1: MIS8}, "`residual`"), ({3: NULL}, "`weight`"), ({3: MIS8}, "`weight`"), ({8: MIS8}, "`residual_out`"),
    ({9: NULL, 10: NULL}, "neither"), ({9: MIS8}, "`y`"), ({10: MIS}, "`record` is not 8-byte")])
def test_norm_refuses(lib, changes, needle):
    refused(lib, "moe_rms_norm", NORM, changes, needle)


#            d_y, h, type, weight, type, d_residual, rows, H, eps, d_h, d_x, d_weight, ws, bytes, stream
NORM_BACK = [FAKE, FAKE, 0, FAKE, 0, NULL, 8, 64, 1e-6, FAKE, NULL, FAKE, FAKE, BIG, ST]


@pytest.mark.parametrize("changes,needle", [
    ({2: 2}, "h_type=2"), ({4: 9}, "weight_type=9"), ({6: -4}, "rows=-4"), ({7: 4}, "H=4"), ({8: 0.0}, "eps"),
    ({0: NULL}, "`d_y`"), ({1: MIS8}, "`h`"), ({3: NULL}, "`weight`"), ({5: MIS8}, "`d_residual`"),
    ({9: NULL}, "`d_h`"), ({10: MIS8}, "`d_x`"), ({11: MIS}, "`d_weight`"), ({12: NULL}, "`ws`"),
    ({13: 8}, "ws_bytes=8")])
def test_norm_backward_refuses(lib, changes, needle):
    refused(lib, "moe_rms_norm_backward", NORM_BACK, changes, needle)


def test_workspace_sizes(lib):
    assert m.moe_expert_product_workspace_bytes(0, 1, 8, 8) % 256 == 0
    assert m.moe_expert_product_workspace_bytes(-1, 1, 8, 8) == 0
    assert m.moe_expert_product_backward_workspace_bytes(64, 0, 8, 8) == 0
    assert m.moe_rms_norm_backward_workspace_bytes(0, 64) > 0
    assert m.moe_rms_norm_backward_workspace_bytes(8, 12) == 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_rms_norm(x.bfloat16(), x[0], y=x.bfloat16())
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_rms_norm_backward(x.bfloat16(), x, x[0], x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_expert_product(x.bfloat16(), x.view(1, 4, 8).bfloat16(), x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_expert_product_backward(x, x, x, x)
    with pytest.raises(TypeError, match="w: expected a torch.Tensor"):
        m.moe_expert_product_backward(x, x, None, x)
