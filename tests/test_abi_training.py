"""Refusals of the training calls: bad sizes, types, pointers and alignments are rejected before
anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

import combine_moe_route_06_gb300 as m

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced: the calls are rejected first
MIS = ctypes.c_void_p((1 << 20) + 2)
NULL = ST = ctypes.c_void_p(0)
BIG = 1 << 30


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


LOSS = [FAKE, 0, 2, 64, 16, 2, FAKE, NULL, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, NULL, ST]


@pytest.mark.parametrize("changes,needle", [
    ({1: 2}, "logits_type=2"), ({2: 0}, "S=0"), ({2: 70000, 3: 1}, "S=70000"), ({3: -1}, "T=-1"),
    ({4: 2000}, "E=2000"), ({5: 17}, "E=16"), ({5: 0}, "k=0"), ({0: NULL}, "`logits`"),
    ({0: MIS}, "`logits` is not 4-byte"), ({6: NULL}, "`topk_ids`"), ({8: NULL}, "`counts`"),
    ({9: MIS}, "`prob_mean`"), ({10: NULL}, "`lse`"), ({11: NULL}, "`n_valid`"),
    ({12: NULL}, "`losses`"), ({13: NULL}, "`ws`"), ({13: ctypes.c_void_p((1 << 20) + 64)}, "256-byte"),
    ({14: 16}, "ws_bytes=16"), ({15: MIS}, "dev_status")])
def test_balance_loss_refuses(lib, changes, needle):
    refused(lib, "moe_balance_loss", LOSS, changes, needle)


def test_balance_loss_workspace(lib):
    assert m.moe_balance_loss_workspace_bytes(1, 4096, 384) % 256 == 0
    assert m.moe_balance_loss_workspace_bytes(1, 0, 384) > 0
    assert m.moe_balance_loss_workspace_bytes(1, 16, 2000) == 0
    assert m.moe_balance_loss_workspace_bytes(0, 16, 16) == 0


ROUTE = [FAKE, 0, 2, 64, 16, 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, NULL, FAKE, NULL, ST]


@pytest.mark.parametrize("changes,needle", [
    ({1: 5}, "logits_type=5"), ({3: -2}, "T=-2"), ({5: 33, 4: 64}, "k=33"),
    ({7: NULL}, "come together"), ({8: NULL}, "come together"),
    ({7: NULL, 8: NULL, 12: NULL}, "no gradient comes in"), ({6: NULL}, "`topk_ids`"),
    ({0: NULL}, "`logits`"), ({9: NULL}, "`lse`"), ({10: NULL}, "`counts`"),
    ({11: MIS}, "`n_valid`"), ({12: MIS}, "`d_losses`"), ({14: NULL}, "`d_logits`"),
    ({14: MIS}, "`d_logits` is not 4-byte"), ({15: MIS}, "dev_status")])
def test_route_backward_refuses(lib, changes, needle):
    refused(lib, "moe_route_backward", ROUTE, changes, needle)


COMBINE = [FAKE, FAKE, 64, FAKE, FAKE, FAKE, 1, 32, 2, 64, FAKE, FAKE, NULL, ST]


@pytest.mark.parametrize("changes,needle", [
    ({2: -1}, "y_rows=-1"), ({6: 0}, "S=0"), ({8: 33}, "k=33"), ({9: 12}, "H=12"), ({9: 0}, "H=0"),
    ({0: NULL}, "`d_out`"), ({0: ctypes.c_void_p((1 << 20) + 8)}, "16-byte"), ({1: NULL}, "`y`"),
    ({3: NULL}, "`pair_row`"), ({4: MIS}, "`topk_w`"), ({5: MIS}, "`recv_pair`"),
    ({10: NULL}, "`d_y`"), ({11: NULL}, "`d_topk_w`"), ({12: MIS}, "dev_status")])
def test_combine_backward_refuses(lib, changes, needle):
    refused(lib, "moe_combine_backward", COMBINE, changes, needle)


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_balance_loss(x, x.int(), x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_route_backward(x, x.int(), None, None, x, x, x, x, x)
    with pytest.raises(ValueError, match="topk_ids: needed"):
        m.moe_route_backward(x, None, x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        m.moe_combine_backward(x, x[0], x.int(), x, x[0], x)
